"""Dropout, the residual's norm and the microscaled 4-bit operators on the host: the
references' own checks, and refusals of the C ABI, none of which launches a kernel."""
import numpy as np
import pytest
import torch

import __graft_entry__
import branch_ref
from row_wise_softmax_warp_gb300 import binding
from test_abi_host import A, ALIAS, ALIGN, B, C, D, E, F, G, H, NULL, OK, SHAPE, W, WORKSPACE

F32, F16, BF16, E4M3, E2M1 = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    lib = binding.library()
    before = lib.rowops_kernel_launches()
    yield lib
    assert lib.rowops_kernel_launches() == before


def test_philox_known_answers():
    """The published vectors of the generator (Random123, kat_vectors)."""
    ones = 0xFFFFFFFF
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((ones,) * 4, (ones,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
             (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        assert tuple(int(v) for v in branch_ref.philox(key, [counter])[0]) == want


def test_kept_share():
    """A share of 0.3 of 2^18 values drops, off by less than six standard deviations."""
    k = branch_ref.kept((5, -7), 64, 4096, 0.3)
    n = k.size
    assert abs((~k).sum() - 0.3 * n) < 6 * (0.21 * n) ** 0.5


def test_gradient_of_the_reference():
    """add_norm_bwd against central differences of add_norm in 64 bits."""
    rng = np.random.default_rng(0)
    rows, cols, p, eps, key = 3, 11, 0.3, 1e-3, (1, 2)
    x, r, g = rng.normal(size=(rows, cols)), rng.normal(size=(rows, cols)), 1 + 0.1 * rng.normal(size=cols)
    dy, dh = rng.normal(size=(rows, cols)), rng.normal(size=(rows, cols))

    def loss(x, r, g):
        h, _, y = branch_ref.add_norm(x, r, g, key, p, eps)
        return (dy * y).sum() + (dh * h).sum()

    h, rms, _ = branch_ref.add_norm(x, r, g, key, p, eps)
    got = branch_ref.add_norm_bwd(dy, g, h, rms, dh, key, p)
    for which, grad in zip((0, 1, 2), got):
        args = [x, r, g]
        for at in np.ndindex(*args[which].shape):
            d = np.zeros_like(args[which])
            d[at] = 1e-5
            up, down = ([a + s * d if i == which else a for i, a in enumerate(args)] for s in (1, -1))
            # differences: 1e-10 times a third derivative below 100, and 1e-16 / 1e-5 of rounding
            assert abs((loss(*up) - loss(*down)) / 2e-5 - grad[at]) < 1e-6


def test_e2m1_reference():
    v = np.array([0, 0.24, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 7, 100, -0.75, -2.5, -5])
    assert branch_ref.nearest_e2m1(v).tolist() == [0, 0, 0, 0.5, 1, 1, 2, 2, 4, 4, 6, 6, 6, -1, -2, -4]
    q, code = branch_ref.quantize_mx4(np.array([[6.0, 1.0] + [0.0] * 30 + [2.0 ** -140, np.inf]]))
    assert code.tolist() == [[127, 255]] and q[0, :2].tolist() == [6, 1] and (q[0, 32:] == 0).all()


def test_dropout_refusals(lib):
    def call(x=A, residual=B, rng=C, y=D, rows=4, cols=16, p=0.5, x_type=BF16, y_type=F32):
        return lib.rowops_dropout(x, residual, rng, y, rows, cols, p, x_type, y_type, None)

    for bad in (dict(rows=-1), dict(cols=-1), dict(cols=2 ** 31 - 256), dict(rows=1 << 40, cols=1 << 30), dict(p=-0.1),
                dict(p=1.1), dict(p=float("nan")), dict(x_type=E4M3), dict(y_type=E2M1), dict(x_type=-1)):
        assert call(**bad) == SHAPE, bad
    assert call(x=None) == call(y=None) == call(rng=None) == NULL
    assert call(x=A + 1) == call(residual=B + 2) == call(rng=C + 4) == call(y=D + 2) == ALIGN
    assert call(y=A) == call(y=B + 4) == call(y=A + 64) == call(rng=D + 8) == ALIAS
    assert call(y=A, x_type=F32, residual=A + 64) == ALIAS  # y is x, but overlaps the residual
    assert call(rows=0, x=None, y=None, rng=None) == OK and call(cols=0, x=None) == OK


def test_norm_refusals(lib):
    def call(x=A, residual=B, gamma=C, rng=D, h=E, out=F, scale=G, rms=H, rows=4, cols=16, eps=1e-5, p=0.5,
             x_type=BF16, h_type=F32, out_type=BF16):
        return lib.rowops_add_rmsnorm_fwd(x, residual, gamma, rng, h, out, scale, rms, rows, cols, eps, p, x_type,
                                          h_type, out_type, None)

    for bad in (dict(rows=-1), dict(cols=0), dict(cols=2 ** 31 - 256), dict(eps=-1.0), dict(eps=float("inf")),
                dict(p=2.0), dict(h_type=F16), dict(x_type=F32, h_type=BF16), dict(out_type=F32), dict(out_type=5),
                dict(x_type=E4M3, h_type=E4M3, out_type=E4M3)):
        assert call(**bad) == SHAPE, bad
    assert call(x=None) == call(gamma=None) == call(out=None) == call(rng=None) == NULL
    assert call(scale=None, out_type=E4M3) == call(scale=None, out_type=E2M1) == NULL
    assert call(x=A + 1) == call(residual=B + 2) == call(h=E + 2) == call(rms=H + 2) == ALIGN
    assert call(scale=G + 2, out_type=E4M3) == ALIGN
    assert call(h=A) == call(h=B + 4) == call(out=B) == call(out=E) == call(rms=F) == call(out=C + 4) == ALIAS
    assert call(h=B, out=B + 64) == ALIAS and call(out_type=E2M1, scale=F + 8) == ALIAS
    assert call(rows=0, x=None, out=None) == OK


def test_norm_bwd_refusals(lib):
    need = lib.rowops_add_rmsnorm_bwd_workspace(4, 16)

    def call(dy=A, gamma=B, h=C, rms=D, dh=E, rng=F, dres=G, dx=H, dgamma=W, rows=4, cols=16, p=0.5, x_type=BF16,
             h_type=F32, ws=W + 4096, size=1 << 20):
        return lib.rowops_add_rmsnorm_bwd(dy, gamma, h, rms, dh, rng, dres, dx, dgamma, rows, cols, p, x_type, h_type, ws,
                                          size, None)

    for bad in (dict(rows=-1), dict(cols=0), dict(cols=2 ** 31 - 256), dict(p=-1.0), dict(h_type=F16), dict(x_type=E2M1)):
        assert call(**bad) == SHAPE, bad
    for name in ("dy", "gamma", "h", "rms", "rng", "dgamma"):
        assert call(**{name: None}) == NULL, name
    assert call(dy=A + 1) == call(h=C + 2) == call(dres=G + 2) == call(dgamma=W + 2) == ALIGN
    assert call(dres=C) == call(dx=C) == call(dgamma=B) == call(dx=G) == call(dres=A) == call(dx=E) == call(dres=E + 4) == ALIAS
    assert call(dx=A + 2) == ALIAS
    assert need > 0 and call(ws=None) == call(size=need - 1) == call(ws=W + 4104) == WORKSPACE
    assert call(ws=C) == call(ws=W) == ALIAS
    for bad in ((-1, 4), (4, 0), (4, 2 ** 31 - 1), (0, 4)):
        assert lib.rowops_add_rmsnorm_bwd_workspace(*bad) == 0


def test_mx4_refusals(lib):
    def quantize(x=A, q=B, scale=C, rows=4, cols=64, x_type=BF16):
        return lib.rowops_quantize_mx4(x, q, scale, rows, cols, x_type, None)

    def product(xq=A, xs=B, wq=C, ws=D, offsets=E, y=F, slots=8, cin=64, cout=16, experts=2, y_type=BF16, w=None, n=0):
        return lib.rowops_expert_matmul_mx4(xq, xs, wq, ws, offsets, y, slots, cin, cout, experts, y_type, w, n, None)

    for bad in (dict(rows=-1), dict(cols=-2), dict(cols=2 ** 31 - 256), dict(x_type=E4M3)):
        assert quantize(**bad) == SHAPE, bad
    assert quantize(x=None) == quantize(q=None) == quantize(scale=None) == NULL
    assert quantize(x=A + 1) == ALIGN
    assert quantize(q=A) == quantize(scale=B) == quantize(q=A + 511) == ALIAS
    assert quantize(rows=0) == quantize(cols=0) == OK
    for bad in (dict(slots=-1), dict(cin=0), dict(cin=63), dict(cout=0), dict(experts=0), dict(experts=1025),
                dict(y_type=E4M3), dict(slots=(1 << 30) + 1)):
        assert product(**bad) == SHAPE, bad
    for name in ("xq", "xs", "wq", "ws", "offsets", "y"):
        assert product(**{name: None}) == NULL, name
    assert product(offsets=E + 2) == product(y=F + 1) == ALIGN
    assert product(y=A) == product(y=D) == product(y=E) == product(w=F, n=64) == product(w=B, n=64) == ALIAS
    assert product(w=W + 8, n=64) == WORKSPACE
    assert product(slots=0) == OK
    size = lib.rowops_expert_matmul_mx4_workspace
    assert size(8, 64, 16, 2) == 0 and size(8, 33, 16, 2) == 0 and size(0, 34, 16, 2) == 0
    assert size(8, 34, 16, 2) == 256 + 256 + 32 * 32  # rows of 17 bytes on 32


def test_binding_refuses_without_a_gpu(lib):
    x = torch.zeros(4, 16)
    for call in (lambda: binding.rowops_dropout(x, None, 0.0), lambda: binding.rowops_add_rmsnorm_fwd(x, x[0]),
                 lambda: binding.rowops_add_rmsnorm_bwd(x, x[0], x, x[:, 0]), lambda: binding.rowops_quantize_mx4(x),
                 lambda: binding.rowops_expert_matmul_mx4(x, x, x, x)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
