"""The expert operators on the host: refusals of the C ABI and of the binding,
none of which launches a kernel, and the references' own checks."""
import numpy as np
import pytest
import torch

import __graft_entry__
import expert_ref
from row_wise_softmax_warp_gb300 import binding
from test_abi_host import A, ALIAS, ALIGN, B, C, D, E, F, G, NULL, OK, SHAPE, W, WORKSPACE

F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    lib = binding.library()
    before = lib.rowops_kernel_launches()
    yield lib
    assert lib.rowops_kernel_launches() == before


def test_plan_refusals(lib):
    def plan(indices=A, values=B, offsets=C, order=D, slot=E, rows=32, k=2, experts=8, ws=W, size=1 << 20):
        return lib.rowops_expert_plan(indices, values, offsets, order, slot, rows, k, experts, ws, size, None)

    for bad in (dict(rows=-1), dict(k=0), dict(k=-1), dict(experts=0), dict(experts=1025), dict(rows=1 << 30),
                dict(rows=(1 << 30) + 1, k=1), dict(rows=1 << 62, k=4)):
        assert plan(**bad) == SHAPE, bad
    for name in ("indices", "offsets", "order", "slot"):
        assert plan(**{name: None}) == NULL, name
    for name, at in (("indices", A), ("values", B), ("offsets", C), ("order", D), ("slot", E)):
        assert plan(**{name: at + 2}) == ALIGN, name
    assert plan(order=A) == ALIAS and plan(slot=B + 8) == ALIAS and plan(slot=D) == ALIAS
    assert plan(offsets=E + 4) == ALIAS and plan(offsets=A + 4 * 60) == ALIAS
    n = 1 << 16  # more than one block's pairs: a workspace is needed (its size needs a device's SM count)
    need = lib.rowops_expert_plan_workspace(n, 2, 64)
    if need:
        assert plan(rows=n, experts=64, ws=None) == WORKSPACE
        assert plan(rows=n, experts=64, size=need - 1) == WORKSPACE
        assert plan(rows=n, experts=64, ws=W + 8) == WORKSPACE
        assert plan(rows=n, experts=64, ws=D) == ALIAS
    assert lib.rowops_expert_plan_workspace(512, 4, 64) == 0
    for bad in ((-1, 2, 8), (4, 0, 8), (4, 2, 0), (4, 2, 1025), (1 << 40, 2, 8)):
        assert lib.rowops_expert_plan_workspace(*bad) == 0


def test_row_refusals(lib):
    def gather(x=A, slot=B, out=C, rows=8, k=2, cols=16, slots=16, x_type=F32, out_type=BF16):
        return lib.rowops_expert_gather(x, slot, out, rows, k, cols, slots, x_type, out_type, None)

    def combine(y=A, slot=B, weights=C, out=D, rows=8, k=2, cols=16, slots=16, y_type=F32, out_type=BF16):
        return lib.rowops_expert_combine(y, slot, weights, out, rows, k, cols, slots, y_type, out_type, None)

    def bwd(dout=A, y=B, slot=C, weights=D, dy=E, dweights=F, rows=8, k=2, cols=16, slots=16, out_type=F32,
            y_type=F16):
        return lib.rowops_expert_combine_bwd(dout, y, slot, weights, dy, dweights, rows, k, cols, slots, out_type,
                                             y_type, None)

    for op in (gather, combine, bwd):
        for bad in (dict(rows=-1), dict(k=0), dict(cols=-1), dict(slots=-1), dict(slots=(1 << 30) + 1),
                    dict(rows=1 << 30), dict(cols=1 << 31), dict(out_type=3), dict(out_type=-1)):
            assert op(**bad) == SHAPE, (op, bad)
        assert op(rows=0) == OK
    assert gather(cols=0) == OK and combine(cols=0) == OK and gather(slots=0) == OK
    for op, names in ((gather, ("x", "slot", "out")), (combine, ("y", "slot", "out")),
                      (bwd, ("dout", "y", "slot", "weights", "dy", "dweights"))):
        for name in names:
            assert op(**{name: None}) == NULL, (op, name)
    assert gather(x=A + 2) == ALIGN and gather(out=C + 1) == ALIGN and gather(slot=B + 2) == ALIGN
    assert combine(weights=C + 2) == ALIGN and bwd(dweights=F + 2) == ALIGN and bwd(dy=E + 1) == ALIGN
    assert gather(out=A) == ALIAS and gather(out=B + 60) == ALIAS
    assert combine(out=A + 64) == ALIAS and combine(out=C + 32) == ALIAS
    assert bwd(dy=B) == ALIAS and bwd(dweights=D) == ALIAS and bwd(dweights=E + 8) == ALIAS


def test_product_refusals(lib):
    def matmul(x=A, w=B, offsets=C, y=D, slots=64, cin=32, cout=48, experts=4, transposed=0, dtype=BF16, ws=None,
               size=0):
        return lib.rowops_expert_matmul(x, w, offsets, y, slots, cin, cout, experts, transposed, dtype, ws, size, None)

    def wgrad(dy=A, x=B, offsets=C, dw=D, slots=64, cin=32, cout=48, experts=4, dtype=BF16, dw_type=BF16, ws=None,
              size=0):
        return lib.rowops_expert_matmul_wgrad(dy, x, offsets, dw, slots, cin, cout, experts, dtype, dw_type, ws,
                                              size, None)

    def fp8(xq=A, xs=B, wq=C, ws=D, offsets=E, y=F, slots=64, cin=160, cout=48, experts=4, y_type=BF16, work=None,
            size=0):
        return lib.rowops_expert_matmul_fp8(xq, xs, wq, ws, offsets, y, slots, cin, cout, experts, y_type, work, size,
                                            None)

    for op in (matmul, wgrad, fp8):
        for bad in (dict(slots=-1), dict(slots=(1 << 30) + 1), dict(cin=0), dict(cout=0), dict(cin=-4),
                    dict(experts=0), dict(experts=1025), dict(cin=(1 << 31) - 1), dict(cout=(1 << 31) - 1),
                    dict(slots=1 << 30, cin=1 << 30, cout=1 << 30)):
            assert op(**bad) == SHAPE, (op, bad)
        assert op(offsets=None) == NULL
        assert op(offsets=(E if op is fp8 else C) + 2) == ALIGN
    assert matmul(dtype=F32) == SHAPE and matmul(dtype=7) == SHAPE and wgrad(dtype=F32) == SHAPE
    assert wgrad(dw_type=F16) == SHAPE and fp8(y_type=3) == SHAPE
    assert matmul(slots=0) == OK and fp8(slots=0) == OK
    for op, names in ((matmul, "x w y"), (wgrad, "dy x dw"), (fp8, "xq xs wq ws y")):
        for name in names.split():
            assert op(**{name: None}) == NULL, (op, name)
    assert matmul(x=A + 1) == ALIGN and wgrad(dw=D + 2, dw_type=F32) == ALIGN and fp8(xs=B + 2) == ALIGN
    assert matmul(y=A + 2) == ALIAS and matmul(y=B) == ALIAS and matmul(y=C) == ALIAS
    assert wgrad(dw=B + 2) == ALIAS and fp8(y=D) == ALIAS and fp8(y=A + 64) == ALIAS
    for op, name in ((matmul, "ws"), (wgrad, "ws"), (fp8, "work")):
        assert op(**{name: W + 8, "size": 1 << 20}) == WORKSPACE
        for at in (A, B, C, D):
            assert op(**{name: at + 16, "size": 1 << 20}) == ALIAS


def test_workspace_sizes(lib):
    """A copy for each matrix whose rows are no multiple of 16 bytes; none for others and for refused sizes."""
    assert lib.rowops_expert_matmul_workspace(100, 64, 128, 4, 0) == 0
    assert lib.rowops_expert_matmul_workspace(100, 64, 77, 4, 0) == 0  # rows of in values only
    assert lib.rowops_expert_matmul_workspace(100, 64, 77, 4, 1) >= 4 * 64 * 160
    assert lib.rowops_expert_matmul_workspace(100, 33, 128, 4, 0) >= (100 + 4 * 128) * 80
    assert lib.rowops_expert_matmul_wgrad_workspace(100, 64, 128) == 0
    assert lib.rowops_expert_matmul_wgrad_workspace(100, 33, 50) >= 100 * (80 + 112)
    assert lib.rowops_expert_matmul_fp8_workspace(100, 64, 77, 4) == 0
    assert lib.rowops_expert_matmul_fp8_workspace(100, 65, 77, 4) >= (100 + 4 * 77) * 80
    for bad in ((-1, 33, 8), (4, 0, 8), (4, 33, 0), (1 << 40, 33, 8)):
        assert lib.rowops_expert_matmul_workspace(*bad, 4, 0) == 0
        assert lib.rowops_expert_matmul_wgrad_workspace(*bad) == 0
        assert lib.rowops_expert_matmul_fp8_workspace(*bad, 4) == 0


def test_quantize_refusals(lib):
    def quantize(x=A, q=B, scale=C, batches=2, rows=8, cols=160, block_rows=1, x_type=BF16):
        return lib.rowops_quantize_blocks(x, q, scale, batches, rows, cols, block_rows, x_type, None)

    for bad in (dict(block_rows=0), dict(block_rows=64), dict(x_type=3), dict(batches=-1), dict(rows=-1),
                dict(cols=-1), dict(cols=1 << 31), dict(rows=1 << 31), dict(batches=1 << 40),
                dict(rows=1 << 20, batches=1 << 20), dict(rows=1 << 20, batches=1 << 10, cols=1 << 20)):
        assert quantize(**bad) == SHAPE, bad
    assert quantize(rows=0) == OK and quantize(cols=0) == OK and quantize(batches=0) == OK
    for name in ("x", "q", "scale"):
        assert quantize(**{name: None}) == NULL, name
    assert quantize(x=A + 1) == ALIGN and quantize(scale=C + 2) == ALIGN
    assert quantize(q=A + 64) == ALIAS and quantize(scale=B + 4) == ALIAS


def test_binding_refuses_host_tensors():
    ro = binding
    f, i = torch.zeros(4, 2), torch.zeros(4, 2, dtype=torch.int32)
    h = torch.zeros(4, 8, dtype=torch.float16)
    for call in (lambda: ro.rowops_expert_plan(f, 8), lambda: ro.rowops_expert_gather(f, i),
                 lambda: ro.rowops_expert_combine(f, i), lambda: ro.rowops_expert_combine_bwd(f, f, i, f),
                 lambda: ro.rowops_expert_matmul(h, h[None]), lambda: ro.rowops_expert_matmul_wgrad(h, h),
                 lambda: ro.rowops_quantize_blocks(f),
                 lambda: ro.rowops_expert_matmul_fp8(f, f, f, f)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()


def test_references():
    """The references against torch's own 64-bit operations and casts."""
    rng = np.random.default_rng(0)
    indices = rng.integers(0, 6, (50, 3)).astype(np.float32)
    offsets, order, slot = expert_ref.plan(indices, None, 6)
    assert (np.argsort(indices.reshape(-1), kind="stable") == order).all()
    assert (order[slot.reshape(-1)] == np.arange(150)).all()
    assert (np.diff(offsets) == np.bincount(indices.reshape(-1).astype(int), minlength=6)).all()
    v = np.concatenate([rng.normal(0, 100, 20000), np.exp2(rng.uniform(-12, 8.7, 20000))]).astype(np.float32)
    v = np.clip(v, -448, 448)
    cast = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    assert (expert_ref.e4m3(v.astype(np.float64)) == cast).all()
    x, w, dy = rng.normal(size=(9, 5)), rng.normal(size=(2, 4, 5)), rng.normal(size=(9, 4))
    y = expert_ref.matmul(x, w, [0, 4, 9])
    h = 1e-6  # the product is linear in w: the difference quotient is the gradient up to rounding
    w2 = w.copy()
    w2[1, 2, 3] += h
    diff = ((expert_ref.matmul(x, w2, [0, 4, 9]) - y) * dy).sum() / h
    assert abs(diff - expert_ref.wgrad(dy, x, [0, 4, 9])[1, 2, 3]) < 1e-8


def test_workspace_has_its_bytes():
    """A view that names more bytes than it holds, or skips some, is no workspace."""
    like = torch.empty(1)
    whole = torch.empty(512, dtype=torch.uint8)
    assert binding._scratch(whole, 64, like) == (whole, 512)
    for view in (torch.empty(1, dtype=torch.uint8).expand(1 << 20), whole[::2]):
        with pytest.raises(ValueError):
            binding._scratch(view, 64, like)
    with pytest.raises(ValueError):
        binding._scratch(bytearray(64), 64, like)
