"""Dropout against its definition in 64 bits.

What drops and what stays has to agree in every place.  A kept value is x * s with s
rounded to fp32 (2^-24 each), the residual's addition rounds once (2^-24), and the
result is rounded to its type (u_t); a dropped value is exactly the residual or +0.0."""
import numpy as np
import pytest
import torch

import branch_ref
from test_gpu_expert_matmul import TINY, TYPES, UNIT, f64

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 8), (3, 7), (5, 16), (2, 255), (7, 256), (4, 257), (9, 768), (3, 1023), (2, 4104), (33, 64), (1, 20000), (70, 33), (19, 100), (5, 129)]


def rng_of(key, offset):
    return torch.tensor([key, offset], dtype=torch.int64, device="cuda")


def placed(a, dtype, shift):
    """a as a tensor that starts `shift` values behind a 16-byte boundary."""
    buf = torch.zeros(a.size + shift, dtype=dtype, device="cuda")
    buf[shift:] = torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype).reshape(-1)
    return buf[shift:].view(a.shape)


def check(y, x64, r64, keep, p, out):
    t = branch_ref.threshold(p)
    s = 65536.0 / (65536 - t) if t < 65536 else 0.0
    want = np.where(keep, x64 * s, 0.0) + r64
    slack = 2.0 ** -23 * np.abs(x64 * s) + 2.0 ** -24 * (np.abs(x64 * s) + np.abs(r64))
    got = f64(y)
    assert (np.abs(got - want) <= UNIT[out] * np.abs(want) + (1 + UNIT[out]) * slack + TINY[out]).all()
    assert (got[~keep] == np.broadcast_to(r64, got.shape)[~keep]).all()


@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16"),
                                   ("f16", "bf16"), ("f16", "f32"), ("f32", "f16"), ("bf16", "f16")])
@pytest.mark.parametrize("shape", SHAPES)
def test_dropout(ro, shape, types):
    g = np.random.default_rng(sum(shape))
    a, b = types
    for shift, residual, p in ((0, True, 0.1), (1, True, 0.5), (0, False, 0.9)):
        x = placed(1 + g.random(shape), TYPES[a], shift)  # no zeros: what dropped can be told
        r = placed(g.normal(size=shape), TYPES[b], shift) if residual else None
        key, offset = (int(v) for v in g.integers(-2 ** 62, 2 ** 62, 2))
        y = ro.rowops_dropout(x, rng_of(key, offset), p, residual=r, dtype=TYPES[b])
        assert y.dtype == TYPES[b] and y.shape == x.shape
        keep = branch_ref.kept((key, offset), *shape, p)
        check(y, f64(x), f64(r) if residual else np.zeros(shape), keep, p, b)
        # the backward pass: the same mask on a gradient, in the branch's type
        dy = placed(1 + g.random(shape), TYPES[b], shift)
        check(ro.rowops_dropout(dy, rng_of(key, offset), p, dtype=TYPES[a]), f64(dy), np.zeros(shape), keep, p, a)


@pytest.mark.parametrize("cols", [24, 33])
def test_ends_of_the_probability(ro, cols):
    x = torch.randn(5, cols, device="cuda")
    r = torch.randn(5, cols, device="cuda")
    rng = rng_of(3, 4)
    assert torch.equal(ro.rowops_dropout(x, None, 0.0, residual=r), x + r)
    assert torch.equal(ro.rowops_dropout(x, rng, 1e-6), x)  # rounds to 0
    assert torch.equal(ro.rowops_dropout(x, None, 1.0, residual=r), r)
    assert (ro.rowops_dropout(x, rng, 1.0 - 1e-6) == 0).all()  # rounds to 1
    y = ro.rowops_dropout(torch.ones(4096, cols, device="cuda"), rng, 65535 / 65536)
    keep = branch_ref.kept((3, 4), 4096, cols, 65535 / 65536)
    assert ((f64(y) == 65536) == keep).all() and ((f64(y) == 0) == ~keep).all()


@pytest.mark.parametrize("cols", [40, 41])
def test_what_drops_is_zero_whatever_it_was(ro, cols):
    bad = torch.full((64, cols), float("nan"), device="cuda")
    bad[::2] = float("inf")
    y = ro.rowops_dropout(bad, rng_of(1, 1), 0.5)
    keep = torch.from_numpy(branch_ref.kept((1, 1), 64, cols, 0.5)).cuda()
    assert (y[~keep] == 0).all() and not torch.signbit(y[~keep]).any() and not torch.isfinite(y[keep]).any()


@pytest.mark.parametrize("cols", [64, 65])
def test_in_place(ro, cols):
    x, r, rng = torch.randn(300, cols, device="cuda"), torch.randn(300, cols, device="cuda"), rng_of(9, 9)
    want = ro.rowops_dropout(x, rng, 0.3, residual=r)
    for y in (x.clone(), r.clone()):
        a, b = (y, r) if torch.equal(y, x) else (x, y)
        assert torch.equal(ro.rowops_dropout(a, rng, 0.3, residual=b, y=y), want)


def test_offsets_and_keys_give_other_masks(ro):
    x = torch.ones(64, 1024, device="cuda")
    masks = [ro.rowops_dropout(x, rng_of(*kv), 0.5) != 0 for kv in ((1, 0), (1, 1), (1, 2 ** 32), (2, 0), (1 + 2 ** 32, 0))]
    for i, a in enumerate(masks):
        for b in masks[:i]:  # alike in half of 65536 places, off by less than six standard deviations
            assert abs((a == b).double().mean().item() - 0.5) < 6 * 0.5 / 256


def test_leading_dimensions_and_a_long_matrix(ro):
    """Rows are counted over all leading dimensions, and blocks in 64 bits."""
    rng = rng_of(12, 13)
    x = torch.ones(2, 3, 5, 72, device="cuda").half()
    assert torch.equal(ro.rowops_dropout(x, rng, 0.4).view(30, 72), ro.rowops_dropout(x.view(30, 72), rng, 0.4))
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    rows, cols = 2 ** 20 + 1, 4096  # 2^32 + 4096 values
    big = torch.ones(rows, cols, dtype=torch.float16, device="cuda")
    y = ro.rowops_dropout(big, rng, 0.5, y=big)
    tail = f64(y[-1]) != 0
    per = cols // 8
    j = np.arange((rows - 1) * per, rows * per, dtype=np.uint64)
    counter = np.stack([j & np.uint64(0xFFFFFFFF), j >> np.uint64(32), np.full_like(j, 13), np.zeros_like(j)], 1)
    words = branch_ref.philox((12, 0), counter)
    halves = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], 2).reshape(-1)
    assert (tail == (halves >= 32768)).all()


def test_refusals(ro):
    x, rng = torch.zeros(4, 16, device="cuda"), rng_of(0, 0)
    for call in (lambda: ro.rowops_dropout(x, None, 0.5), lambda: ro.rowops_dropout(x.T, rng, 0.5),
                 lambda: ro.rowops_dropout(x, rng[:1], 0.5), lambda: ro.rowops_dropout(x, rng, 0.5, residual=x[:2])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ro.rowops_dropout(x.double(), rng, 0.5), lambda: ro.rowops_dropout(x, rng.int(), 0.5),
                 lambda: ro.rowops_dropout(x, rng.cpu(), 0.5), lambda: ro.rowops_dropout(x, rng, 0.5, residual=x.half(), dtype=torch.float32)):
        with pytest.raises(TypeError):
            call()
    for p in (-0.5, 1.5, float("nan")):
        with pytest.raises(ro.RowopsError):
            ro.rowops_dropout(x, rng, p)
    assert ro.rowops_dropout(x[:0], rng, 0.5).shape == (0, 16)
