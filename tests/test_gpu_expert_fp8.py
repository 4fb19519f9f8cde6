"""The block quantiser and the 8-bit product against plain 64-bit forms.

The quantiser's values are compared with the definition in 64 bits: a 16-bit x
times 448 is exact and the quotient is rounded once to fp32 before it is rounded to
e4m3, which moves it across a border between two e4m3 values only where it lies
within 2^-24 of one without being on it; a quotient of two 16-bit numbers' multiples
that close to a border needs more bits than they have, so values are equal.  For
fp32 x the neighbouring e4m3 value is allowed where the quotient is that close.

The product is compared with the 64-bit product of what the bytes stand for: a
product of two e4m3 is exact in fp32, a sum of 128 of them is off by at most
136 * 2^-23 of its terms' sum (cut at every step), each block's scale product and
the additions of the blocks add 2^-24 each."""
import numpy as np
import pytest
import torch

import expert_ref
from test_gpu_expert_matmul import GROUPS, TINY, TYPES, UNIT, f64, offsets_of

pytestmark = pytest.mark.gpu


def quantized(ro, x, block_rows):
    q, scale = ro.rowops_quantize_blocks(x, block_rows=block_rows)
    return q, scale, f64(q.float()), f64(scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("shape", [(1, 1), (3, 128), (130, 257), (1, 5, 768), (3, 200, 136), (2, 2, 129, 33), (128, 128)])
def test_quantize(ro, shape, block_rows, dtype):
    rng = np.random.default_rng(sum(shape))
    x = rng.normal(size=shape) * np.exp2(rng.integers(-6, 7, (*shape[:-1], 1)))
    x = torch.from_numpy(x).cuda().to(TYPES[dtype])
    for shift in (0, 1):
        buf = torch.zeros(x.numel() + shift, dtype=x.dtype, device="cuda")
        buf[shift:] = x.reshape(-1)
        q, scale, got, got_scale = quantized(ro, buf[shift:].view(x.shape), block_rows)
        want, want_scale = expert_ref.quantize(f64(x), block_rows)
        assert (got_scale == want_scale.astype(np.float32)).all()
        if dtype != "f32":
            assert (got == want).all()
        else:
            v = f64(x) / expert_ref.spread(want_scale, block_rows, *shape[-2:])
            low, high = expert_ref.e4m3(v * (1 - 2.0 ** -22)), expert_ref.e4m3(v * (1 + 2.0 ** -22))
            assert ((got == low) | (got == high)).all()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_odd_values(ro, block_rows):
    """Zeros, subnormals, the largest values, infinities and NaN."""
    big = torch.finfo(torch.float32).max
    x = torch.zeros(256, 256, device="cuda")
    x[0, :128] = 1e-42
    x[0, 130], x[0, 131], x[0, 132] = big, -big, big / 1000
    x[200, 0], x[200, 1], x[200, 2], x[200, 3] = float("inf"), float("nan"), -float("inf"), 2.0
    q, scale, got, got_scale = quantized(ro, x, block_rows)
    assert np.isfinite(got_scale).all() and (got_scale > 0).all()
    bad = ~np.isfinite(f64(x))
    assert (np.isnan(got) == bad).all()
    want, want_scale = expert_ref.quantize(f64(x), block_rows)
    assert (got_scale == want_scale.astype(np.float32)).all() and (got[~bad] == want[~bad]).all()
    assert got[0, 130] == 448 and got[0, 131] == -448 and got[200, 3] == 448


def test_quantize_empty_and_refusals(ro):
    q, scale = ro.rowops_quantize_blocks(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 64) and scale.shape == (0, 1)
    x = torch.zeros(4, 64, device="cuda")
    for call in (lambda: ro.rowops_quantize_blocks(x, block_rows=64), lambda: ro.rowops_quantize_blocks(x[0]),
                 lambda: ro.rowops_quantize_blocks(x.T), lambda: ro.rowops_quantize_blocks(x, scale=x)):
        with pytest.raises(ValueError):
            call()


def operands(ro, rng, sizes, cin, cout, extra):
    rows = sum(sizes)
    x = np.concatenate([rng.normal(size=(rows, cin)), np.full((extra, cin), np.nan)])
    w = rng.normal(size=(len(sizes), cout, cin)) * np.exp2(rng.integers(-3, 4, (len(sizes), 1, 1)))
    x = torch.from_numpy(x).cuda().to(torch.bfloat16)
    w = torch.from_numpy(w).cuda().to(torch.bfloat16)
    xq, xs = ro.rowops_quantize_blocks(x)
    wq, ws = ro.rowops_quantize_blocks(w, block_rows=128)
    x64 = f64(xq.float()) * expert_ref.spread(f64(xs), 1, rows + extra, cin)
    w64 = f64(wq.float()) * expert_ref.spread(f64(ws), 128, cout, cin)
    return (xq, xs, wq, ws), x64, w64


def check(got, want, terms, cin, out):
    blocks = -(-cin // 128)
    slack = (min(cin, 128) + 8) * 2.0 ** -23 + (blocks + 2) * 2.0 ** -24
    assert (np.abs(f64(got) - want) <= UNIT[out] * np.abs(want) + (1 + UNIT[out]) * slack * terms + TINY[out]).all()


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("widths", [(128, 128), (768, 256), (16, 8), (400, 136), (144, 520), (33, 50), (257, 130), (1, 1)])
@pytest.mark.parametrize("groups", sorted(GROUPS))
def test_product(ro, groups, widths, out):
    sizes, (cin, cout), extra = GROUPS[groups], widths, 3
    rng = np.random.default_rng(cin + len(sizes))
    args, x64, w64 = operands(ro, rng, sizes, cin, cout, extra)
    offsets = offsets_of(sizes)
    rows = int(offsets[-1])
    y = torch.full((rows + extra, cout), 5.0, dtype=TYPES[out], device="cuda")
    ro.rowops_expert_matmul_fp8(*args, torch.from_numpy(offsets).cuda(), y=y)
    check(y[:rows], expert_ref.matmul(x64, w64, offsets)[:rows], expert_ref.matmul(abs(x64), abs(w64), offsets)[:rows],
          cin, out)
    assert (y[rows:] == 5).all()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("widths", [(33, 50), (257, 130), (1, 1)])
@pytest.mark.parametrize("groups", sorted(GROUPS))
def test_product_without_a_workspace(ro, groups, widths, out):
    sizes, (cin, cout) = GROUPS[groups], widths
    rng = np.random.default_rng(cin + len(sizes))
    args, x64, w64 = operands(ro, rng, sizes, cin, cout, 0)
    offsets = offsets_of(sizes)
    y = ro.rowops_expert_matmul_fp8(*args, torch.from_numpy(offsets).cuda(), dtype=TYPES[out],
                                    workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    check(y, expert_ref.matmul(x64, w64, offsets), expert_ref.matmul(abs(x64), abs(w64), offsets), cin, out)


@pytest.mark.parametrize("widths", [(1040, 384), (1001, 131)])
def test_product_long(ro, widths):
    cin, cout = widths
    sizes = [1200, 0, 3, 700]
    rng = np.random.default_rng(4)
    args, x64, w64 = operands(ro, rng, sizes, cin, cout, 0)
    offsets = offsets_of(sizes)
    y = ro.rowops_expert_matmul_fp8(*args, torch.from_numpy(offsets).cuda(), dtype=torch.float32)
    check(y, expert_ref.matmul(x64, w64, offsets), expert_ref.matmul(abs(x64), abs(w64), offsets), cin, "f32")


def test_product_dense(ro):
    rng = np.random.default_rng(5)
    args, x64, w64 = operands(ro, rng, [300], 256, 384, 0)
    y = ro.rowops_expert_matmul_fp8(*args)
    assert y.dtype == torch.bfloat16
    check(y, expert_ref.matmul(x64, w64, None), expert_ref.matmul(abs(x64), abs(w64), None), 256, "bf16")


@pytest.mark.parametrize("widths", [(256, 384), (257, 130)])
def test_scales_far_apart(ro, widths):
    """Blocks whose scales differ by 2^40 keep their own."""
    cin, cout = widths
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.normal(size=(90, cin))).cuda()
    x[:, :128] *= 2.0 ** 20
    x[:, 128:] *= 2.0 ** -20
    w = torch.from_numpy(rng.normal(size=(2, cout, cin))).cuda()
    w[:, :, :128] = 0  # the first block adds nothing, whatever its scale
    xq, xs = ro.rowops_quantize_blocks(x.float())
    wq, ws = ro.rowops_quantize_blocks(w.float(), block_rows=128)
    offsets = np.array([0, 40, 90], np.int32)
    y = ro.rowops_expert_matmul_fp8(xq, xs, wq, ws, torch.from_numpy(offsets).cuda(), dtype=torch.float32)
    x64 = f64(xq.float()) * expert_ref.spread(f64(xs), 1, 90, cin)
    w64 = f64(wq.float()) * expert_ref.spread(f64(ws), 128, cout, cin)
    check(y, expert_ref.matmul(x64, w64, offsets), expert_ref.matmul(abs(x64), abs(w64), offsets), cin, "f32")


@pytest.mark.parametrize("widths", [(256, 384), (257, 130)])
def test_nan_stays_in_its_row(ro, widths):
    cin, cout = widths
    x = torch.randn(80, cin, device="cuda")
    x[41, 130] = float("inf")
    w = torch.randn(2, cout, cin, device="cuda")
    xq, xs = ro.rowops_quantize_blocks(x)
    wq, ws = ro.rowops_quantize_blocks(w, block_rows=128)
    y = ro.rowops_expert_matmul_fp8(xq, xs, wq, ws, torch.tensor([0, 41, 80], dtype=torch.int32, device="cuda"))
    bad = torch.isnan(y)
    assert bad[41].all() and bad.sum() == cout


def test_refusals(ro):
    rng = np.random.default_rng(7)
    (xq, xs, wq, ws), _, _ = operands(ro, rng, [4, 4], 256, 128, 0)
    at = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    for call in (lambda: ro.rowops_expert_matmul_fp8(xq, xs, wq, ws), lambda: ro.rowops_expert_matmul_fp8(xq, xs[:, :1], wq, ws, at),
                 lambda: ro.rowops_expert_matmul_fp8(xq, xs, wq, ws[:1].contiguous(), at),
                 lambda: ro.rowops_expert_matmul_fp8(xq, xs, wq[:, :, :128].contiguous(), ws, at)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ro.rowops_expert_matmul_fp8(xq.float(), xs, wq, ws, at)
