"""Microscaled 4-bit values and their product against 64 bits.

The quantiser's scales are powers of two, so a division is exact and its bytes have to
agree with the definition's for every type.  A product of two e2m1 values is exact, and
so is its power of two; an fp32 sum of K of them, taken in any order and rounded or cut at
every step, is off by at most (K + 8) 2^-23 sum |products|, and the result is rounded
once (u_t)."""
import numpy as np
import pytest
import torch

import branch_ref
import expert_ref
from test_gpu_dropout import placed
from test_gpu_expert_matmul import GROUPS, TINY, TYPES, UNIT, f64, offsets_of

pytestmark = pytest.mark.gpu

WIDTHS = [(256, 128), (768, 256), (32, 8), (64, 520), (544, 136), (160, 300), (34, 50), (258, 130), (1, 1), (2, 7), (33, 33), (515, 257)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 31), (5, 32), (2, 33), (7, 64), (4, 100), (9, 256), (3, 264), (2, 3, 517), (33, 768), (1, 4096), (2, 12345)])
def test_quantize(ro, shape, dtype):
    g = np.random.default_rng(sum(shape))
    a = g.normal(size=shape) * np.exp2(g.integers(-6, 7, (*shape[:-1], 1)))
    a[..., ::5] = np.rint(4 * a[..., ::5]) / 4  # ties among them
    for shift in (0, 1):
        x = placed(a, TYPES[dtype], shift)
        q, scale = ro.rowops_quantize_mx4(x)
        assert q.shape == (*shape[:-1], (shape[-1] + 1) // 2) and scale.shape == (*shape[:-1], -(-shape[-1] // 32))
        want, code = branch_ref.quantize_mx4(f64(x))
        assert (scale.cpu().numpy() == code).all()
        packed = q.cpu().numpy()
        assert (branch_ref.unpack_mx4(packed, shape[-1]) == want).all()
        if shape[-1] % 2:
            assert (packed[..., -1] >> 4 == 0).all()


@pytest.mark.parametrize("cols", [96, 97])
def test_quantize_odd_values(ro, cols):
    """Zeros, subnormals, the largest values, infinities and NaN."""
    big = torch.finfo(torch.float32).max
    x = torch.zeros(8, cols, device="cuda")
    x[1, :32], x[2, 3], x[2, 4], x[3, 40] = 1e-42, big, -big / 1.5, float("inf")
    x[4, 70], x[5, 0], x[6, 5], x[7, 33], x[7, 34] = float("nan"), -0.0, 2.0 ** -127, 2.0 ** -126 * 6, 2.0 ** -149
    q, scale = ro.rowops_quantize_mx4(x)
    want, code = branch_ref.quantize_mx4(f64(x))
    assert (scale.cpu().numpy() == code).all() and (branch_ref.unpack_mx4(q.cpu().numpy(), cols) == want).all()
    assert scale[3, 1] == 255 and scale[4, 2] == 255 and (scale == 255).sum() == 2 and scale[0, 0] == 0
    assert (q[3, 16:32] == 0).all()
    q, scale = ro.rowops_quantize_mx4(x[:0])
    assert q.shape == (0, (cols + 1) // 2)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(4001, 777), (3999, 1000), (70001, 40), (90001, 33), (1200001, 3), (3, 3000001)])
def test_quantize_many_odd_rows(ro, rows, cols, dtype):
    """Long runs of rows that are no whole blocks give what the same rows filled up with zeros give."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    full = torch.zeros(rows, (cols + 31) // 32 * 32, dtype=TYPES[dtype], device="cuda")
    full[:, :cols] = torch.randn(rows, cols, generator=g, device="cuda")
    want, code = ro.rowops_quantize_mx4(full)
    for shift in (0, 1):
        buf = torch.full((rows * cols + 16,), float("nan"), dtype=TYPES[dtype], device="cuda")
        x = buf[shift:shift + rows * cols].view(rows, cols)
        x.copy_(full[:, :cols])
        q, scale = ro.rowops_quantize_mx4(x)
        assert torch.equal(q, want[:, :(cols + 1) // 2]) and torch.equal(scale, code)


def operands(ro, g, sizes, cin, cout, extra):
    rows = sum(sizes)
    x = np.concatenate([g.normal(size=(rows, cin)), np.full((extra, cin), np.nan)])
    w = g.normal(size=(len(sizes), cout, cin)) * np.exp2(g.integers(-3, 4, (len(sizes), cout, 1)))
    x, w = (torch.from_numpy(a).cuda().to(torch.bfloat16) for a in (x, w))
    xq, xs = ro.rowops_quantize_mx4(x)
    wq, ws = ro.rowops_quantize_mx4(w)
    return (xq, xs, wq, ws), values(xq, xs, cin), values(wq, ws, cin)


def values(q, scale, cols):
    return branch_ref.unpack_mx4(q.cpu().numpy(), cols) * branch_ref.spread_mx4(scale.cpu().numpy(), cols)


def check(got, x64, w64, offsets, out):
    want, terms = expert_ref.matmul(x64, w64, offsets), expert_ref.matmul(abs(x64), abs(w64), offsets)
    slack = (x64.shape[1] + 8) * 2.0 ** -23
    assert (np.abs(f64(got) - want) <= UNIT[out] * np.abs(want) + (1 + UNIT[out]) * slack * terms + TINY[out]).all()


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("widths", WIDTHS)
@pytest.mark.parametrize("groups", sorted(GROUPS))
def test_product(ro, groups, widths, out):
    sizes, (cin, cout), extra = GROUPS[groups], widths, 3
    args, x64, w64 = operands(ro, np.random.default_rng(cin + len(sizes)), sizes, cin, cout, extra)
    offsets = offsets_of(sizes)
    rows = int(offsets[-1])
    y = torch.full((rows + extra, cout), 5.0, dtype=TYPES[out], device="cuda")
    ro.rowops_expert_matmul_mx4(*args, torch.from_numpy(offsets).cuda(), y=y)
    check(y[:rows], x64[:rows], w64, offsets, out)
    assert (y[rows:] == 5).all()
    assert ro.library().rowops_pipeline_timeouts() == 0


@pytest.mark.parametrize("widths", [(34, 50), (258, 130), (1, 1)])
@pytest.mark.parametrize("groups", ["ragged", "wide", "empty ends"])
def test_product_without_a_workspace(ro, groups, widths):
    sizes, (cin, cout) = GROUPS[groups], widths
    args, x64, w64 = operands(ro, np.random.default_rng(cin), sizes, cin, cout, 0)
    offsets = offsets_of(sizes)
    y = ro.rowops_expert_matmul_mx4(*args, torch.from_numpy(offsets).cuda(), dtype=torch.float32,
                                    workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    check(y, x64, w64, offsets, "f32")


@pytest.mark.parametrize("shift", [(1, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("widths", [(256, 96), (96, 200), (66, 31)])
def test_product_off_a_boundary(ro, widths, shift):
    """Bytes and scales that start anywhere."""
    cin, cout = widths
    sizes = [70, 0, 300]
    args, x64, w64 = operands(ro, np.random.default_rng(9), sizes, cin, cout, 0)

    def moved(t, by):
        buf = torch.zeros(t.numel() + 16, dtype=torch.uint8, device="cuda")
        buf[by:by + t.numel()] = t.reshape(-1)
        return buf[by:by + t.numel()].view(t.shape)

    xq, xs, wq, ws = args
    offsets = offsets_of(sizes)
    y = ro.rowops_expert_matmul_mx4(moved(xq, shift[0]), moved(xs, shift[1]), moved(wq, shift[1]), moved(ws, shift[0]),
                                    torch.from_numpy(offsets).cuda(), dtype=torch.float32)
    check(y, x64, w64, offsets, "f32")


@pytest.mark.parametrize("shift", [0, 3])
def test_many_short_odd_rows(ro, shift):
    """More than 2^15 rows of 35 and of 66 bytes, which are copied to 16-byte boundaries; an expert between has none."""
    sizes, cout = [9, 0, 31], 12501
    args, x64, w64 = operands(ro, np.random.default_rng(11), sizes, 70, cout, 0)
    at = torch.from_numpy(offsets_of(sizes)).cuda()

    def moved(t):
        buf = torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
        buf[shift:shift + t.numel()] = t.reshape(-1)
        return buf[shift:shift + t.numel()].view(t.shape)

    y = ro.rowops_expert_matmul_mx4(*(moved(t) for t in args), at, dtype=torch.float32)
    check(y, x64, w64, offsets_of(sizes), "f32")
    g = torch.Generator(device="cuda").manual_seed(12)
    x = moved(torch.randint(-2, 3, (40, 33), generator=g, device="cuda").half())
    w = moved(torch.randint(-2, 3, (3, cout, 33), generator=g, device="cuda").half())
    y = ro.rowops_expert_matmul(x, w, at)  # of whole numbers below 2^11: exact
    for e, rows in ((0, slice(0, 9)), (2, slice(9, 40))):
        assert torch.equal(y[rows].double(), x[rows].double() @ w[e].double().T)
    assert ro.library().rowops_pipeline_timeouts() == 0


@pytest.mark.parametrize("widths", [(1056, 384), (4096, 256), (2050, 131)])
def test_product_long(ro, widths):
    cin, cout = widths
    sizes = [1200, 0, 3, 700]
    args, x64, w64 = operands(ro, np.random.default_rng(4), sizes, cin, cout, 0)
    offsets = offsets_of(sizes)
    y = ro.rowops_expert_matmul_mx4(*args, torch.from_numpy(offsets).cuda(), dtype=torch.float32)
    check(y, x64, w64, offsets, "f32")


def test_product_dense(ro):
    args, x64, w64 = operands(ro, np.random.default_rng(5), [300], 256, 384, 0)
    y = ro.rowops_expert_matmul_mx4(*args)
    assert y.dtype == torch.bfloat16
    check(y, x64, w64, None, "bf16")


@pytest.mark.parametrize("widths", [(256, 384), (288, 40), (66, 31)])
def test_every_byte_counts(ro, widths):
    """Random bytes and scales: every code in every place, and rows that share no scale."""
    cin, cout = widths
    g = np.random.default_rng(7)
    sizes = [90, 5, 41]
    rows, blocks = sum(sizes), -(-cin // 32)
    xq, wq = g.integers(0, 256, (rows, cin // 2), np.uint8), g.integers(0, 256, (3, cout, cin // 2), np.uint8)
    xs, ws = g.integers(120, 135, (rows, blocks), np.uint8), g.integers(118, 130, (3, cout, blocks), np.uint8)
    t = [torch.from_numpy(a).cuda() for a in (xq, xs, wq, ws)]
    offsets = offsets_of(sizes)
    y = ro.rowops_expert_matmul_mx4(*t, torch.from_numpy(offsets).cuda(), dtype=torch.float32)
    check(y, values(*t[:2], cin), values(*t[2:], cin), offsets, "f32")


@pytest.mark.parametrize("widths", [(256, 384), (66, 31)])
def test_scales_far_apart(ro, widths):
    """Pairs of scales at the ends of their range whose product is an ordinary number."""
    cin, cout = widths
    for a, b in ((254, 0), (0, 254), (1, 253), (200, 60)):
        xq, wq = (torch.full((n, cin // 2), 0x22, dtype=torch.uint8, device="cuda") for n in (40, cout))  # ones
        xs, ws = (torch.full((n, -(-cin // 32)), c, dtype=torch.uint8, device="cuda") for n, c in ((40, a), (cout, b)))
        y = ro.rowops_expert_matmul_mx4(xq, xs, wq[None], ws[None], dtype=torch.float32)
        assert (y == cin * 2.0 ** (a + b - 254)).all(), (a, b)


@pytest.mark.parametrize("widths", [(256, 384), (258, 130)])
def test_nan_stays_in_its_row(ro, widths):
    cin, cout = widths
    x = torch.randn(80, cin, device="cuda")
    x[41, 130] = float("inf")
    w = torch.randn(2, cout, cin, device="cuda")
    w[1, 3, 7] = float("nan")
    xq, xs = ro.rowops_quantize_mx4(x)
    wq, ws = ro.rowops_quantize_mx4(w)
    y = ro.rowops_expert_matmul_mx4(xq, xs, wq, ws, torch.tensor([0, 41, 80], dtype=torch.int32, device="cuda"))
    bad = torch.isnan(y)
    assert bad[41].all() and bad[41:, 3].all() and bad.sum() == cout + 38


def test_bad_offsets_stay_in_bounds(ro):
    """Offsets outside the rows, falling or overlapping: rows that a group names are written, others stay."""
    args, _, _ = operands(ro, np.random.default_rng(11), [60, 60], 64, 48, 0)
    for offsets in ([0, -5, 120], [500, 600, 700], [-9, 1 << 30, 60], [100, 20, 90]):
        y = torch.full((120, 48), 7.0, dtype=torch.bfloat16, device="cuda")
        ro.rowops_expert_matmul_mx4(*args, torch.tensor(offsets, dtype=torch.int32, device="cuda"), y=y)
        named = np.zeros(120, bool)
        for e in range(2):
            lo = min(max(offsets[e], 0), 120)
            named[lo:min(max(offsets[e + 1], lo), 120)] = True
        assert (f64(y)[~named] == 7).all()


def test_refusals(ro):
    (xq, xs, wq, ws), _, _ = operands(ro, np.random.default_rng(7), [4, 4], 256, 128, 0)
    at = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    f = ro.rowops_expert_matmul_mx4
    for call in (lambda: f(xq, xs, wq, ws), lambda: f(xq, xs[:, :1].contiguous(), wq, ws, at), lambda: f(xq, xs, wq, ws[:1].contiguous(), at),
                 lambda: f(xq, xs, wq[:, :, :64].contiguous(), ws, at), lambda: f(xq, xs, wq, ws, at[:2].contiguous()),
                 lambda: f(xq.T, xs, wq, ws, at), lambda: ro.rowops_quantize_mx4(torch.zeros((), device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f(xq.int(), xs, wq, ws, at), lambda: f(xq, xs.float(), wq, ws, at),
                 lambda: ro.rowops_quantize_mx4(xq), lambda: f(xq, xs, wq, ws, at, y=torch.empty(8, 128, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(TypeError):
            call()
