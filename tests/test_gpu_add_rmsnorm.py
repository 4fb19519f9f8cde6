"""The residual's addition with its RMS norm, forward and backward, against 64 bits.

Bounds, u = 2^-24.  h: x * s (2 u) and an addition (u).  The squares' sum has at most
16 + cols / 1024 terms in a row for one lane and 10 steps over lanes and warps, so rms is
off by (26 + cols / 1024) u and what h's error makes of it; y adds a reciprocal, two
products and the gamma's, 4 u.  Backward: a mean of as many terms off by that many u of
the magnitudes' mean, seven operations behind it, and one more product and sum for dh.
dgamma: rows + 10 additions at most.  Each result is rounded to its type once (u_t)."""
import numpy as np
import pytest
import torch

import branch_ref
from test_gpu_dropout import placed, rng_of
from test_gpu_expert_matmul import TINY, TYPES, UNIT, f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
PAIRS = [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")]
SHAPES = [(1, 1), (5, 8), (3, 33), (9, 64), (7, 72), (6, 128), (5, 136), (4, 255), (3, 256), (700, 264), (2, 768),
          (3, 1023), (5, 1024), (2, 2056), (2, 4096), (700, 2048), (1, 8192), (3, 8200), (2, 16384), (2, 16392), (1, 20001),
          (1, 50000), (1300, 40), (1300, 120), (1300, 200), (700, 1023), (650, 4104)]


def inputs(seed, shape, types, shift=0, residual=True):
    g = np.random.default_rng(seed)
    a, b = (TYPES[t] for t in types)
    x = placed(g.normal(size=shape), a, shift)
    r = placed(g.normal(size=shape) * np.exp2(g.integers(-3, 4, (shape[0], 1))), b, shift) if residual else None
    gamma = placed(1 + 0.1 * g.normal(size=shape[1]), torch.float32, shift)
    return x, r, gamma, tuple(int(v) for v in g.integers(-2 ** 62, 2 ** 62, 2))


def chain(cols):
    return 26 + cols / 1024


def forward_bounds(x, r, gamma, key, p):
    """64-bit h, rms and y with their bounds before the last rounding."""
    x64, g64 = f64(x), f64(gamma)
    r64 = None if r is None else f64(r)
    h, rms, y = branch_ref.add_norm(x64, r64, g64, key, p, EPS)
    xs = np.abs(branch_ref.drop(x64, key, p))
    eh = U * (2 * xs + (0 if r is None else xs + np.abs(r64)))
    erms = rms * (chain(x.shape[1]) * U) + np.sqrt((eh * eh).mean(1))
    ey = np.abs(y) * (erms / rms + 4 * U)[:, None] + np.abs(g64) * eh / rms[:, None]
    return (h, eh), (rms, erms), (y, ey)


def near(got, want, e, t):
    want, got = np.asarray(want), f64(got)
    far = np.abs(got - want)
    limit = UNIT[t] * np.abs(want) + (1 + UNIT[t]) * 1.01 * e + TINY[t]
    assert (far <= limit).all(), f"{(far / limit).max()} times the bound"


@pytest.mark.parametrize("types", PAIRS)
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(ro, shape, types):
    for shift, residual, p in ((0, True, 0.0), (0, True, 0.2), (1, True, 0.2), (0, False, 0.0)):
        x, r, gamma, key = inputs(sum(shape), shape, types, shift, residual)
        rng = rng_of(*key)
        y, scale, h, rms = ro.rowops_add_rmsnorm_fwd(x, gamma, residual=r, rng=rng, p=p, eps=EPS)
        assert scale is None and y.dtype == x.dtype and h.dtype == (x.dtype if r is None else r.dtype)
        if r is None:
            assert h is x
        (h64, eh), (rms64, erms), (y64, ey) = forward_bounds(x, r, gamma, key, p)
        near(h, h64, eh, types[1] if residual else types[0])
        near(rms, rms64, erms, "f32")
        near(y, y64, ey, types[0])


@pytest.mark.parametrize("types", PAIRS)
@pytest.mark.parametrize("shape", SHAPES)
def test_quantised_answers(ro, shape, types):
    """The values stand for y within a rounding to e4m3 (2^-4, and half the least step) or e2m1 (as the reference
    rounds, or its neighbour where y lies that close to a border)."""
    for shift, p in ((0, 0.0), (1, 0.3)):
        x, r, gamma, key = inputs(sum(shape) + 1, shape, types, shift)
        _, _, (y64, ey) = forward_bounds(x, r, gamma, key, p)
        kw = dict(residual=r, rng=rng_of(*key), p=p, eps=EPS)
        q, scale, h, rms = ro.rowops_add_rmsnorm_fwd(x, gamma, quantize="e4m3", **kw)
        plain = ro.rowops_add_rmsnorm_fwd(x, gamma, **kw)
        assert torch.equal(h, plain[2]) and torch.equal(rms, plain[3])
        s64 = np.repeat(f64(scale), 128, 1)[:, :shape[1]]
        got = f64(q.float()) * s64
        assert (np.abs(got - y64) <= 2.0 ** -4 * np.abs(y64) + 2.0 ** -10 * s64 + 1.1 * ey + 2 * U * np.abs(y64)).all()
        for b in range(scale.shape[1]):
            most, off = np.abs(y64[:, b * 128:b * 128 + 128]).max(1), ey[:, b * 128:b * 128 + 128].max(1)
            assert (np.abs(f64(scale)[:, b] * 448 - most) <= off + 4 * U * most).all()
        q, scale, h, _ = ro.rowops_add_rmsnorm_fwd(x, gamma, quantize="mx4", **kw)
        assert torch.equal(h, plain[2])
        code = scale.cpu().numpy()
        low, high = (branch_ref.quantize_mx4(y64 * (1 + s * 1e-5))[1] for s in (-1, 1))  # ey is below 1e-5 |max|
        assert ((code == low) | (code == high)).all()
        unit = branch_ref.spread_mx4(code, shape[1])
        values = branch_ref.unpack_mx4(q.cpu().numpy(), shape[1])
        low, high = (branch_ref.nearest_e2m1((y64 + s * (1.1 * ey + 2.0 ** -149)) / unit) for s in (-1, 1))
        assert ((values >= low) & (values <= high)).all()


@pytest.mark.parametrize("cols", [40, 64, 100, 128, 256, 768, 1001, 4096, 16384, 16400, 16401])
def test_quantised_answers_are_the_quantisers(ro, cols):
    """fp32 answers are not rounded, so quantising them afterwards gives the same bytes."""
    x, r, gamma, key = inputs(cols, (6, cols), ("f32", "f32"))
    y = ro.rowops_add_rmsnorm_fwd(x, gamma, residual=r)[0]
    q, scale = ro.rowops_add_rmsnorm_fwd(x, gamma, residual=r, quantize="e4m3")[:2]
    q2, scale2 = ro.rowops_quantize_blocks(y)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(scale, scale2)
    for a, b in zip(ro.rowops_add_rmsnorm_fwd(x, gamma, residual=r, quantize="mx4")[:2], ro.rowops_quantize_mx4(y)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("quantize", [None, "e4m3", "mx4"])
@pytest.mark.parametrize("cols", [48, 120, 768, 1001, 20000])
def test_bad_values_stay_in_their_rows(ro, cols, quantize):
    x, r, gamma, _ = inputs(3, (6, cols), ("bf16", "f32"))
    clean = ro.rowops_add_rmsnorm_fwd(x, gamma, residual=r, quantize=quantize)
    x[2, cols // 2], r[4, cols - 1] = float("nan"), float("inf")
    out, scale, h, rms = ro.rowops_add_rmsnorm_fwd(x, gamma, residual=r, quantize=quantize)
    good = [0, 1, 3, 5]
    for a, b in zip((out, h, rms), (clean[0], clean[2], clean[3])):
        assert torch.equal(a[good].view(torch.uint8), b[good].view(torch.uint8))
    assert torch.isnan(rms[2]) and torch.isinf(rms[4])
    if quantize == "mx4":  # the whole row is NaN, or the block of inf / inf is
        assert (scale[2] == 255).all() and scale[4, -1] == 255 and (scale[good] != 255).all()
    else:
        y = out.float()
        assert torch.isnan(y[2]).all() and torch.isnan(y[4, cols - 1]) and (y[4, :cols - 1] == 0).all()


@pytest.mark.parametrize("types", PAIRS)
@pytest.mark.parametrize("shape", SHAPES + [(1500, 64), (1000, 33), (400, 8192), (300, 9000), (170, 16384), (90, 24584), (50, 65536), (3, 65544)])
def test_backward(ro, shape, types):
    a, b = types
    rows, cols = shape
    for shift, with_dh, p in ((0, True, 0.25), (1, True, 0.25), (0, False, 0.0)):
        g = np.random.default_rng(rows + cols)
        dy, h = placed(g.normal(size=shape), TYPES[a], shift), placed(g.normal(size=shape) * 3, TYPES[b], shift)
        dh = placed(g.normal(size=shape), TYPES[b], shift) if with_dh else None
        gamma = placed(1 + 0.1 * g.normal(size=cols), torch.float32, shift)
        rms = torch.sqrt(h.double().square().mean(1) + EPS).float()
        key = (7, -5)
        dx, dres, dgamma = ro.rowops_add_rmsnorm_bwd(dy, gamma, h, rms, dh=dh, rng=rng_of(*key), p=p)
        assert dx.dtype == dy.dtype and dres.dtype == h.dtype and (dx is dres) == (p == 0 and a == b)
        dy64, h64, g64, rms64 = f64(dy), f64(h), f64(gamma), f64(rms)
        wdx, wres, wgamma = branch_ref.add_norm_bwd(dy64, g64, h64, rms64, None if dh is None else f64(dh), key, p)
        n, gy, inv = np.abs(h64) / rms64[:, None], np.abs(dy64 * g64), 1 / rms64[:, None]
        mean = (gy * n).mean(1, keepdims=True)
        e = U * (inv * (7 * gy + n * mean * (chain(cols) + 12)) + np.abs(wres) + (0 if dh is None else np.abs(f64(dh))))
        near(dres, wres, e, b)
        t = branch_ref.threshold(p)
        s = 65536 / (65536 - t)
        near(dx, wdx, np.where(wdx != 0, s * (e + 2 * U * np.abs(wres)), 0), a)
        near(dgamma, wgamma, (rows + 10) * U * (np.abs(dy64) * n).sum(0), "f32")


@pytest.mark.parametrize("cols", [64, 100, 2048, 17000])
def test_in_place(ro, cols):
    x, r, gamma, key = inputs(cols, (50, cols), ("f32", "f32"))
    rng = rng_of(*key)
    want = ro.rowops_add_rmsnorm_fwd(x, gamma, residual=r, rng=rng, p=0.1)
    stream = r.clone()
    got = ro.rowops_add_rmsnorm_fwd(x, gamma, residual=stream, rng=rng, p=0.1, h=stream)
    assert got[2] is stream and all(torch.equal(got[i], want[i]) for i in (0, 2, 3))
    dy, dh = torch.randn_like(x), torch.randn_like(x)
    want = ro.rowops_add_rmsnorm_bwd(dy, gamma, want[2], want[3], dh=dh, rng=rng, p=0.1)
    got = ro.rowops_add_rmsnorm_bwd(dy, gamma, stream, got[3], dh=dh, rng=rng, p=0.1, dx=dy, dresidual=dh)
    assert got[0] is dy and got[1] is dh and all(torch.equal(u, v) for u, v in zip(got, want))


def test_repeats_bit_for_bit_and_empty(ro):
    x, r, gamma, key = inputs(1, (5000, 768), ("bf16", "f32"))
    _, _, h, rms = ro.rowops_add_rmsnorm_fwd(x, gamma, residual=r)
    first = ro.rowops_add_rmsnorm_bwd(x, gamma, h, rms, dh=r, rng=rng_of(*key), p=0.1)
    for _ in range(3):
        again = ro.rowops_add_rmsnorm_bwd(x, gamma, h, rms, dh=r, rng=rng_of(*key), p=0.1)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    out, _, h0, rms0 = ro.rowops_add_rmsnorm_fwd(x[:0], gamma, residual=r[:0])
    assert out.shape == (0, 768) and rms0.shape == (0,)
    dgamma = torch.full((768,), 3.0, device="cuda")
    ro.rowops_add_rmsnorm_bwd(x[:0], gamma, h0, rms0, dgamma=dgamma)
    assert (dgamma == 0).all()


@pytest.mark.parametrize("rows,cols", [(2, 8200), (37, 12064), (500, 16384), (60, 40000), (41, 65536)])
def test_long_rows_on_three_streams(ro, rows, cols):
    """Rows that a cluster shares: calls at once, and replayed from a graph, give what one call gives, bit for bit."""
    x, r, gamma, key = inputs(cols, (rows, cols), ("bf16", "f32"))
    rng = rng_of(*key)
    _, _, h, rms = ro.rowops_add_rmsnorm_fwd(x, gamma, residual=r, rng=rng, p=0.1)
    want = ro.rowops_add_rmsnorm_bwd(x, gamma, h, rms, dh=r, rng=rng, p=0.1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = ro.rowops_add_rmsnorm_bwd(x, gamma, h, rms, dh=r, rng=rng, p=0.1)
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for _ in range(10):
        for stream in streams[:2]:
            with torch.cuda.stream(stream):
                got.append(ro.rowops_add_rmsnorm_bwd(x, gamma, h, rms, dh=r, rng=rng, p=0.1))
        with torch.cuda.stream(streams[2]):
            graph.replay()
    torch.cuda.synchronize()
    for out in [captured, *got]:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert ro.library().rowops_pipeline_timeouts() == 0


def test_leading_dimensions(ro):
    x, r, gamma, _ = inputs(2, (24, 136), ("f16", "f32"))
    flat = ro.rowops_add_rmsnorm_fwd(x, gamma, residual=r, quantize="mx4")
    deep = ro.rowops_add_rmsnorm_fwd(x.view(2, 3, 4, 136), gamma, residual=r.view(2, 3, 4, 136), quantize="mx4")
    assert deep[0].shape == (2, 3, 4, 68) and deep[1].shape == (2, 3, 4, 5) and deep[3].shape == (2, 3, 4)
    assert all(torch.equal(a.view(b.shape), b) for a, b in zip(deep, flat))


def test_guard_bands(ro):
    """Outputs and the workspace between bands of a fixed pattern, which stay."""
    def banded(shape, dtype):
        n = int(np.prod(shape)) * dtype.itemsize
        buf = torch.full((n + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
        return buf, buf[4096:4096 + n].view(dtype).view(shape)

    for rows, cols in ((5, 8), (33, 64), (3, 100), (9, 128), (7, 777), (5, 2048), (2, 16384), (2, 17001)):
        x, r, gamma, key = inputs(cols, (rows, cols), ("bf16", "f32"))
        rng = rng_of(*key)
        bufs = {name: banded(shape, dtype) for name, shape, dtype in (
            ("h", (rows, cols), torch.float32), ("row_rms", (rows,), torch.float32), ("out", (rows, cols), torch.bfloat16),
            ("q", (rows, cols), torch.float8_e4m3fn), ("s", (rows, -(-cols // 128)), torch.float32),
            ("q4", (rows, -(-cols // 2)), torch.uint8), ("s4", (rows, -(-cols // 32)), torch.uint8),
            ("dx", (rows, cols), torch.bfloat16), ("dresidual", (rows, cols), torch.float32), ("dgamma", (cols,), torch.float32),
            ("ws", (ro.rowops_add_rmsnorm_bwd_workspace(rows, cols),), torch.uint8), ("y", (rows, cols), torch.float32))}
        at = {k: v[1] for k, v in bufs.items()}
        kw = dict(residual=r, rng=rng, p=0.2, h=at["h"], row_rms=at["row_rms"])
        ro.rowops_add_rmsnorm_fwd(x, gamma, out=at["out"], **kw)
        ro.rowops_add_rmsnorm_fwd(x, gamma, quantize="e4m3", out=at["q"], scale=at["s"], **kw)
        ro.rowops_add_rmsnorm_fwd(x, gamma, quantize="mx4", out=at["q4"], scale=at["s4"], **kw)
        ro.rowops_add_rmsnorm_bwd(x, gamma, at["h"], at["row_rms"], dh=r, rng=rng, p=0.2, dx=at["dx"],
                                  dresidual=at["dresidual"], dgamma=at["dgamma"], workspace=at["ws"])
        ro.rowops_dropout(x, rng, 0.2, residual=r, y=at["y"])
        ro.rowops_quantize_mx4(x, q=at["q4"], scale=at["s4"])
        for name, (buf, _) in bufs.items():
            assert (buf[:4096] == 0x5A).all() and (buf[-4096:] == 0x5A).all(), (name, rows, cols)


@pytest.mark.parametrize("cols", [33, 768, 9000])
def test_answers_that_are_not_wanted(ro, cols):
    """C calls with NULL for an answer: the others are what they are with all.  Without dx no mask is made, and rng is NULL."""
    lib, stream = ro.library(), torch.cuda.current_stream().cuda_stream
    x, r, gamma, key = inputs(cols, (40, cols), ("bf16", "f32"))
    rng = rng_of(*key)
    y, _, h, rms = ro.rowops_add_rmsnorm_fwd(x, gamma, residual=r, rng=rng, p=0.2)
    want = ro.rowops_add_rmsnorm_bwd(x, gamma, h, rms, dh=r, rng=rng, p=0.2)
    out = torch.empty_like(y)
    status = lib.rowops_add_rmsnorm_fwd(x.data_ptr(), r.data_ptr(), gamma.data_ptr(), rng.data_ptr(), None, out.data_ptr(), None,
                                        None, 40, cols, EPS, 0.2, 2, 0, 2, stream)
    assert status == 0 and torch.equal(out, ro.rowops_add_rmsnorm_fwd(x, gamma, residual=r, rng=rng, p=0.2, eps=EPS)[0])
    ws = torch.empty(ro.rowops_add_rmsnorm_bwd_workspace(40, cols), dtype=torch.uint8, device="cuda")
    for with_dx, with_res in ((False, True), (True, False), (False, False)):
        dx, dres, dgamma = torch.empty_like(x), torch.empty_like(r), torch.empty_like(gamma)
        status = lib.rowops_add_rmsnorm_bwd(x.data_ptr(), gamma.data_ptr(), h.data_ptr(), rms.data_ptr(), r.data_ptr(),
                                            rng.data_ptr() if with_dx else None, dres.data_ptr() if with_res else None,
                                            dx.data_ptr() if with_dx else None, dgamma.data_ptr(), 40, cols, 0.2, 2, 0,
                                            ws.data_ptr(), ws.numel(), stream)
        assert status == 0 and torch.equal(dgamma, want[2])
        assert not with_dx or torch.equal(dx, want[0])
        assert not with_res or torch.equal(dres, want[1])


def test_refusals(ro):
    x, gamma = torch.zeros(4, 16, device="cuda"), torch.ones(16, device="cuda")
    rms, rng = torch.ones(4, device="cuda"), rng_of(0, 0)
    fwd, bwd = ro.rowops_add_rmsnorm_fwd, ro.rowops_add_rmsnorm_bwd
    for call in (lambda: fwd(x, gamma, p=0.5), lambda: fwd(x, gamma[:8]), lambda: fwd(x, gamma, residual=x[:2]),
                 lambda: fwd(x, gamma, quantize="int8"), lambda: fwd(x, gamma, scale=x), lambda: fwd(x.T, rms),
                 lambda: bwd(x, gamma, x, rms[:2]), lambda: bwd(x, gamma, x, rms, p=0.5),
                 lambda: bwd(x, gamma, x[:2], rms)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fwd(x, gamma.half()), lambda: fwd(x, gamma, h=x.half(), residual=x), lambda: fwd(x.int(), gamma),
                 lambda: bwd(x, gamma, x, rms, dh=x.half())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: fwd(x.half(), gamma, residual=x.bfloat16()), lambda: fwd(x, gamma, residual=x.half()),
                 lambda: fwd(x, gamma, eps=-1.0), lambda: fwd(x, gamma, rng=rng, p=1.5),
                 lambda: bwd(x, gamma, x, rms, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                 lambda: fwd(x, gamma, residual=x, out=x)):
        with pytest.raises(ro.RowopsError):
            call()
