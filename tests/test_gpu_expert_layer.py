"""The expert operators together, as a layer runs them: router, plan, gather,
product, activation, product, combine, and the whole way back; replayed as a CUDA
graph, on other streams, and with more than 2^32 bytes.

The layer's bound is propagated: every stage's error is its inputs' errors through
the stage (magnitudes in place of values) plus its own rounding, u = 2^-11 of an
fp16 result, and (K + 8) 2^-23 of the magnitudes summed for a product of K terms."""
import numpy as np
import pytest
import torch

import expert_ref

pytestmark = pytest.mark.gpu

U16, TINY16 = 2.0 ** -11, 2.0 ** -25


def f64(t):
    return t.double().cpu().numpy()


class Near:
    """A 64-bit value and a bound on how far the computed one may be from it."""

    def __init__(self, v, e=0.0):
        self.v, self.e = np.asarray(v, np.float64), np.zeros_like(v, np.float64) + e

    def rounded(self):
        return Near(self.v, self.e * (1 + U16) + U16 * np.abs(self.v) + TINY16)

    def map2(self, other, f, terms):
        """f bilinear, over sums of `terms` products."""
        a, b = np.abs(self.v), np.abs(other.v)
        e = f(self.e, b) + f(a, other.e) + f(self.e, other.e)
        return Near(f(self.v, other.v), e + (terms + 8) * 2.0 ** -23 * f(a + self.e, b + other.e))

    def check(self, t, what):
        far = np.abs(f64(t) - self.v)
        assert (far <= self.e).all(), f"{what}: {(far / np.maximum(self.e, 1e-300)).max()} times the bound"


def layer(ro, x, logits, mask, w1, w2, k, dout):
    """One mixture-of-experts layer with h = a^2, forward and backward; returns everything."""
    p = ro.rowops_masked_softmax(logits, mask)
    weights, indices = ro.rowops_top_k_rows(p, k)
    offsets, order, slot = ro.rowops_expert_plan(indices, w1.shape[0], values=weights)
    rows = torch.zeros(x.shape[0] * k, x.shape[1], dtype=w1.dtype, device=x.device)
    ro.rowops_expert_gather(x, slot, out=rows)
    a = torch.zeros(rows.shape[0], w1.shape[1], dtype=w1.dtype, device=x.device)
    ro.rowops_expert_matmul(rows, w1, offsets, y=a)
    h = a * a
    y = torch.zeros(rows.shape[0], w2.shape[1], dtype=w1.dtype, device=x.device)
    ro.rowops_expert_matmul(h, w2, offsets, y=y)
    out = ro.rowops_expert_combine(y, slot, weights=weights, dtype=torch.float32)
    dy, dweights = ro.rowops_expert_combine_bwd(dout, y, slot, weights, dy=torch.zeros_like(y))
    dw2 = ro.rowops_expert_matmul_wgrad(dy, h, offsets)
    dh = ro.rowops_expert_matmul(dy, w2, offsets, y=torch.zeros_like(h), transposed=True)
    da = 2 * a * dh
    dw1 = ro.rowops_expert_matmul_wgrad(da, rows, offsets)
    drows = ro.rowops_expert_matmul(da, w1, offsets, y=torch.zeros_like(rows), transposed=True)
    dx = ro.rowops_expert_combine(drows, slot, dtype=torch.float32)
    return {"weights": weights, "indices": indices, "offsets": offsets, "slot": slot, "out": out, "dweights": dweights,
            "dw2": dw2, "dw1": dw1, "dx": dx}


def inputs(rng, tokens, experts, cols, hidden, scale=1.0):
    def cuda(a, dtype=torch.float32):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)

    mask = (rng.random((tokens, experts)) < 0.8).astype(np.uint8)
    mask[::7] = 0  # tokens whose mask leaves nothing
    return (cuda(rng.normal(size=(tokens, cols)) * scale), cuda(rng.normal(size=(tokens, experts))),
            torch.from_numpy(mask).cuda(),
            cuda(rng.normal(size=(experts, hidden, cols)) * cols ** -0.5, torch.float16),
            cuda(rng.normal(size=(experts, cols, hidden)) * hidden ** -0.5, torch.float16),
            cuda(rng.normal(size=(tokens, cols))))


@pytest.mark.parametrize("tokens,experts,k,cols,hidden", [(1, 4, 2, 64, 96), (37, 8, 2, 64, 96), (300, 4, 3, 72, 40),
                                                          (64, 3, 1, 33, 57)])
def test_layer(ro, tokens, experts, k, cols, hidden):
    rng = np.random.default_rng(tokens)
    x, logits, mask, w1, w2, dout = inputs(rng, tokens, experts, cols, hidden)
    got = layer(ro, x, logits, mask, w1, w2, k, dout)
    weights, indices = f64(got["weights"]), f64(got["indices"])
    offsets, order, slot = expert_ref.plan(indices, weights, experts)
    assert (got["offsets"].cpu().numpy() == offsets).all() and (got["slot"].cpu().numpy() == slot).all()
    assert offsets[-1] == (weights != 0).sum()
    n = offsets[-1]
    bounds = list(zip(offsets[:-1], offsets[1:]))
    token, w = order[:n] // k, weights.reshape(-1)[order[:n]][:, None]

    def each(f, rows):  # by expert, rows grouped
        out = [f(e, a, b) for e, (a, b) in enumerate(bounds)]
        join = np.concatenate if rows else np.stack
        return Near(join([o.v for o in out]), join([o.e for o in out]))

    def part(t, a, b):
        return Near(t.v[a:b], t.e[a:b])

    W1, W2 = f64(w1), f64(w2)
    rows = Near(f64(x)[token]).rounded()
    a = each(lambda e, i, j: part(rows, i, j).map2(Near(W1[e].T), np.matmul, cols), True).rounded()
    h = a.map2(a, np.multiply, 0).rounded()
    y = each(lambda e, i, j: part(h, i, j).map2(Near(W2[e].T), np.matmul, hidden), True).rounded()

    def sum_by_token(t, scale):
        v, e = np.zeros((tokens, t.v.shape[1])), np.zeros((tokens, t.v.shape[1]))
        np.add.at(v, token, scale * t.v)
        np.add.at(e, token, np.abs(scale) * (t.e + k * 2.0 ** -23 * np.abs(t.v)) + 1e-30)
        return Near(v, e)

    sum_by_token(y, w).check(got["out"], "out")
    dy = Near(w * f64(dout)[token], 2.0 ** -23 * np.abs(w * f64(dout)[token])).rounded()
    dots = y.map2(Near(f64(dout)[token]), lambda p, q: (p * q).sum(1), cols)
    dw = Near(np.zeros(tokens * k))
    dw.v[order[:n]], dw.e[order[:n]] = dots.v, dots.e
    Near(dw.v.reshape(tokens, k), dw.e.reshape(tokens, k)).check(got["dweights"], "dweights")

    def outer(p, q):
        return lambda e, i, j: (Near(part(p, i, j).v.T, part(p, i, j).e.T)).map2(part(q, i, j), np.matmul, j - i)

    each(outer(dy, h), False).rounded().check(got["dw2"], "dw2")
    dh = each(lambda e, i, j: part(dy, i, j).map2(Near(W2[e]), np.matmul, cols), True).rounded()
    da = Near(2 * a.v, 2 * a.e).map2(dh, np.multiply, 0).rounded()
    each(outer(da, rows), False).rounded().check(got["dw1"], "dw1")
    drows = each(lambda e, i, j: part(da, i, j).map2(Near(W1[e]), np.matmul, hidden), True).rounded()
    sum_by_token(drows, 1.0).check(got["dx"], "dx")
    gone = (weights == 0).all(1)
    assert (f64(got["out"])[gone] == 0).all() and (f64(got["dx"])[gone] == 0).all()


def test_layer_8bit(ro):
    """The serving layer in e4m3: each product is within its own bound of the 64-bit product of its bytes."""
    rng = np.random.default_rng(3)
    x, logits, mask, w1, w2, _ = inputs(rng, 50, 6, 160, 144)
    p = ro.rowops_masked_softmax(logits, mask)
    weights, indices = ro.rowops_top_k_rows(p, 2)
    offsets, order, slot = ro.rowops_expert_plan(indices, 6, values=weights)
    bounds = offsets.cpu().numpy()
    n = bounds[-1]
    rows = ro.rowops_expert_gather(x, slot, dtype=torch.bfloat16)
    y = None
    for w in (w1, w2):
        q, s = ro.rowops_quantize_blocks(rows)
        wq, ws = ro.rowops_quantize_blocks(w, block_rows=128)
        y = ro.rowops_expert_matmul_fp8(q, s, wq, ws, offsets)
        x64 = f64(q.float())[:n] * expert_ref.spread(f64(s), 1, len(rows), w.shape[2])[:n]
        w64 = f64(wq.float()) * expert_ref.spread(f64(ws), 128, w.shape[1], w.shape[2])
        want = expert_ref.matmul(x64, w64, bounds)
        terms = expert_ref.matmul(abs(x64), abs(w64), bounds)
        assert (np.abs(f64(y)[:n] - want) <= 2.0 ** -8 * np.abs(want) + 140 * 2.0 ** -23 * terms).all()
        rows = y
    out = ro.rowops_expert_combine(y, slot, weights=weights, dtype=torch.float32)
    assert torch.isfinite(out).all() and (out[::7] == 0).all()


@pytest.mark.parametrize("tokens", [40, 3000])  # a plan of one launch, and of two
def test_graph(ro, tokens):
    """Captured once, replayed on new inputs: bit for bit what eager calls give."""
    rng = np.random.default_rng(tokens)
    static = inputs(rng, tokens, 8, 64, 96)
    layer(ro, *static[:5], 2, static[5])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer(ro, *static[:5], 2, static[5])
    for _ in range(3):
        fresh = inputs(rng, tokens, 8, 64, 96)
        for a, b in zip(static, fresh):
            a.copy_(b)
        graph.replay()
        want = layer(ro, *fresh[:5], 2, fresh[5])
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(captured[name], want[name]), name
    assert ro.library().rowops_pipeline_timeouts() == 0


def test_two_graphs_and_eager_calls_at_once(ro):
    """Two captured graphs with their own workspaces replayed on two streams while eager calls run on a third."""
    rng = np.random.default_rng(5)
    sets = [inputs(rng, 2500, 8, 65, 90) for _ in range(3)]  # odd widths: products with workspaces
    want = [layer(ro, *s[:5], 2, s[5]) for s in sets]
    torch.cuda.synchronize()
    graphs = []
    for s in sets[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer(ro, *s[:5], 2, s[5])
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        for (g, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = layer(ro, *sets[2][:5], 2, sets[2][5])
    torch.cuda.synchronize()
    for got, ref in zip([graphs[0][1], graphs[1][1], eager], want):
        for name in ref:
            assert torch.equal(got[name], ref[name]), name


def test_repeats_bit_for_bit(ro):
    rng = np.random.default_rng(6)
    s = inputs(rng, 5000, 16, 96, 136)
    first = layer(ro, *s[:5], 4, s[5])
    for _ in range(3):
        again = layer(ro, *s[:5], 4, s[5])
        assert all(torch.equal(first[name], again[name]) for name in first)


def test_stream_argument(ro):
    """A call on a named stream (object or handle) after work that only that stream orders."""
    side = torch.cuda.Stream()
    x, w = torch.zeros(600, 65, device="cuda").half(), torch.ones(1, 50, 65, device="cuda").half()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            x.zero_()
            torch.cuda._sleep(20_000_000)
            x.fill_(1.0)
        y = ro.rowops_expert_matmul(x, w, stream=stream)
        side.synchronize()
        assert (y == 65).all()
        idx = torch.zeros(5000, 1, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            idx.fill_(3.0)
        offsets, _, slot = ro.rowops_expert_plan(idx, 4, stream=stream)
        side.synchronize()
        assert offsets.tolist() == [0, 0, 0, 0, 5000] and torch.equal(slot[:, 0].cpu(), torch.arange(5000).int())


def test_guard_bands(ro):
    """Outputs between bands of a fixed pattern, which stay, over the kernels' shapes."""
    rng = np.random.default_rng(8)

    def banded(shape, dtype):
        n = int(np.prod(shape)) * dtype.itemsize
        buf = torch.full((n + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
        return buf, buf[4096:4096 + n].view(dtype).view(shape)

    def intact(buf):
        return bool((buf[:4096] == 0x5A).all() and (buf[-4096:] == 0x5A).all())

    for sizes, cin, cout in (([100, 0, 41, 300], 64, 200), ([5], 40, 24), ([31, 290], 136, 264), ([70, 9], 33, 50)):
        rows = sum(sizes)
        at = torch.from_numpy(np.cumsum([0] + sizes).astype(np.int32)).cuda()
        x = torch.from_numpy(rng.normal(size=(rows, cin))).cuda().half()
        dy = torch.from_numpy(rng.normal(size=(rows, cout))).cuda().half()
        w = torch.from_numpy(rng.normal(size=(len(sizes), cout, cin))).cuda().half()
        for shape, dtype, call in (((rows, cout), torch.float16, lambda o: ro.rowops_expert_matmul(x, w, at, y=o)),
                                   ((rows, cin), torch.float16,
                                    lambda o: ro.rowops_expert_matmul(dy, w, at, y=o, transposed=True)),
                                   (w.shape, torch.float16, lambda o: ro.rowops_expert_matmul_wgrad(dy, x, at, dw=o)),
                                   (w.shape, torch.float32, lambda o: ro.rowops_expert_matmul_wgrad(dy, x, at, dw=o))):
            buf, out = banded(tuple(shape), dtype)
            call(out)
            assert intact(buf)
        xq, xs = ro.rowops_quantize_blocks(x)
        wq, ws = ro.rowops_quantize_blocks(w, block_rows=128)
        for dtype in (torch.bfloat16, torch.float32):
            buf, out = banded((rows, cout), dtype)
            ro.rowops_expert_matmul_fp8(xq, xs, wq, ws, at, y=out)
            assert intact(buf)
        for block in (1, 128):
            qbuf, q = banded(tuple(w.shape), torch.float8_e4m3fn)
            sbuf, s = banded((len(sizes), -(-cout // block), -(-cin // 128)), torch.float32)
            ro.rowops_quantize_blocks(w, block_rows=block, q=q, scale=s)
            assert intact(qbuf) and intact(sbuf)
    for tokens, k, experts in ((33, 2, 7), (5000, 3, 1024)):
        idx = torch.from_numpy(rng.integers(0, experts, (tokens, k)).astype(np.float32)).cuda()
        bufs = [banded(shape, torch.int32) for shape in ((experts + 1,), (tokens * k,), (tokens, k))]
        ro.rowops_expert_plan(idx, experts, offsets=bufs[0][1], order=bufs[1][1], slot=bufs[2][1])
        assert all(intact(b) for b, _ in bufs)


def test_more_than_32_bits(ro):
    """Matrices of more than 2^32 bytes: sampled rows and weights against 64 bits."""
    slots, cin, cout = 300_000, 8192, 64  # x: 2.46e9 values, 4.9e9 bytes
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(slots, cin, dtype=torch.float16, device="cuda")
    for r in range(0, slots, 50_000):
        x[r:r + 50_000] = torch.randint(-1, 2, (50_000, cin), generator=g, device="cuda").half()
    w = torch.randint(-1, 2, (2, cout, cin), generator=g, device="cuda").half()
    at = torch.tensor([0, 100_001, slots], dtype=torch.int32, device="cuda")
    y = ro.rowops_expert_matmul(x, w, at)
    for r in (0, 100_000, 100_001, 262_143, 262_145, slots - 1):
        e = int(r >= 100_001)
        assert torch.equal(y[r].double(), (w[e].double() @ x[r].double()).half().double()), r
    back = ro.rowops_expert_matmul(y.sign(), w, at, transposed=True)  # an output of more than 2^32 bytes
    for r in (0, 100_001, slots - 1):
        e = int(r >= 100_001)
        assert torch.equal(back[r].double(), (w[e].double().T @ y[r].sign().double()).half().double()), r
    slot = torch.arange(slots, dtype=torch.int32, device="cuda").flip(0)[:, None].contiguous()
    ro.rowops_expert_gather(x, slot, out=back)
    assert torch.equal(back[0], x[-1]) and torch.equal(back[-1], x[0]) and torch.equal(back[270_000], x[29_999])
    q, s = ro.rowops_quantize_blocks(x)
    assert torch.equal(q[-1].float() * s[-1].repeat_interleave(128), x[-1].float())
    wq, ws = ro.rowops_quantize_blocks(w, block_rows=128)
    y8 = ro.rowops_expert_matmul_fp8(q, s, wq, ws, at, dtype=torch.float32)
    assert torch.allclose(y8[-1], y[-1].float(), rtol=0, atol=1e-2)  # values are +-1: scales of 1 / 448 both ways
