"""Dropout, the residual's norm and the quantised products together, as a layer runs
them; replayed as CUDA graphs, on other streams, from several threads, and with more
than 2^32 values.

The training step's bound is propagated stage by stage as in test_gpu_expert_layer: a
product of K terms is off by (K + 8) 2^-23 of the magnitudes summed and what its
operands' errors make of it, a norm by what test_gpu_add_rmsnorm derives, and each
16-bit result by u = 2^-8 of its value.  The serving layers' products are compared with
the 64-bit products of the bytes that the norm answered."""
import threading

import numpy as np
import pytest
import torch

import branch_ref
import expert_ref
from test_gpu_add_rmsnorm import EPS, U, chain, forward_bounds
from test_gpu_dropout import rng_of
from test_gpu_expert_matmul import TINY, UNIT, f64
from test_gpu_mx4 import values

pytestmark = pytest.mark.gpu

P = 0.2


def inputs(seed, rows, cols, hidden, dtype=torch.bfloat16):
    g = np.random.default_rng(seed)

    def cuda(shape, scale=1.0, t=dtype):
        return torch.from_numpy(g.normal(size=shape) * scale).cuda().to(t)

    return dict(x=cuda((rows, cols)), residual=cuda((rows, cols), 2.0, torch.float32), gamma=1 + cuda(cols, 0.1, torch.float32),
                w=cuda((1, hidden, cols), cols ** -0.5), dz=cuda((rows, hidden)), dh=cuda((rows, cols), 1.0, torch.float32),
                rng=torch.from_numpy(g.integers(-2 ** 62, 2 ** 62, 2)).cuda())


def step(ro, s):
    """One sublayer's training step: norm, product, and the gradients of all."""
    y, _, h, rms = ro.rowops_add_rmsnorm_fwd(s["x"], s["gamma"], residual=s["residual"], rng=s["rng"], p=P, eps=EPS)
    z = ro.rowops_expert_matmul(y, s["w"])
    dw = ro.rowops_expert_matmul_wgrad(s["dz"], y, dtype=torch.float32)
    dy = ro.rowops_expert_matmul(s["dz"], s["w"], transposed=True)
    dx, dresidual, dgamma = ro.rowops_add_rmsnorm_bwd(dy, s["gamma"], h, rms, dh=s["dh"], rng=s["rng"], p=P)
    again = ro.rowops_dropout(s["x"], s["rng"], P, residual=s["residual"])  # the same mask by itself
    return {"y": y, "h": h, "z": z, "dw": dw, "dy": dy, "dx": dx, "dresidual": dresidual, "dgamma": dgamma, "again": again}


def serve(ro, s, quantize):
    """Norm to quantised rows and the product that takes them."""
    q, scale, h, _ = ro.rowops_add_rmsnorm_fwd(s["x"], s["gamma"], residual=s["residual"], quantize=quantize)
    if quantize == "e4m3":
        wq, ws = ro.rowops_quantize_blocks(s["w"], block_rows=128)
        z = ro.rowops_expert_matmul_fp8(q, scale, wq, ws)
    else:
        wq, ws = ro.rowops_quantize_mx4(s["w"])
        z = ro.rowops_expert_matmul_mx4(q, scale, wq, ws)
    return {"q": q, "scale": scale, "h": h, "wq": wq, "ws": ws, "z": z}


@pytest.mark.parametrize("rows,cols,hidden", [(1, 64, 96), (37, 200, 72), (700, 768, 256), (130, 33, 57)])
def test_training_step(ro, rows, cols, hidden):
    s = inputs(rows, rows, cols, hidden)
    got = step(ro, s)
    key = tuple(int(v) for v in s["rng"].cpu())
    (h64, eh), (rms, erms), (y64, ey) = forward_bounds(s["x"], s["residual"], s["gamma"], key, P)
    u = UNIT["bf16"]

    def check(name, want, e, unit=0.0, tiny=0.0):
        far = np.abs(f64(got[name]) - want)
        limit = 1.01 * e + unit * np.abs(want) + tiny
        assert (far <= limit).all(), f"{name}: {(far / np.maximum(limit, 1e-300)).max()} times the bound"

    check("h", h64, eh, U)
    assert torch.equal(got["again"], got["h"])
    y_err = ey * (1 + u) + u * np.abs(y64) + TINY["bf16"]
    check("y", y64, y_err)
    w64, dz64 = f64(s["w"])[0], f64(s["dz"])

    def product(a, ea, b, k):  # b exact
        terms = (np.abs(a) + ea) @ np.abs(b)
        return a @ b, ea @ np.abs(b) + (k + 8) * 2.0 ** -23 * terms

    z, ez = product(y64, y_err, w64.T, cols)
    check("z", z, ez * (1 + u), u, TINY["bf16"])
    dw, edw = product(dz64.T, 0 * dz64.T, y64, rows)
    check("dw", dw[None], edw + np.abs(dz64.T) @ y_err, U)
    dy, edy = product(dz64, 0 * dz64, w64, hidden)
    edy = edy * (1 + u) + u * np.abs(dy) + TINY["bf16"]
    check("dy", dy, edy)
    # the backward pass takes the dy, h and rms that were computed: its own bound around those
    dy64, hh, gamma = f64(got["dy"]), f64(got["h"]), f64(s["gamma"])
    _, _, _, rms_t = ro.rowops_add_rmsnorm_fwd(s["x"], s["gamma"], residual=s["residual"], rng=s["rng"], p=P, eps=EPS)
    rms64 = f64(rms_t)
    wdx, wres, wgamma = branch_ref.add_norm_bwd(dy64, gamma, hh, rms64, f64(s["dh"]), key, P)
    n, gy, inv = np.abs(hh) / rms64[:, None], np.abs(dy64 * gamma), 1 / rms64[:, None]
    e = U * (inv * (7 * gy + n * (gy * n).mean(1, keepdims=True) * (chain(cols) + 12)) + np.abs(wres) + np.abs(f64(s["dh"])))
    check("dresidual", wres, e, U)
    scale = 65536 / (65536 - branch_ref.threshold(P))
    check("dx", wdx, np.where(wdx != 0, scale * (e + 2 * U * np.abs(wres)), 0) * (1 + u), u, TINY["bf16"])
    check("dgamma", wgamma, (rows + 10) * U * (np.abs(dy64) * n).sum(0), U)


@pytest.mark.parametrize("rows,cols,hidden", [(1, 128, 64), (40, 768, 256), (700, 256, 384), (33, 97, 50)])
@pytest.mark.parametrize("quantize", ["e4m3", "mx4"])
def test_serving_layer(ro, rows, cols, hidden, quantize):
    s = inputs(rows + 1, rows, cols, hidden)
    got = serve(ro, s, quantize)
    if quantize == "e4m3":
        x64 = f64(got["q"].float()) * expert_ref.spread(f64(got["scale"]), 1, rows, cols)
        w64 = f64(got["wq"].float()) * expert_ref.spread(f64(got["ws"]), 128, hidden, cols)
    else:
        x64, w64 = values(got["q"], got["scale"], cols), values(got["wq"], got["ws"], cols)
    want, terms = x64 @ w64[0].T, np.abs(x64) @ np.abs(w64[0]).T
    slack = (cols + 16 + cols / 64) * 2.0 ** -23
    u = UNIT["bf16"]
    assert (np.abs(f64(got["z"]) - want) <= u * np.abs(want) + (1 + u) * slack * terms + TINY["bf16"]).all()


def test_graph_drops_anew(ro):
    """Captured once with the generator's offset advanced in the graph; replays on new inputs are what eager calls give."""
    static = inputs(5, 600, 136, 72)
    step(ro, static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(ro, static)
        served = serve(ro, static, "mx4")
        static["rng"][1:].add_(1)
    masks = []
    for i in range(3):
        fresh = inputs(50 + i, 600, 136, 72)
        if i:
            fresh["rng"].copy_(static["rng"])  # as the last replay left it
        for name in static:
            static[name].copy_(fresh[name])
        graph.replay()
        want = step(ro, fresh)
        want_served = serve(ro, fresh, "mx4")
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(captured[name], want[name]), name
        for name in want_served:
            assert torch.equal(served[name], want_served[name]), name
        assert int(static["rng"][1]) == int(fresh["rng"][1]) + 1
        masks.append((captured["dx"] == 0).clone())
    assert not torch.equal(masks[1], masks[2])
    assert ro.library().rowops_pipeline_timeouts() == 0


def test_two_graphs_and_eager_calls_at_once(ro):
    """Two captured graphs replayed on two streams while eager calls run on a third; odd widths take workspaces."""
    sets = [inputs(70 + i, 900, 65, 90) for i in range(3)]

    def work(s):
        out = step(ro, s)
        out.update(serve(ro, s, "mx4"))
        out.update({"8bit " + k: v for k, v in serve(ro, s, "e4m3").items()})
        return out

    want = [work(s) for s in sets]
    torch.cuda.synchronize()
    graphs = []
    for s in sets[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = work(s)
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        for (g, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = work(sets[2])
    torch.cuda.synchronize()
    for got, ref in zip([graphs[0][1], graphs[1][1], eager], want):
        for name in ref:
            assert torch.equal(got[name].view(torch.uint8), ref[name].view(torch.uint8)), name


def test_stream_argument(ro):
    """Calls on a named stream (object or handle) after work that only that stream orders."""
    side = torch.cuda.Stream()
    x, gamma = torch.zeros(600, 64, device="cuda"), torch.ones(64, device="cuda")
    rng = rng_of(1, 2)
    wq, ws = ro.rowops_quantize_mx4(torch.ones(1, 32, 64, device="cuda"))
    rms = torch.ones(600, device="cuda")

    def late():
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            x.zero_()
            torch.cuda._sleep(20_000_000)
            x.fill_(1.0)

    for stream in (side, side.cuda_stream):
        late()
        y = ro.rowops_dropout(x, rng, 0.0, stream=stream)
        side.synchronize()
        assert (y == 1).all()
        late()
        q, s = ro.rowops_quantize_mx4(x, stream=stream)
        z = ro.rowops_expert_matmul_mx4(q, s, wq, ws, dtype=torch.float32, stream=stream)
        side.synchronize()
        assert (z == 64).all()
        late()
        out, _, h, _ = ro.rowops_add_rmsnorm_fwd(x, gamma, residual=x, eps=0.0, stream=stream)
        side.synchronize()
        assert (out == 1).all() and (h == 2).all()
        late()
        dx, _, dgamma = ro.rowops_add_rmsnorm_bwd(x, gamma, x, rms, stream=stream)
        side.synchronize()
        assert (dx == 0).all() and (dgamma == 600).all()


def test_threads(ro):
    """Three threads with streams of their own: every call gives what it gives alone."""
    sets = [inputs(80, 900, 264, 96), inputs(81, 33, 4104, 130), inputs(82, 3000, 72, 40)]
    jobs = [lambda s=s: {**step(ro, s), **serve(ro, s, "mx4")} for s in sets]
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    failed, got, gate = [], [[] for _ in jobs], threading.Barrier(len(jobs))

    def loop(job, out):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait()
                for _ in range(20):
                    out.append(job())
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 - raised again below
            failed.append(e)

    threads = [threading.Thread(target=loop, args=a) for a in zip(jobs, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[0]
    for outs, ref in zip(got, want):
        assert len(outs) == 20
        for out in outs:
            assert all(torch.equal(out[name], ref[name]) for name in ref)
    assert ro.library().rowops_pipeline_timeouts() == 0


def test_more_than_32_bits(ro):
    """Matrices of more than 2^32 values: sampled rows against 64 bits."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    rows, cols = 1_050_000, 4096  # 4.3e9 values
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for r in range(0, rows, 50_000):
        x[r:r + 50_000] = torch.randint(-2, 3, (50_000, cols), generator=g, device="cuda").bfloat16()
    gamma = torch.ones(cols, device="cuda")
    q, scale, h, rms = ro.rowops_add_rmsnorm_fwd(x, gamma, quantize="mx4")
    assert h is x
    probe = [0, 524_287, 524_289, rows - 1]
    for r in probe:
        x64 = f64(x[r])
        want = np.sqrt((x64 * x64).mean() + 1e-5)
        assert abs(float(rms[r]) - want) < 30 * U * want
        val, code = branch_ref.quantize_mx4((x64 / float(rms[r]))[None])
        assert (scale[r].cpu().numpy() == code[0]).all() and (branch_ref.unpack_mx4(q[r].cpu().numpy(), cols) == val[0]).all()
    wq, ws = ro.rowops_quantize_mx4(torch.randint(-2, 3, (2, 64, cols), generator=g, device="cuda").float())
    at = torch.tensor([0, 524_288, rows], dtype=torch.int32, device="cuda")
    y = ro.rowops_expert_matmul_mx4(q, scale, wq, ws, at, dtype=torch.float32)
    for r in probe:
        a = values(q[r][None], scale[r][None], cols)
        w = values(wq[int(r >= 524_288)], ws[int(r >= 524_288)], cols)
        assert (np.abs(f64(y[r]) - (a @ w.T)[0]) <= (cols + 8) * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T)[0]).all()
    dx, dres, dgamma = ro.rowops_add_rmsnorm_bwd(x, gamma, x, rms)
    assert dx is dres
    for r in probe:
        x64, m = f64(x[r])[None], float(rms[r])
        want = branch_ref.add_norm_bwd(x64, np.ones(cols), x64, np.array([m]), None, (0, 0), 0.0)[1]
        # a mean of cols magnitudes in chains of 40, and eight operations
        e = U * (8 * np.abs(x64) + np.abs(x64) / m * (x64 * x64 / m).mean() * 60) / m + UNIT["bf16"] * np.abs(want)
        assert (np.abs(f64(dx[r]) - want[0]) <= e[0] + TINY["bf16"]).all()
    total = torch.zeros(cols, dtype=torch.float64, device="cuda")
    for r in range(0, rows, 50_000):
        total += (x[r:r + 50_000].double().square() / rms[r:r + 50_000, None].double()).sum(0)
    # 152 blocks of 6908 rows: at most that many additions of positive terms in a row
    assert ((dgamma.double() - total).abs() <= 7000 * U * total).all()
