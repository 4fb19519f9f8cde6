"""Calls of several host threads at once, each with its own stream, buffers and
workspace: every one gives what it gives alone."""
import ctypes
import os
import subprocess
import threading

import numpy as np
import pytest
import torch

import expert_ref

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


class PlanCall(ctypes.Structure):
    _fields_ = [("pointers", ctypes.c_void_p * 5), ("sizes", ctypes.c_int64 * 3), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p)]


@pytest.fixture(scope="module")
def plan_threads(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("plan_threads") / "plan_threads.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-pthread", "-shared", "-fPIC", "-o", out,
                    os.path.join(HERE, "csrc", "plan_threads.cpp")], check=True, capture_output=True)
    return ctypes.CDLL(out).plan_threads


@pytest.mark.parametrize("tokens", [1000, 5000])  # a plan of one launch, and of two
def test_plans_of_different_numbers_of_experts(ro, plan_threads, tokens):
    """Each number of experts needs another amount of shared memory; threads that hold no lock between calls."""
    rng = np.random.default_rng(tokens)
    calls, kept = [], []
    for experts in (1024, 512, 1024, 700):
        indices = rng.integers(0, experts, (tokens, 2)).astype(np.float32)
        idx = torch.from_numpy(indices).cuda()
        out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (experts + 1, 2 * tokens, 2 * tokens)]
        ws = torch.empty(max(1, ro.rowops_expert_plan_workspace(tokens, 2, experts)), dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        calls.append(PlanCall((ctypes.c_void_p * 5)(idx.data_ptr(), None, *(o.data_ptr() for o in out)),
                              (ctypes.c_int64 * 3)(tokens, 2, experts), ws.data_ptr(), ws.numel(), stream.cuda_stream))
        kept.append((idx, out, ws, stream, expert_ref.plan(indices, None, experts)))
    torch.cuda.synchronize()
    fn = ctypes.cast(ro.library().rowops_expert_plan, ctypes.c_void_p)
    assert plan_threads(fn, (PlanCall * len(calls))(*calls), len(calls), 2000) == 0
    torch.cuda.synchronize()
    for _, out, _, _, want in kept:
        for a, b in zip(out, want):
            assert (a.cpu().numpy() == b.reshape(-1)).all()


def test_layers_in_threads(ro):
    """A layer's calls from three threads through the binding, of sizes and types of their own."""
    rng = np.random.default_rng(2)
    works, checks = [], []
    for tokens, experts, cols, hidden, dtype in ((900, 300, 64, 96, torch.float16), (3000, 8, 65, 130, torch.bfloat16),
                                                 (64, 450, 136, 72, torch.float16)):
        x = torch.from_numpy(rng.normal(size=(tokens, cols)).astype(np.float32)).cuda()
        w = torch.from_numpy(rng.normal(size=(experts, hidden, cols))).cuda().to(dtype)
        idx = torch.from_numpy(rng.integers(0, experts, (tokens, 2)).astype(np.float32)).cuda()
        scale = torch.from_numpy(rng.random((tokens, 2)).astype(np.float32)).cuda()

        def layer(x=x, w=w, idx=idx, scale=scale, dtype=dtype):
            offsets, _, slot = ro.rowops_expert_plan(idx, w.shape[0], values=scale)
            rows = ro.rowops_expert_gather(x, slot, out=torch.zeros(idx.numel(), x.shape[1], dtype=dtype, device="cuda"))
            y = ro.rowops_expert_matmul(rows, w, offsets, y=torch.zeros(len(rows), w.shape[1], dtype=dtype, device="cuda"))
            dw = ro.rowops_expert_matmul_wgrad(y, rows, offsets)
            q, qs = ro.rowops_quantize_blocks(rows)
            wq, ws = ro.rowops_quantize_blocks(w, block_rows=128)
            y8 = ro.rowops_expert_matmul_fp8(q, qs, wq, ws, offsets, y=torch.zeros_like(y))
            return ro.rowops_expert_combine(y, slot, weights=scale, dtype=torch.float32), dw, y8

        want = layer()
        got = []
        works.append(lambda layer=layer, got=got: got.append(layer()))
        checks.append((got, want))
    torch.cuda.synchronize()
    failed, gate = [], threading.Barrier(len(works))

    def loop(work):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait()
                for _ in range(20):
                    work()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 - raised again below
            failed.append(e)

    threads = [threading.Thread(target=loop, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[0]
    for got, want in checks:
        assert len(got) == 20 and all(torch.equal(a, b) for outs in got for a, b in zip(outs, want))
    assert ro.library().rowops_pipeline_timeouts() == 0
