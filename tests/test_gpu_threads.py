"""Rows of different lengths from several host threads at once: the long-row kernels
need a ring of another size for each length, and every call gives what it gives alone."""
import ctypes
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


class RowCall(ctypes.Structure):
    _fields_ = [("pointers", ctypes.c_void_p * 3), ("sizes", ctypes.c_int64 * 2), ("stream", ctypes.c_void_p)]


@pytest.fixture(scope="module")
def row_threads(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("row_threads") / "row_threads.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-pthread", "-shared", "-fPIC", "-o", out,
                    os.path.join(HERE, "csrc", "row_threads.cpp")], check=True, capture_output=True)
    return ctypes.CDLL(out).row_threads


@pytest.mark.parametrize("backward", [False, True])
def test_softmax_of_different_lengths(ro, row_threads, backward):
    op = "rowops_softmax_bwd" if backward else "rowops_softmax_fwd"
    calls, kept = [], []
    for cols in (17000, 25000, 33000, 52000):
        g = torch.Generator(device="cuda").manual_seed(cols)
        a, b = torch.softmax(torch.randn(4, cols, generator=g, device="cuda"), 1), torch.randn(4, cols, generator=g, device="cuda")
        ins = (a, b) if backward else (b,)
        want, out, stream = getattr(ro, op)(*ins), torch.empty_like(a), torch.cuda.Stream()
        calls.append(RowCall((ctypes.c_void_p * 3)(ins[0].data_ptr(), ins[-1].data_ptr(), out.data_ptr()),
                             (ctypes.c_int64 * 2)(4, cols), stream.cuda_stream))
        kept.append((ins, want, out, stream))
    torch.cuda.synchronize()
    fn = ctypes.cast(getattr(ro.library(), op), ctypes.c_void_p)
    assert row_threads(fn, int(backward), (RowCall * len(calls))(*calls), len(calls), 2000) == 0
    torch.cuda.synchronize()
    for _, want, out, _ in kept:
        assert torch.equal(out, want)
    assert ro.library().rowops_pipeline_timeouts() == 0
