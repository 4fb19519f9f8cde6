"""The expert operators at their limits: sums so long that one wait spans most of
the kernel, and the wait itself."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import expert_ref

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "row_wise_softmax_warp_gb300", "csrc")


def compiled(tmp, name):
    """tests/csrc/<name>.cu as a shared library."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    out = str(tmp / (name + ".so"))
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "--expt-relaxed-constexpr",
                    "-I", CSRC, "-I", os.path.join(HERE, "..", "include"), "-shared", "-Xcompiler", "-fPIC", "-o", out,
                    os.path.join(HERE, "csrc", name + ".cu")], check=True, capture_output=True)
    return ctypes.CDLL(out)


@pytest.fixture(scope="module")
def wait(tmp_path_factory):
    lib = compiled(tmp_path_factory.mktemp("wait_probe"), "wait_probe")
    lib.run_wait_probe.argtypes = [ctypes.c_uint32, ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p]

    def run(polls, steps, gap, arrive):
        out = torch.full((2,), -1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        before = lib.run_wait_probe_timeouts()
        assert lib.run_wait_probe(polls, steps, gap, arrive, out.data_ptr()) == 0
        return (*out.tolist(), lib.run_wait_probe_timeouts() - before)

    return run


POLLS = 1 << 14  # 35 clocks each: 0.6 million in all


def test_wait_outlasts_its_polls_while_stages_pass(wait):
    """100 steps of 50000 clocks, eight times the polls' own time."""
    assert wait(POLLS, 100, 50_000, 1) == (1, 0, 0)


def test_wait_runs_out_where_nothing_moves(wait):
    """Nothing arrives: an answer, the abort flag and one timeout counted."""
    assert wait(POLLS, 0, 0, 0) == (0, 1, 1)
    assert wait(POLLS, 20, 50_000, 0) == (0, 1, 1)


def alternating(shape, along, dtype=torch.bfloat16):
    """+1, -1, +1, ... along a dimension."""
    n = shape[along]
    v = torch.ones(n, dtype=dtype, device="cuda")
    v[1::2] = -1
    return v.view([n if i == along else 1 for i in range(len(shape))]).expand(shape).contiguous()


LONG = 1 << 26  # 2^20 stages of 0.25 us in one cluster: some four times the polls of one wait on an idle SM


def room():
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")


def test_long_sums_of_weights(ro):
    """One expert of 2^26 rows, a multiple of 16, before 200 of 7: the epilogue waits for its whole sum, and the
    warp that zeroes the last rows of the 7 waits for it too."""
    room()
    before = ro.library().rowops_pipeline_timeouts()
    rows = LONG + 200 * 7
    x, dy = alternating((rows, 8), 0), torch.ones(rows, 8, dtype=torch.bfloat16, device="cuda")
    x[LONG - 3], x[LONG - 9] = 5, 7  # for -1 each
    at = torch.from_numpy(np.cumsum([0, LONG] + [7] * 200).astype(np.int32)).cuda()
    dw = ro.rowops_expert_matmul_wgrad(dy, x, at, dtype=torch.float32)
    assert ro.library().rowops_pipeline_timeouts() == before
    assert (dw[0] == 14).all()
    assert (dw[1::2] == 1).all() and (dw[2::2] == -1).all()


@pytest.mark.parametrize("transposed", [False, True])
def test_long_sums_of_rows(ro, transposed):
    room()
    before = ro.library().rowops_pipeline_timeouts()
    x = alternating((3, LONG), 1)
    x[1, LONG - 3], x[2, LONG - 9] = 5, 7
    w = torch.ones(1, LONG, 8, dtype=torch.bfloat16, device="cuda")
    if not transposed:
        w = w.view(1, 8, LONG)
    y = ro.rowops_expert_matmul(x, w, transposed=transposed)
    assert ro.library().rowops_pipeline_timeouts() == before
    assert y.tolist() == [[0.0] * 8, [6.0] * 8, [8.0] * 8]


@pytest.mark.parametrize("experts", [225, 449, 1024])
def test_many_experts(ro, experts):
    """More experts than a block of the products has threads: whole numbers, so sums are exact."""
    rng = np.random.default_rng(experts)
    sizes = rng.choice([0, 0, 1, 2, 7, 33], experts)
    sizes[0], sizes[-1], sizes[experts // 2] = 3, 5, 300
    offsets = np.cumsum([0, *sizes]).astype(np.int32)
    at, rows = torch.from_numpy(offsets).cuda(), int(offsets[-1])
    x, w, dy = (torch.from_numpy(rng.integers(-1, 2, shape).astype(np.float32)).cuda().half()
                for shape in ((rows, 128), (experts, 136, 128), (rows, 136)))
    x64, w64, dy64 = (t.double().cpu().numpy() for t in (x, w, dy))
    want = expert_ref.matmul(x64, w64, offsets)
    assert (ro.rowops_expert_matmul(x, w, at).double().cpu().numpy() == want).all()
    dx = ro.rowops_expert_matmul(dy, w, at, transposed=True)
    assert (dx.double().cpu().numpy() == expert_ref.matmul(dy64, w64.transpose(0, 2, 1), offsets)).all()
    dw = ro.rowops_expert_matmul_wgrad(dy, x, at)
    assert (dw.double().cpu().numpy() == expert_ref.wgrad(dy64, x64, offsets)).all()
    # -1, 0 and 1 are exact in e4m3; with scales of powers of two so are the products
    xs = torch.full((rows, 1), 2.0, device="cuda")
    ws = torch.from_numpy(2.0 ** rng.integers(-2, 3, (experts, 2, 1))).float().cuda()
    y = ro.rowops_expert_matmul_fp8(x.to(torch.float8_e4m3fn), xs, w.to(torch.float8_e4m3fn), ws, at,
                                    dtype=torch.float32)
    scale = 2.0 * expert_ref.spread(ws.double().cpu().numpy(), 128, 136, 1)
    assert (y.double().cpu().numpy() == expert_ref.matmul(x64, w64 * scale, offsets)).all()


def test_plans_that_need_no_workspace(ro):
    """The binding asks for a workspace only above the pairs that the header names."""
    from row_wise_softmax_warp_gb300 import binding
    most = binding._ONE_LAUNCH_PAIRS
    for k in (1, 2, 8):
        assert ro.rowops_expert_plan_workspace(most // k, k, 1024) == 0
        assert ro.rowops_expert_plan_workspace(most // k + 1, k, 1024) > 0
