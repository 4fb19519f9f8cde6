"""The compiled binding on tensors that have no storage of their own, as function transforms
and tracing hand them over: each call raises, and the process lives on."""
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

CHILD = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import row_wise_softmax_warp_gb300 as ro

x, rms = torch.ones(3, 4, 32, device="cuda"), torch.ones(3, 4, device="cuda")
gamma, rng = torch.ones(32, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
q, s = ro.rowops_quantize_mx4(x)
wq, ws = ro.rowops_quantize_mx4(torch.ones(1, 8, 32, device="cuda"))
calls = [(lambda t: ro.rowops_quantize_mx4(t), x), (lambda t: ro.rowops_dropout(t, rng, 0.5), x),
         (lambda t: ro.rowops_add_rmsnorm_fwd(t, gamma), x),
         (lambda t: ro.rowops_add_rmsnorm_bwd(t, gamma, x[0], rms[0]), x),
         (lambda t: ro.rowops_expert_matmul_mx4(t, s[0], wq, ws), q)]
for f, over in calls:
    try:
        torch.func.vmap(f)(over)
    except (RuntimeError, TypeError, ValueError):
        print("raised")
with FakeTensorMode():
    fake = torch.empty(4, 32, device="cuda")
    try:
        ro.rowops_dropout(fake, None, 0.0)
    except (RuntimeError, TypeError, ValueError):
        print("raised")
assert (ro.rowops_dropout(x, None, 0.0) == 1).all()
print("lives on")
"""


def test_tensors_without_storage(ro):
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split("\n")[-2] == "lives on" and r.stdout.count("raised") >= 5
