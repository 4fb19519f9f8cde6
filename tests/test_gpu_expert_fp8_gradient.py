"""The rows' gradient of the 8-bit product by the call that the header names: the
forward call on dy with the weights' bytes and scales transposed within each expert."""
import numpy as np
import pytest
import torch

import expert_ref
from test_gpu_expert_fp8 import check
from test_gpu_expert_matmul import TYPES, f64, offsets_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("widths", [(128, 128), (768, 256), (144, 520), (33, 50)])
def test_gradient_of_the_rows(ro, widths, out):
    cin, cout = widths
    sizes, rng = [40, 0, 300, 1], np.random.default_rng(cin)
    offsets, rows = offsets_of(sizes), sum(sizes)
    at = torch.from_numpy(offsets).cuda()
    w = torch.from_numpy(rng.normal(size=(len(sizes), cout, cin)) * np.exp2(rng.integers(-3, 4, (4, 1, 1)))).cuda().half()
    dy = torch.from_numpy(rng.normal(size=(rows, cout))).cuda().bfloat16()
    wq, ws = ro.rowops_quantize_blocks(w, block_rows=128)
    dq, ds = ro.rowops_quantize_blocks(dy)
    turned = wq.view(torch.uint8).transpose(1, 2).contiguous().view(torch.float8_e4m3fn)
    dx = ro.rowops_expert_matmul_fp8(dq, ds, turned, ws.transpose(1, 2).contiguous(), at, dtype=TYPES[out])
    # the same quantised weights as the forward call's, so the gradient is of what it computes
    w64 = (f64(wq.float()) * expert_ref.spread(f64(ws), 128, cout, cin)).transpose(0, 2, 1)
    dy64 = f64(dq.float()) * expert_ref.spread(f64(ds), 1, rows, cout)
    check(dx, expert_ref.matmul(dy64, w64, offsets), expert_ref.matmul(abs(dy64), abs(w64), offsets), cout, out)
    # and by differences: y is linear in a row's value, so a step of 1 in one of them gives its gradient
    at_step = [(0, 0), (39, cin - 1), (200, cin // 2)]
    xq = torch.zeros(rows, cin, device="cuda")
    for s, c in at_step:
        xq[s, c] = 1
    xs = torch.ones(rows, -(-cin // 128), device="cuda")
    step = f64(ro.rowops_expert_matmul_fp8(xq.to(torch.float8_e4m3fn), xs, wq, ws, at, dtype=torch.float32))
    for s, c in at_step:
        terms = dy64[s] * step[s]
        # one product each way, a sum of cout of them, and the rounding of dx (2^-8 of bf16)
        assert abs(terms.sum() - f64(dx)[s, c]) <= 2.0 ** -8 * abs(terms.sum()) + (cout + 8) * 2.0 ** -22 * abs(terms).sum()
