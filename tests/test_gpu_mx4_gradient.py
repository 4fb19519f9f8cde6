"""The rows' gradient of the 4-bit product by the call that the header names: the product
of dy, quantised by rows, with the weights transposed within each expert and quantised from
their own values.  Bounds as test_gpu_mx4 derives them."""
import numpy as np
import pytest
import torch

from test_gpu_expert_matmul import TYPES, f64, offsets_of
from test_gpu_mx4 import check, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("widths", [(256, 128), (768, 256), (144, 520), (50, 34), (33, 50), (130, 33), (257, 515), (7, 1)])
def test_gradient_of_the_rows(ro, widths, out):
    cin, cout = widths
    sizes, g = [40, 0, 300, 1], np.random.default_rng(cin)
    offsets, rows = offsets_of(sizes), sum(sizes)
    at = torch.from_numpy(offsets).cuda()
    w = torch.from_numpy(g.normal(size=(len(sizes), cout, cin)) * np.exp2(g.integers(-3, 4, (4, 1, 1)))).cuda().bfloat16()
    dy = torch.from_numpy(g.normal(size=(rows + 2, cout))).cuda().bfloat16()
    dq, ds = ro.rowops_quantize_mx4(dy)
    wq, ws = ro.rowops_quantize_mx4(w.transpose(1, 2).contiguous())  # (experts, in, out), blocks along out
    assert dq.shape == (rows + 2, (cout + 1) // 2) and wq.shape == (len(sizes), cin, (cout + 1) // 2)
    dx = torch.full((rows + 2, cin), 5.0, dtype=TYPES[out], device="cuda")
    ro.rowops_expert_matmul_mx4(dq, ds, wq, ws, at, y=dx)
    assert (dx[rows:] == 5).all()  # rows behind the last group
    dy64, w64 = values(dq, ds, cout), values(wq, ws, cout)
    check(dx[:rows], dy64[:rows], w64, offsets, out)
    # and by differences: y is linear in a row's value, so a step of 1 in one of them gives
    # its gradient; the quantised weights are bf16 numbers, and a product with one 1 is one of them
    steps = [(0, 0), (39, cin - 1), (200, cin // 2), (340, 0)]
    x = torch.zeros(rows, cin, dtype=torch.bfloat16, device="cuda")
    for s, c in steps:
        x[s, c] = 1
    forward = torch.from_numpy(np.ascontiguousarray(w64.transpose(0, 2, 1))).cuda().bfloat16()
    assert (f64(forward) == w64.transpose(0, 2, 1)).all()
    step = f64(ro.rowops_expert_matmul(x, forward, at))
    for s, c in steps:
        terms = dy64[s] * step[s]
        # a sum of cout products, and the rounding of dx (2^-8 of bf16)
        assert abs(terms.sum() - f64(dx)[s, c]) <= 2.0 ** -8 * abs(terms.sum()) + (cout + 8) * 2.0 ** -22 * abs(terms).sum()
    assert ro.library().rowops_pipeline_timeouts() == 0
