"""Dropout of matrices that are large enough for its other kernels and loops: four blocks a
thread, and rows past one turn of the grid.  Bounds as test_gpu_dropout derives them."""
import numpy as np
import pytest
import torch

import branch_ref
from test_gpu_dropout import check, placed, rng_of
from test_gpu_expert_matmul import TYPES, f64

pytestmark = pytest.mark.gpu


def rows_of_four(cols):
    """Rows for 16-bit matrices to be taken four blocks of 8 a thread, the last thread blocks in part."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = 2048 * sms // (cols // 8) + 5
    while rows * (cols // 8) % 1024 in (0, 256, 512, 768):
        rows += 1
    return rows


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f16", "f16"), ("f16", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("cols", [1000, 8])
def test_four_blocks_a_thread(ro, cols, types):
    """Every value, with a residual and without."""
    shape = (rows_of_four(cols), cols)
    g = np.random.default_rng(cols)
    a, b = types
    key, p = (11, -12), 0.3
    x = placed(1 + g.random(shape), TYPES[a], 0)
    r = placed(g.normal(size=shape), TYPES[b], 0)
    keep = branch_ref.kept(key, *shape, p)
    for residual in (r, None):
        y = ro.rowops_dropout(x, rng_of(*key), p, residual=residual, dtype=TYPES[b])
        check(y, f64(x), np.zeros(shape) if residual is None else f64(r), keep, p, b)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_four_blocks_a_thread_in_place(ro, dtype):
    """Onto the residual and onto x, as into a matrix of its own; parts that are whole rows give the same values."""
    cols = 1000
    rows = rows_of_four(cols)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(rows, cols, generator=g, device="cuda").to(TYPES[dtype]) for _ in range(2))
    rng = rng_of(21, 22)
    want = ro.rowops_dropout(x, rng, 0.4, residual=r)
    few = ro.rowops_dropout(x[:rows // 2], rng, 0.4, residual=r[:rows // 2])  # one block a thread
    assert torch.equal(want[:rows // 2], few)
    y = r.clone()
    assert torch.equal(ro.rowops_dropout(x, rng, 0.4, residual=y, y=y), want)
    y = x.clone()
    assert torch.equal(ro.rowops_dropout(y, rng, 0.4, residual=r, y=y), want)


def test_rows_past_one_turn_of_the_grid(ro):
    """More short odd rows than 2^20 thread blocks take at once: rows of both turns, place by place."""
    turn = 2 ** 20 * 32
    rows, cols, key, p = turn + 4099, 3, (5, 2 ** 40), 0.5
    x = torch.ones(rows, cols, dtype=torch.float16, device="cuda")
    y = ro.rowops_dropout(x, rng_of(*key), p, y=x)
    probe = np.unique(np.concatenate([np.arange(3000), turn + np.arange(-3000, 4099), np.linspace(0, rows - 1, 5000).astype(np.int64)]))
    j = probe.astype(np.uint64)
    counter = np.stack([j & np.uint64(0xFFFFFFFF), j >> np.uint64(32), np.full_like(j, key[1] % 2 ** 32), np.full_like(j, key[1] >> 32)], 1)
    words = branch_ref.philox((key[0], 0), counter)
    halves = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], 2).reshape(len(probe), 8)[:, :cols]
    got = f64(y[torch.from_numpy(probe).cuda()])
    assert (got == np.where(halves >= branch_ref.threshold(p), 2.0, 0.0)).all()
    assert ((y == 0) | (y == 2)).all()
