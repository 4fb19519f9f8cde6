"""Slots that are named more than once: what is read is added up, what is written is
one of the rows' values, and nothing else changes."""
import numpy as np
import pytest
import torch

import expert_ref

pytestmark = pytest.mark.gpu

SLOTS = 9


def inputs(tokens, k, cols, seed):
    rng = np.random.default_rng(seed)
    slot = rng.integers(0, SLOTS - 2, (tokens, k)).astype(np.int32)  # the last two slots are never named
    slot[rng.random((tokens, k)) < 0.2] = -1
    x = rng.integers(-100, 101, (tokens, cols)).astype(np.float32)
    return slot, x, rng


def one_of(got, named, values, rest):
    """Each value of a row is that of one of the pairs that name it; the others are `rest`."""
    for s in range(SLOTS):
        if named[s]:
            assert (got[s][None] == np.stack([values(p) for p in named[s]])).any(0).all(), s
        else:
            assert (got[s] == rest).all(), s


@pytest.mark.parametrize("tokens,k,cols", [(2, 1, 5), (40, 2, 64), (300, 3, 1000), (50, 2, 5003)])
def test_named_twice(ro, tokens, k, cols):
    slot, x, rng = inputs(tokens, k, cols, cols)
    at, cuda = torch.from_numpy(slot).cuda(), lambda a: torch.from_numpy(a).cuda()
    named = [[(t, j) for t in range(tokens) for j in range(k) if slot[t, j] == s] for s in range(SLOTS)]
    for dtype in (torch.float32, torch.float16):
        out = ro.rowops_expert_gather(cuda(x), at, out=torch.full((SLOTS, cols), 7.5, dtype=dtype, device="cuda"))
        one_of(out.double().cpu().numpy(), named, lambda p: x[p[0]], 7.5)
    y = rng.integers(-8, 9, (SLOTS, cols)).astype(np.float32)
    w = rng.integers(-3, 4, (tokens, k)).astype(np.float32)
    got = ro.rowops_expert_combine(cuda(y), at, weights=cuda(w))
    assert (got.double().cpu().numpy() == expert_ref.combine(y.astype(np.float64), slot, w)).all()
    dy, dw = ro.rowops_expert_combine_bwd(cuda(x), cuda(y), at, cuda(w),
                                          dy=torch.full((SLOTS, cols), 7.5, device="cuda"))
    one_of(dy.double().cpu().numpy(), named, lambda p: w[p] * x[p[0]], 7.5)
    _, want = expert_ref.combine_bwd(x.astype(np.float64), y.astype(np.float64), slot, w, np.zeros((SLOTS, cols)))
    assert (dw.double().cpu().numpy() == want).all()  # sums below 2^24: exact
