"""Plan, gather, combine and its backward against plain 64-bit forms.

Bounds: a result rounded to type t is off by at most u_t |value| (half a step:
2^-24, 2^-11, 2^-8; plus half the smallest subnormal), and an fp32 sum of n terms
by at most n 2^-24 sum |terms|, fused multiply-adds rounding once a term."""
import numpy as np
import pytest
import torch

import expert_ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}


def cuda(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype) if dtype else \
        torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def odd(t):
    """The same values one element past a 16-byte boundary."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    buf[1:] = t.reshape(-1)
    return buf[1:].view(t.shape)


def routing(rng, tokens, experts, k, blocked=0.2):
    """Distinct experts per token, and weights of which some are 0 or a whole row is."""
    indices = np.argsort(rng.random((tokens, experts)), axis=1)[:, :k].astype(np.float32)
    values = rng.random((tokens, k)).astype(np.float32) + 0.01
    values[rng.random(tokens) < blocked] = 0.0
    values[rng.random((tokens, k)) < 0.05] = 0.0
    return indices, values


@pytest.mark.parametrize("tokens,experts,k", [
    (1, 1, 1), (1, 64, 2), (32, 64, 2), (33, 7, 7), (509, 16, 4), (1024, 64, 2), (1025, 64, 2), (2049, 64, 2), (4097, 1, 1),
    (5000, 1024, 3), (70001, 5, 1), (20000, 256, 8)])
def test_plan(ro, tokens, experts, k):
    rng = np.random.default_rng(tokens + experts)
    indices, values = routing(rng, tokens, experts, k)
    for v in (values, None):
        got = ro.rowops_expert_plan(cuda(indices), experts, values=None if v is None else cuda(v))
        for name, a, b in zip(("offsets", "order", "slot"), got, expert_ref.plan(indices, v, experts)):
            assert (a.cpu().numpy() == b).all(), name


def test_plan_odd_indices(ro):
    """Indices that name no expert, and zero and NaN values."""
    nan, inf = np.nan, np.inf
    indices = np.array([[0, 3], [-1, 2.75], [4, 1e9], [nan, inf], [-inf, -0.0], [3, 1], [2, -0.5]], np.float32)
    values = np.array([[1, nan], [1, 1], [1, 1], [1, 1], [1, -1], [-0.0, 1e-45], [inf, 1]], np.float32)
    got = ro.rowops_expert_plan(cuda(indices), 4, values=cuda(values))
    for a, b in zip(got, expert_ref.plan(indices, values, 4)):
        assert (a.cpu().numpy() == b).all()


def test_plan_nothing(ro):
    """No rows, and rows whose mask leaves nothing."""
    offsets, order, slot = ro.rowops_expert_plan(torch.empty(0, 2, device="cuda"), 5)
    assert (offsets == 0).all() and offsets.numel() == 6 and order.numel() == 0
    for tokens in (3, 5000):
        zero = torch.zeros(tokens, 2, device="cuda")
        offsets, order, slot = ro.rowops_expert_plan(zero, 5, values=zero)
        assert (offsets == 0).all() and (order == -1).all() and (slot == -1).all()


def test_plan_of_the_router(ro):
    """top_k_rows of a masked softmax: masked experts, and rows with none, lose their pairs."""
    rng = np.random.default_rng(3)
    x = rng.normal(size=(700, 16)).astype(np.float32)
    mask = (rng.random((700, 16)) < 0.3).astype(np.uint8)
    mask[::50] = 0
    mask[1::50] = 0
    mask[1::50, 5] = 1
    p, kept = ro.rowops_router_masked_topk(cuda(x), cuda(mask), 2)
    values, indices = ro.rowops_top_k_rows(p, 2)
    offsets, order, slot = ro.rowops_expert_plan(indices, 16, values=values)
    ref = expert_ref.plan(indices.cpu().numpy(), values.cpu().numpy(), 16)
    for a, b in zip((offsets, order, slot), ref):
        assert (a.cpu().numpy() == b).all()
    counts = np.diff(offsets.cpu().numpy())
    assert (counts == (kept.cpu().numpy() * (p.cpu().numpy() > 0)).sum(0)).all()
    assert (slot[::50] == -1).all() and ((slot[1::50] >= 0).sum(1) == 1).all()


SHAPES = [(1, 1, 1), (1, 2, 768), (5, 3, 7), (33, 2, 1023), (64, 1, 64), (40, 4, 520), (3, 2, 5003), (300, 2, 256)]
PAIRS = [("f32", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32"), ("bf16", "f16")]


def slots_of(rng, tokens, k, extra):
    """slot (tokens, k): distinct rows of tokens * k + extra, some left out, one far out of range."""
    slots = tokens * k + extra
    slot = rng.permutation(slots)[:tokens * k].reshape(tokens, k).astype(np.int32)
    slot[rng.random((tokens, k)) < 0.15] = -1
    if tokens > 2:
        slot[0, 0], slot[1, 0], slot[2] = 2 ** 31 - 1, slots, -5
    return slot, slots


@pytest.mark.parametrize("types", PAIRS)
@pytest.mark.parametrize("tokens,k,cols", SHAPES)
def test_gather(ro, tokens, k, cols, types):
    rng = np.random.default_rng(cols)
    slot, slots = slots_of(rng, tokens, k, 4)
    tx, to = types
    x = cuda(rng.normal(size=(tokens, cols)), TYPES[tx])
    for shift in (lambda t: t, odd):
        out = shift(torch.full((slots, cols), 7.0, dtype=TYPES[to], device="cuda"))
        want = out.clone()
        for t in range(tokens):
            for s in slot[t]:
                if 0 <= s < slots:
                    want[s] = x[t].to(TYPES[to])
        got = ro.rowops_expert_gather(shift(x), cuda(slot), out=out)
        assert got is out and torch.equal(got, want)  # rows that no slot names are as they were


@pytest.mark.parametrize("types", PAIRS)
@pytest.mark.parametrize("tokens,k,cols", SHAPES)
def test_combine(ro, tokens, k, cols, types):
    rng = np.random.default_rng(cols + 1)
    slot, slots = slots_of(rng, tokens, k, 4)
    ty, to = types
    y = cuda(rng.normal(size=(slots, cols)), TYPES[ty])
    weights = rng.normal(size=(tokens, k)).astype(np.float32)
    for w in (weights, None):
        for shift in (lambda t: t, odd):
            got = ro.rowops_expert_combine(shift(y), cuda(slot), weights=None if w is None else cuda(w),
                                           dtype=TYPES[to])
            want = expert_ref.combine(f64(y), slot, w)
            size = expert_ref.combine_magnitude(f64(y), slot, w)
            bound = UNIT[to] * np.abs(want) + (1 + UNIT[to]) * k * 2.0 ** -24 * size + TINY[to]
            assert (np.abs(f64(got) - want) <= bound).all()
            none = ~((slot >= 0) & (slot < slots)).any(1)
            assert (f64(got)[none] == 0).all() and not np.signbit(f64(got)[none]).any()


@pytest.mark.parametrize("types", PAIRS)
@pytest.mark.parametrize("tokens,k,cols", SHAPES + [(1500, 2, 96)])
def test_combine_bwd(ro, tokens, k, cols, types):
    rng = np.random.default_rng(cols + 2)
    slot, slots = slots_of(rng, tokens, k, 4)
    to, ty = types
    y = cuda(rng.normal(size=(slots, cols)), TYPES[ty])
    dout = cuda(rng.normal(size=(tokens, cols)), TYPES[to])
    weights = rng.normal(size=(tokens, k)).astype(np.float32)
    for shift in (lambda t: t, odd):
        dy = shift(torch.full((slots, cols), 3.0, dtype=TYPES[ty], device="cuda"))
        got, dw = ro.rowops_expert_combine_bwd(shift(dout), shift(y), cuda(slot), cuda(weights), dy=dy)
        want, want_dw = expert_ref.combine_bwd(f64(dout), f64(y), slot, weights, np.full((slots, cols), 3.0))
        bound = UNIT[ty] * np.abs(want) + 2.0 ** -24 * np.abs(want) * 1.01 + TINY[ty]
        assert (np.abs(f64(got) - want) <= bound).all()
        _, size = expert_ref.combine_bwd(np.abs(f64(dout)), np.abs(f64(y)), slot, weights, np.zeros((slots, cols)))
        assert (np.abs(f64(dw) - want_dw) <= (cols + 8) * 2.0 ** -24 * size).all()
        gone = ~((slot >= 0) & (slot < slots))
        assert (f64(dw)[gone] == 0).all()


def test_combine_gradient_by_differences(ro):
    """combine is linear in y and in the weights, so differences with steps of powers of two are exact up to rounding."""
    rng = np.random.default_rng(9)
    tokens, k, cols = 6, 2, 40
    slot = rng.permutation(tokens * k).reshape(tokens, k).astype(np.int32)
    y, w = rng.normal(size=(tokens * k, cols)).astype(np.float32), rng.normal(size=(tokens, k)).astype(np.float32)
    dout = rng.normal(size=(tokens, cols)).astype(np.float32)

    def loss(y, w):
        out = ro.rowops_expert_combine(cuda(y), cuda(slot), weights=cuda(w))
        return (f64(out) * dout).sum()

    dy, dw = ro.rowops_expert_combine_bwd(cuda(dout), cuda(y), cuda(slot), cuda(w))
    for t, j, c in ((0, 0, 3), (3, 1, 39), (5, 0, 0)):
        # an output is off by at most 3 * 2^-24 * (|w||y| sums < 40); cols of them, over the step of 8
        slack = 2 * 3 * 2.0 ** -24 * 80 * np.abs(dout).sum() / 8
        y2, w2 = y.copy(), w.copy()
        y2[slot[t, j], c] += 8
        w2[t, j] += 8
        assert abs((loss(y2, w) - loss(y, w)) / (float(y2[slot[t, j], c]) - float(y[slot[t, j], c]))
                   - f64(dy)[slot[t, j], c]) < slack
        assert abs((loss(y, w2) - loss(y, w)) / (float(w2[t, j]) - float(w[t, j])) - f64(dw)[t, j]) < slack


def test_gather_gradient_is_combine(ro):
    """<gather(x), d> == <x, combine(d)> exactly for whole numbers."""
    rng = np.random.default_rng(11)
    slot, slots = slots_of(rng, 50, 3, 0)
    x = cuda(rng.integers(-8, 9, (50, 96)).astype(np.float32))
    d = cuda(rng.integers(-8, 9, (slots, 96)).astype(np.float32))
    rows = ro.rowops_expert_gather(x, cuda(slot), out=torch.zeros(slots, 96, device="cuda"))
    assert (rows.double() * d.double()).sum() == (x.double() * ro.rowops_expert_combine(d, cuda(slot)).double()).sum()


def test_non_finite_rows_stay_where_they_are(ro):
    x = torch.ones(4, 64, device="cuda")
    x[1], x[2, 5] = float("nan"), float("inf")
    slot = torch.tensor([[0], [1], [2], [3]], dtype=torch.int32, device="cuda")
    rows = ro.rowops_expert_gather(x, slot, dtype=torch.float16)
    assert torch.isnan(rows[1]).all() and torch.isinf(rows[2, 5]) and torch.isfinite(rows[[0, 3]]).all()
    left = torch.tensor([[0, -1], [-1, 3]], dtype=torch.int32, device="cuda")  # rows 1 and 2 are not read
    out = ro.rowops_expert_combine(rows, left, weights=torch.ones(2, 2, device="cuda"))
    assert (out == 1).all()


def test_binding_refusals(ro):
    f = torch.zeros(4, 8, device="cuda")
    slot = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        ro.rowops_expert_gather(f, slot[:3])
    with pytest.raises(ValueError):
        ro.rowops_expert_gather(f.T, torch.zeros(8, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        ro.rowops_expert_gather(f, slot.long())
    with pytest.raises(ValueError):
        ro.rowops_expert_combine(f, slot, weights=f)
    with pytest.raises(TypeError):
        ro.rowops_expert_combine(f, slot, weights=torch.zeros(4, 2, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        ro.rowops_expert_combine(f, slot, out=torch.zeros(4, 9, device="cuda"))
    with pytest.raises(ValueError):
        ro.rowops_expert_plan(f[0], 4)
    with pytest.raises(ro.RowopsError):
        ro.rowops_expert_plan(f[:, :2].contiguous(), 1025)
