"""Measured cases of the mixture-of-experts operators that follow the router.

The router (masked softmax, top-k) says which experts a token goes to.  What a
layer does next, and what is measured here:

* ``plan``     the (token, choice) pairs grouped by expert, stably;
* ``gather``   the tokens' rows in the plan's order, and its gradient;
* ``combine``  the experts' rows added up per token with the router's weights,
               and the gradients of the rows and of the weights;
* ``matmul``   the matrix product of each expert's rows with its weights, and
               the gradients of the rows and of the weights;
* ``fp8``      that product in e4m3 with one scale for each block of 128, rows
               quantised within the pass (dense where there is one expert).

``run`` computes an operator in plain torch where ``own`` is false and through
the library's entry points where it is true.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of a batch of 32: what a plan costs when it is all latency
        {"name": "plan decode", "kind": "plan", "tokens": 32, "experts": 64, "k": 2, "blocked": 0.0},
        # the benchmark's router workload: 262144 rows of 64 experts, 1% of them fully masked
        {"name": "plan training", "kind": "plan", "tokens": 262144, "experts": 64, "k": 2, "blocked": 0.01},
        # a decoding step's rows, fp16 activations
        {"name": "gather decode", "kind": "gather", "tokens": 32, "experts": 64, "k": 2, "cols": 768, "dtype": "f16",
         "grad": False},
        # a training step: fp32 activations to the products' bf16, and the gradient back to fp32
        {"name": "gather training", "kind": "gather", "tokens": 16384, "experts": 64, "k": 2, "cols": 768,
         "dtype": "bf16", "grad": True},
        # one prompt's tokens back from their experts, a row length that is not a multiple of four
        {"name": "combine odd prompt", "kind": "combine", "tokens": 509, "experts": 16, "k": 4, "cols": 1023,
         "dtype": "f16", "grad": False},
        # a training step with both gradients
        {"name": "combine training", "kind": "combine", "tokens": 16384, "experts": 64, "k": 2, "cols": 768,
         "dtype": "bf16", "grad": True},
        # a decoding step of a batch of 16: reads the weights of the experts that are hit
        {"name": "matmul decode", "kind": "matmul", "slots": 32, "experts": 64, "in": 768, "out": 2048,
         "dtype": "bf16", "skew": 0.0, "grad": False},
        # a prompt batch of 4096 tokens, two experts each, uneven experts
        {"name": "matmul prompt", "kind": "matmul", "slots": 8192, "experts": 64, "in": 768, "out": 2048,
         "dtype": "f16", "skew": 0.7, "grad": False},
        # rows that no 16-byte copy can follow, forward and both gradients
        {"name": "matmul odd training", "kind": "matmul", "slots": 1021, "experts": 5, "in": 773, "out": 517,
         "dtype": "f16", "skew": 0.5, "grad": True},
        # a training step's product and both gradients, wide experts
        {"name": "matmul training", "kind": "matmul", "slots": 32768, "experts": 16, "in": 2048, "out": 4096,
         "dtype": "bf16", "skew": 0.3, "grad": True},
        # a prompt batch through 8-bit experts whose weights were quantised at load
        {"name": "fp8 prompt", "kind": "fp8", "slots": 8192, "experts": 64, "in": 768, "out": 2048, "dtype": "bf16",
         "skew": 0.7, "requantize": False},
        # a dense 8-bit layer of a training step: the weights changed, so they are quantised again
        {"name": "fp8 dense training", "kind": "fp8", "slots": 16384, "experts": 1, "in": 4096, "out": 4096,
         "dtype": "bf16", "skew": 0.0, "requantize": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row length: three in four a multiple of 16, as layers have them; else any."""
    n = _log(rng, lo, hi)
    return max(16, n // 16 * 16) if rng.random() < 0.75 else n


def draw(rng):
    kind = rng.choice(["plan", "gather", "combine", "matmul", "matmul", "fp8"])
    if kind == "plan":
        experts = _log(rng, 2, 256)
        k = rng.randint(1, min(8, experts))
        return {"kind": kind, "tokens": _log(rng, 1, 524288 // k), "experts": experts, "k": k,
                "blocked": rng.choice([0.0, 0.01, 0.2])}
    if kind in ("gather", "combine"):
        experts = _log(rng, 4, 128)
        k, cols = rng.randint(1, 4), _width(rng, 32, 4096)
        return {"kind": kind, "tokens": _log(rng, 1, 16384 * 2 * 768 // (k * cols)), "experts": experts, "k": k,
                "cols": cols, "dtype": rng.choice(["bf16", "f16"]), "grad": rng.random() < 0.5}
    experts = _log(rng, 1, 128)
    wide, deep = _width(rng, 64, 4096), _width(rng, 64, 4096)
    while experts * wide * deep > 16 * 2048 * 4096:
        experts = (experts + 1) // 2
    case = {"kind": kind, "slots": _log(rng, 1, 32768), "experts": experts, "in": deep, "out": wide,
            "dtype": rng.choice(["bf16", "f16"]), "skew": round(rng.uniform(0.0, 1.0), 2)}
    if kind == "matmul":
        return {**case, "grad": rng.random() < 0.4}
    return {**case, "slots": min(case["slots"], 16384), "requantize": rng.random() < 0.3}


# ------------------------------------------------------------------ the inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _route(g, tokens, experts, k):
    """indices (tokens, k) of distinct experts in falling probability, and the probabilities, as a router gives them."""
    p = torch.softmax(torch.randn(tokens, experts, generator=g, device="cuda"), 1)
    values, indices = torch.topk(p, k, dim=1)
    return indices.float(), values


def _order(indices, values, experts):
    """(offsets, order, slot) of a plan, for the cases that begin with one."""
    pairs = indices.numel()
    e = indices.reshape(-1)
    there = (e >= 0) & (e < experts) & (values.reshape(-1) != 0)
    key = torch.where(there, e, torch.full_like(e, experts)).to(torch.int32)
    by_expert, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(by_expert, torch.arange(experts + 1, device=e.device, dtype=torch.int32))
    count = offsets[-1]
    at = torch.arange(pairs, device=e.device)
    slot = torch.empty_like(order)
    slot[order] = at
    slot = torch.where(there, slot, torch.full_like(slot, -1))
    order = torch.where(at < count, order, torch.full_like(order, -1))
    return offsets.to(torch.int32), order.to(torch.int32), slot.to(torch.int32).reshape(indices.shape)


def _groups(g, slots, experts, skew):
    """offsets (experts + 1) of `slots` rows; skew 0: experts alike, 1: shares as 1/rank, in random order."""
    share = (1.0 + torch.randperm(experts, generator=g, device="cuda").double()) ** -skew
    hit = torch.multinomial(share, slots, replacement=True, generator=g)
    counts = torch.bincount(hit, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    return offsets, int(counts.max())


def prepare(case, seed):
    g = _generator(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case)
    kind = case["kind"]
    if kind == "plan":
        s["indices"], s["values"] = _route(g, case["tokens"], case["experts"], case["k"])
        if case["blocked"]:  # rows whose mask leaves nothing: probabilities 0, first columns
            row = torch.rand(case["tokens"], generator=g, device="cuda") < case["blocked"]
            s["values"][row] = 0.0
            s["indices"][row] = torch.arange(case["k"], device="cuda").float()
        return s
    if kind in ("gather", "combine"):
        experts = max(case["experts"], case["k"])
        dtype = TYPES[case["dtype"]]
        indices, values = _route(g, case["tokens"], experts, case["k"])
        values[torch.rand(case["tokens"], generator=g, device="cuda") < 0.01] = 0.0  # masked tokens
        s["offsets"], s["order"], s["slot"] = _order(indices, values, experts)
        s["weights"] = values.contiguous()
        pairs, cols = case["tokens"] * case["k"], case["cols"]
        s["x"] = normal(case["tokens"], cols)
        s["y"] = normal(pairs, cols, dtype=dtype)
        s["dout"] = normal(case["tokens"], cols)
        s["rows"] = torch.zeros(pairs, cols, dtype=dtype, device="cuda")  # rows past the last pair stay
        return s
    s["offsets"], s["most"] = _groups(g, case["slots"], case["experts"], case["skew"])
    e, n, k, dtype = case["experts"], case["out"], case["in"], TYPES[case["dtype"]]
    s["x"] = normal(case["slots"], k, dtype=dtype)
    s["w"] = normal(e, n, k, std=k ** -0.5, dtype=dtype)
    if kind == "matmul":
        s["dy"] = normal(case["slots"], n, dtype=dtype)
    elif not case["requantize"]:
        q, scale = _quantize(s["w"], 128)
        s["wq"], s["ws"] = q.to(torch.float8_e4m3fn), scale
    return s


# --------------------------------------------------------------- the plain forms

def _quantize(x, block_rows):
    """e4m3 values of x (as fp32) and a scale for each block of block_rows x 128; the last dimension is the columns."""
    rows, cols = x.shape[-2:]
    br, bc = -(-rows // block_rows), -(-cols // 128)
    full = torch.nn.functional.pad(x.float(), (0, bc * 128 - cols, 0, br * block_rows - rows))
    blocks = full.reshape(*x.shape[:-2], br, block_rows, bc, 128)
    most = blocks.abs().amax(dim=(-3, -1), keepdim=True).clamp(min=2.0 ** -100)
    q = (blocks * 448.0 / most).to(torch.float8_e4m3fn).float()
    q = q.reshape(full.shape)[..., :rows, :cols]
    return q.contiguous(), (most / 448.0).reshape(*x.shape[:-2], br, bc)


def _spread(scale, block_rows, rows, cols):
    """The scale of each element."""
    s = scale.repeat_interleave(block_rows, dim=-2)[..., :rows, :]
    return s.repeat_interleave(128, dim=-1)[..., :cols]


def _pad(x, offsets, most):
    """(experts, most, cols): each expert's rows, then zeros."""
    at = offsets[:-1, None] + torch.arange(most, device=x.device)
    there = at < offsets[1:, None]
    return torch.where(there[..., None], x[at.clamp(max=x.shape[0] - 1)].float(), 0.0)


def _unpad(y, offsets, slots):
    at = torch.arange(slots, device=y.device)
    e = torch.searchsorted(offsets[1:].long(), at, right=True)
    return y[e, at - offsets[e]]


def _plain(s):
    kind = s["kind"]
    if kind == "plan":
        return _order(s["indices"], s["values"], s["experts"])
    if kind == "gather":
        token = s["order"].clamp(min=0).long() // s["k"]
        rows = torch.where(s["order"][:, None] >= 0, s["x"][token].to(s["rows"].dtype), s["rows"])
        if not s["grad"]:
            return rows
        there = s["slot"][..., None] >= 0
        return rows, torch.where(there, s["y"][s["slot"].clamp(min=0).long()].float(), 0.0).sum(1)
    if kind == "combine":
        there = s["slot"][..., None] >= 0
        rows = torch.where(there, s["y"][s["slot"].clamp(min=0).long()].float(), 0.0)
        out = (rows * s["weights"][..., None]).sum(1)
        if not s["grad"]:
            return out
        pair = s["order"].clamp(min=0).long()
        dy = s["weights"].reshape(-1)[pair][:, None] * s["dout"][pair // s["k"]]
        dy = torch.where(s["order"][:, None] >= 0, dy.to(s["rows"].dtype), s["rows"])
        return out, dy, (rows * s["dout"][:, None, :]).sum(2)
    offsets, slots, most = s["offsets"], s["slots"], s["most"]
    if kind == "fp8":
        q, scale = _quantize(s["x"], 1)
        x = q * _spread(scale, 1, slots, s["in"])
        if s["requantize"]:
            q, scale = _quantize(s["w"], 128)
        else:
            q, scale = s["wq"].float(), s["ws"]
        w = q * _spread(scale, 128, s["out"], s["in"])
        y = torch.bmm(_pad(x, offsets, most), w.transpose(1, 2))
        return _unpad(y, offsets, slots).to(s["x"].dtype)
    x, w = _pad(s["x"], offsets, most), s["w"].float()
    y = _unpad(torch.bmm(x, w.transpose(1, 2)), offsets, slots).to(s["x"].dtype)
    if not s["grad"]:
        return y
    dy = _pad(s["dy"], offsets, most)
    dx = _unpad(torch.bmm(dy, w), offsets, slots).to(s["x"].dtype)
    return y, dx, torch.bmm(dy.transpose(1, 2), x).to(s["w"].dtype)


# ---------------------------------------------------------- the library's calls

def _calls(s):
    import row_wise_softmax_warp_gb300 as ro

    kind = s["kind"]
    if kind == "plan":
        return ro.rowops_expert_plan(s["indices"], s["experts"], values=s["values"])
    if kind == "gather":
        rows = ro.rowops_expert_gather(s["x"], s["slot"], out=s["rows"])
        if not s["grad"]:
            return rows
        return rows, ro.rowops_expert_combine(s["y"], s["slot"], dtype=torch.float32)
    if kind == "combine":
        out = ro.rowops_expert_combine(s["y"], s["slot"], weights=s["weights"], dtype=torch.float32)
        if not s["grad"]:
            return out
        dy, dweights = ro.rowops_expert_combine_bwd(s["dout"], s["y"], s["slot"], s["weights"], dy=s["rows"])
        return out, dy, dweights
    if kind == "fp8":
        xq, xs = ro.rowops_quantize_blocks(s["x"])
        wq, ws = ro.rowops_quantize_blocks(s["w"], block_rows=128) if s["requantize"] else (s["wq"], s["ws"])
        return ro.rowops_expert_matmul_fp8(xq, xs, wq, ws, s["offsets"], dtype=s["x"].dtype)
    y = ro.rowops_expert_matmul(s["x"], s["w"], s["offsets"])
    if not s["grad"]:
        return y
    dx = ro.rowops_expert_matmul(s["dy"], s["w"], s["offsets"], transposed=True)
    return y, dx, ro.rowops_expert_matmul_wgrad(s["dy"], s["x"], s["offsets"])


def run(state):
    return _calls(state) if own else _plain(state)


# ----------------------------------------------------------- work and exact results

def work(case):
    kind = case["kind"]
    if kind == "plan":
        pairs = case["tokens"] * case["k"]
        return {"bytes": pairs * 16 + 4 * (case["experts"] + 1), "flops": 0}
    if kind in ("gather", "combine"):
        t, k, c, b = case["tokens"], case["k"], case["cols"], BYTES[case["dtype"]]
        one = t * c * 4 + t * k * c * b + t * k * 4  # fp32 rows once, expert rows once, the plan
        if kind == "gather":
            return {"bytes": one * (2 if case["grad"] else 1), "flops": t * k * c if case["grad"] else 0}
        if not case["grad"]:
            return {"bytes": one + t * k * 4, "flops": 2 * t * k * c}
        return {"bytes": 2 * one + t * k * c * b + 3 * t * k * 4, "flops": 5 * t * k * c}
    m, e, n, k, b = case["slots"], case["experts"], case["out"], case["in"], BYTES[case["dtype"]]
    hit = e * (1.0 - (1.0 - 1.0 / e) ** m) if e > 1 else 1.0  # experts that get a row, where they are alike
    if kind == "matmul":
        one = m * (k + n) * b + 4 * (e + 1)
        if not case["grad"]:
            return {"bytes": one + hit * n * k * b, "flops": 2.0 * m * n * k}
        return {"bytes": 2 * one + (hit + e) * n * k * b, "flops": 6.0 * m * n * k}
    weights = hit * n * k * (b if case["requantize"] else 1)
    return {"bytes": m * (k + n) * b + weights + 4 * (e + 1), "flops": 2.0 * m * n * k}


def _e4m3(v):
    """The nearest e4m3 value of v (fp64, magnitude at most 448), ties to even."""
    exponent = torch.frexp(v.abs().clamp(min=2.0 ** -6))[1].double() - 1
    step = torch.exp2(exponent - 3)
    return torch.round(v / step) * step


def _quantize64(x, block_rows):
    """What the quantised x stands for, block by block."""
    out = torch.empty_like(x, dtype=torch.float64)
    step = block_rows if block_rows > 1 else x.shape[-2]
    across = (-2, -1) if block_rows > 1 else -1
    for r in range(0, x.shape[-2], step):
        for c in range(0, x.shape[-1], 128):
            block = x[..., r:r + step, c:c + 128].double()
            most = block.abs().amax(dim=across, keepdim=True).clamp(min=2.0 ** -100)
            out[..., r:r + step, c:c + 128] = _e4m3(block * 448.0 / most) * (most / 448.0)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "plan":
        return None
    if kind in ("gather", "combine"):
        t, k, c = case["tokens"], case["k"], case["cols"]
        slot = s["slot"].long()
        w = s["weights"].double() if kind == "combine" else torch.ones(t, k, dtype=torch.float64, device="cuda")
        total = torch.zeros(t, c, dtype=torch.float64, device="cuda")
        rows = torch.zeros(t * k, c, dtype=torch.float64, device="cuda")
        dw = torch.zeros(t, k, dtype=torch.float64, device="cuda")
        source = s["dout"] if kind == "combine" else s["x"]
        for j in range(k):
            token = torch.nonzero(slot[:, j] >= 0)[:, 0]
            at = slot[token, j]
            y = s["y"][at].double()
            total[token] += w[token, j, None] * y
            rows[at] = w[token, j, None] * source[token].double()
            dw[token, j] = (y * s["dout"][token].double()).sum(1)
        if kind == "gather":
            return (rows, total) if case["grad"] else rows
        return (total, rows, dw) if case["grad"] else total
    if case["slots"] * case["in"] * case["out"] * (6.0 if case.get("grad") else 2.0) > 5e12:
        return None
    bounds = s["offsets"].tolist()
    if kind == "fp8":
        x = _quantize64(s["x"], 1)
        if case["requantize"]:
            w = _quantize64(s["w"], 128)
        else:
            w = s["wq"].double() * _spread(s["ws"].double(), 128, case["out"], case["in"])
    else:
        x, w = s["x"].double(), s["w"].double()
    y = torch.zeros(case["slots"], case["out"], dtype=torch.float64, device="cuda")
    grad = case.get("grad", False)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    for e in range(case["experts"]):
        a, b = bounds[e], bounds[e + 1]
        y[a:b] = x[a:b] @ w[e].T
        if grad:
            dy = s["dy"][a:b].double()
            dx[a:b] = dy @ w[e]
            dw[e] = dy.T @ x[a:b]
    return (y, dx, dw) if grad else y
