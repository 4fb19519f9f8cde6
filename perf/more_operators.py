"""Measured cases of the operators between a model's layers and its 4-bit products.

What a sublayer's result goes through before the next sublayer's products, and
those products in microscaled 4 bits:

* ``dropout``  values dropped by a counter-based generator (Philox4x32-10, whose
               mask is never stored), scaled and added to a residual; the same call
               on a gradient is its backward;
* ``norm``     residual + dropout(x), and its root-mean-square norm, in the
               branch's type or in e4m3 with one scale for each 128 columns;
* ``norm_bwd`` the gradients of ``norm``;
* ``mx4``      the experts' product on e2m1 operands with one power of two for each
               block of 32 (OCP microscaling), rows quantised within the pass;
* ``layer``    ``norm`` with an answer in microscaled 4 bits and the dense product
               that takes it.

``run`` computes an operator in plain torch where ``own`` is false and through
the library's entry points where it is true.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # dropout on the benchmark's attention probabilities, 8 x 12 heads of 1024 x 1024
        {"name": "dropout attention", "kind": "dropout", "rows": 98304, "cols": 1024, "dtype": "f32", "stream": "f32",
         "residual": False, "p": 0.1, "softmax": True},
        # one odd prompt's branch added to its residual, rows that no 16-byte access can follow
        {"name": "dropout odd residual", "kind": "dropout", "rows": 509, "cols": 1023, "dtype": "f16", "stream": "f16",
         "residual": True, "p": 0.25, "softmax": False},
        # one decoding step of a batch of 32 ahead of an 8-bit product: all latency
        {"name": "norm decode e4m3", "kind": "norm", "rows": 32, "cols": 4096, "dtype": "bf16", "stream": "bf16",
         "p": 0.0, "quantize": "e4m3"},
        # an odd prompt ahead of an 8-bit product
        {"name": "norm odd e4m3", "kind": "norm", "rows": 509, "cols": 1023, "dtype": "f16", "stream": "f32",
         "p": 0.0, "quantize": "e4m3"},
        # a training step's forward pass: bf16 branch, fp32 residual stream, dropout
        {"name": "norm training", "kind": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16", "stream": "f32",
         "p": 0.1, "quantize": ""},
        # the benchmark's LayerNorm size (8 x 512 tokens of 768), fp32, no dropout
        {"name": "norm backward", "kind": "norm_bwd", "rows": 4096, "cols": 768, "dtype": "f32", "stream": "f32", "p": 0.0},
        # the backward pass of "norm training"
        {"name": "norm backward training", "kind": "norm_bwd", "rows": 16384, "cols": 4096, "dtype": "bf16",
         "stream": "f32", "p": 0.1},
        # a decoding step of a batch of 16, two experts each: reads the weights of the experts that are hit
        {"name": "mx4 decode", "kind": "mx4", "slots": 32, "experts": 64, "in": 768, "out": 2048, "dtype": "bf16",
         "skew": 0.0, "requantize": False},
        # rows of bytes that no 16-byte copy can follow, an odd number of columns
        {"name": "mx4 odd", "kind": "mx4", "slots": 1021, "experts": 5, "in": 773, "out": 517, "dtype": "f16",
         "skew": 0.5, "requantize": False},
        # a prompt batch of 4096 tokens, two experts each, uneven experts, weights quantised at load
        {"name": "mx4 prompt", "kind": "mx4", "slots": 8192, "experts": 64, "in": 768, "out": 2048, "dtype": "bf16",
         "skew": 0.7, "requantize": False},
        # a dense 4-bit layer of a training step: the weights changed, so they are quantised again
        {"name": "mx4 dense training", "kind": "mx4", "slots": 16384, "experts": 1, "in": 4096, "out": 4096,
         "dtype": "bf16", "skew": 0.0, "requantize": True},
        # a prompt batch through norm and the projection behind it
        {"name": "layer mx4 prompt", "kind": "layer", "rows": 8192, "cols": 2048, "out": 4096, "dtype": "bf16",
         "stream": "bf16", "p": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row length: three in four a multiple of 16, as layers have them; else any."""
    n = _log(rng, lo, hi)
    return max(16, n // 16 * 16) if rng.random() < 0.75 else n


def draw(rng):
    kind = rng.choice(["dropout", "norm", "norm", "norm_bwd", "mx4", "mx4", "layer"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    stream = rng.choice([dtype, "f32"])
    p = rng.choice([0.0, round(rng.uniform(0.05, 0.5), 2)])
    if kind == "dropout":
        cols = _width(rng, 32, 16384)
        return {"kind": kind, "rows": _log(rng, 1, 98304 * 1024 // (3 * cols)), "cols": cols, "dtype": dtype,
                "stream": stream, "residual": rng.random() < 0.5, "p": p or 0.1, "softmax": rng.random() < 0.3}
    if kind in ("norm", "norm_bwd"):
        cols = _width(rng, 32, 16384)
        case = {"kind": kind, "rows": _log(rng, 1, 16384 * 4096 // (2 * cols)), "cols": cols, "dtype": dtype,
                "stream": stream, "p": p}
        return case if kind == "norm_bwd" else {**case, "quantize": rng.choice(["", "e4m3"])}
    half = rng.choice(["bf16", "f16"])
    wide, deep = _width(rng, 64, 4096), _width(rng, 64, 4096)
    if kind == "layer":
        return {"kind": kind, "rows": _log(rng, 1, 8192), "cols": deep, "out": wide, "dtype": half,
                "stream": rng.choice([half, "f32"]), "p": p}
    experts = _log(rng, 1, 128)
    while experts * wide * deep > 16 * 2048 * 4096:
        experts = (experts + 1) // 2
    return {"kind": kind, "slots": _log(rng, 1, 16384), "experts": experts, "in": deep, "out": wide, "dtype": half,
            "skew": round(rng.uniform(0.0, 1.0), 2), "requantize": rng.random() < 0.3}


# ------------------------------------------------------------------ the inputs

def _groups(g, slots, experts, skew):
    """offsets (experts + 1) of `slots` rows; skew 0: experts alike, 1: shares as 1/rank, in random order."""
    share = (1.0 + torch.randperm(experts, generator=g, device="cuda").double()) ** -skew
    hit = torch.multinomial(share, slots, replacement=True, generator=g)
    counts = torch.bincount(hit, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    return offsets, int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case)
    kind, dtype = case["kind"], TYPES[case["dtype"]]
    if kind == "mx4":
        e, n, k = case["experts"], case["out"], case["in"]
        s["offsets"], s["most"] = _groups(g, case["slots"], e, case["skew"])
        s["x"] = normal(case["slots"], k, dtype=dtype)
        s["w"] = normal(e, n, k, std=k ** -0.5, dtype=dtype)
        if not case["requantize"]:
            s["wq"], s["ws"] = _pack_mx4(*_quantize_mx4(s["w"]))
        return s
    rows, cols = case["rows"], case["cols"]
    stream = TYPES[case["stream"]]
    # seed and offset of the generator, as a training loop keeps them on the device
    s["rng"] = torch.randint(-2 ** 62, 2 ** 62, (2,), generator=g, device="cuda")
    if kind == "dropout":
        x = normal(rows, cols)
        s["x"] = (torch.softmax(x, 1) if case["softmax"] else x).to(dtype)
        s["residual"] = normal(rows, cols, dtype=stream) if case["residual"] else None
        return s
    s["gamma"] = 1.0 + normal(cols, std=0.1)
    size = torch.exp(normal(rows, 1, std=0.5))  # residual streams grow unevenly from token to token
    if kind == "norm_bwd":
        s["h"] = (normal(rows, cols) * size).to(stream)
        s["row_rms"] = torch.sqrt(s["h"].float().square().mean(1) + EPS)
        s["dy"] = normal(rows, cols, dtype=dtype)
        s["dh"] = normal(rows, cols, dtype=stream)
        return s
    s["x"] = normal(rows, cols, dtype=dtype)
    s["residual"] = (normal(rows, cols) * size).to(stream)
    if kind == "layer":
        w = normal(1, case["out"], cols, std=cols ** -0.5, dtype=dtype)
        s["wq"], s["ws"] = _pack_mx4(*_quantize_mx4(w))
    return s


# --------------------------------------------------------------- the plain forms

def _philox(rng, blocks):
    """(blocks, 8) random 16-bit numbers, as int64: Philox4x32-10 with the key rng[0] on the counters (block, rng[1])."""
    low = 0xFFFFFFFF
    j = torch.arange(blocks, device=rng.device)
    a, b = j & low, j >> 32
    c, d = (rng[1] & low).expand(blocks), ((rng[1] >> 32) & low).expand(blocks)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        m, n = a * 0xD2511F53, c * 0xCD9E8D57  # wraps modulo 2^64; the halves are what they should be
        a, b, c, d = ((n >> 32) & low) ^ b ^ k0, n & low, ((m >> 32) & low) ^ d ^ k1, m & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([a, b, c, d], 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).reshape(blocks, 8)


def _drop(x, rng, p):
    """x with values dropped and the others scaled, in fp32."""
    threshold = round(p * 65536)
    if threshold == 0:
        return x.float()
    rows, cols = x.shape
    per = -(-cols // 8)
    kept = (_philox(rng, rows * per) >= threshold).reshape(rows, per * 8)[:, :cols]
    return torch.where(kept, x.float() * (65536.0 / (65536 - threshold)), 0.0)


def _quantize_e4m3(y):
    """e4m3 values of y (fp32) and a scale for each 128 columns of a row."""
    rows, cols = y.shape
    blocks = -(-cols // 128)
    full = torch.nn.functional.pad(y, (0, blocks * 128 - cols)).reshape(rows, blocks, 128)
    most = full.abs().amax(dim=2, keepdim=True).clamp(min=2.0 ** -100)
    q = (full * 448.0 / most).reshape(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
    return q.contiguous(), (most / 448.0).reshape(rows, blocks)


def _power_of_two(e):
    """2^e in fp32 for -127 <= e <= 127, exactly."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantize_mx4(x):
    """e2m1 values of x (as fp32) and the exponents of the blocks of 32, from the last dimension's columns."""
    cols = x.shape[-1]
    blocks = -(-cols // 32)
    full = torch.nn.functional.pad(x.float(), (0, blocks * 32 - cols)).unflatten(-1, (blocks, 32))
    exponent = (torch.frexp(full.abs().amax(dim=-1))[1] - 3).clamp(min=-127)  # floor(log2(most)) - 2
    exponent = torch.where(full.abs().amax(dim=-1) == 0, -127, exponent)
    v = full * _power_of_two(-exponent[..., None])
    step = torch.where(v.abs() < 2.0, 0.5, torch.where(v.abs() < 4.0, 1.0, 2.0))
    q = (torch.round(v / step) * step).clamp(-6.0, 6.0)
    return q.flatten(-2)[..., :cols], exponent


def _pack_mx4(q, exponent):
    """Two e2m1 codes a byte (the lower column in the lower half), and exponents with a bias of 127."""
    m = q.abs()
    code = torch.where(m <= 2.0, m * 2.0, torch.where(m <= 4.0, m + 2.0, m / 2.0 + 4.0)).to(torch.uint8)
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    code = torch.nn.functional.pad(code, (0, q.shape[-1] % 2))
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), (exponent + 127).to(torch.uint8).contiguous()


def _unpack_mx4(packed, scale, cols):
    """What packed e2m1 codes with their scales stand for, in fp32."""
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=packed.device)
    values = torch.cat([values, -values])
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)[..., :cols]
    return values[code.long()] * _spread_mx4(scale.int() - 127, cols)


def _spread_mx4(exponent, cols):
    """The scale of each column."""
    return _power_of_two(exponent).repeat_interleave(32, dim=-1)[..., :cols]


def _pad(x, offsets, most):
    """(experts, most, cols): each expert's rows, then zeros."""
    at = offsets[:-1, None] + torch.arange(most, device=x.device)
    there = at < offsets[1:, None]
    return torch.where(there[..., None], x[at.clamp(max=x.shape[0] - 1)], 0.0)


def _unpad(y, offsets, slots):
    at = torch.arange(slots, device=y.device)
    e = torch.searchsorted(offsets[1:].long(), at, right=True)
    return y[e, at - offsets[e]]


def _plain(s):
    kind, dtype = s["kind"], TYPES[s["dtype"]]
    if kind == "mx4":
        q, exponent = _quantize_mx4(s["x"])
        x = q * _spread_mx4(exponent, s["in"])
        if s["requantize"]:
            q, exponent = _quantize_mx4(s["w"])
            w = q * _spread_mx4(exponent, s["in"])
        else:
            w = _unpack_mx4(s["wq"], s["ws"], s["in"])
        y = torch.bmm(_pad(x, s["offsets"], s["most"]), w.transpose(1, 2))
        return _unpad(y, s["offsets"], s["slots"]).to(dtype)
    stream = TYPES[s["stream"]]
    if kind == "dropout":
        y = _drop(s["x"], s["rng"], s["p"])
        return y.to(stream) if s["residual"] is None else (s["residual"].float() + y).to(stream)
    if kind == "norm_bwd":
        dy, h = s["dy"].float(), s["h"].float()
        rms = s["row_rms"][:, None]
        g = dy * s["gamma"]
        dh = s["dh"].float() + (g - h * ((g * h).mean(1, keepdim=True) / rms.square())) / rms
        dgamma = (dy * h / rms).sum(0)
        return _drop(dh, s["rng"], s["p"]).to(dtype), dh.to(stream), dgamma
    h = s["residual"].float() + _drop(s["x"], s["rng"], s["p"])
    rms = torch.sqrt(h.square().mean(1) + EPS)
    y = h / rms[:, None] * s["gamma"]
    if kind == "layer":
        q, exponent = _quantize_mx4(y)
        product = (q * _spread_mx4(exponent, s["cols"])) @ _unpack_mx4(s["wq"], s["ws"], s["cols"])[0].T
        return h.to(stream), product.to(dtype)
    if s["quantize"] == "e4m3":
        return *_quantize_e4m3(y), h.to(stream), rms
    return y.to(dtype), h.to(stream), rms


# ---------------------------------------------------------- the library's calls

def _calls(s):
    import row_wise_softmax_warp_gb300 as ro

    kind, dtype = s["kind"], TYPES[s["dtype"]]
    if kind == "mx4":
        xq, xs = ro.rowops_quantize_mx4(s["x"])
        wq, ws = ro.rowops_quantize_mx4(s["w"]) if s["requantize"] else (s["wq"], s["ws"])
        return ro.rowops_expert_matmul_mx4(xq, xs, wq, ws, s["offsets"], dtype=dtype)
    if kind == "dropout":
        return ro.rowops_dropout(s["x"], s["rng"], s["p"], residual=s["residual"], dtype=TYPES[s["stream"]])
    if kind == "norm_bwd":
        return ro.rowops_add_rmsnorm_bwd(s["dy"], s["gamma"], s["h"], s["row_rms"], dh=s["dh"], rng=s["rng"], p=s["p"])
    if kind == "layer":
        q, scale, h, _ = ro.rowops_add_rmsnorm_fwd(s["x"], s["gamma"], residual=s["residual"], rng=s["rng"], p=s["p"],
                                                   eps=EPS, quantize="mx4")
        return h, ro.rowops_expert_matmul_mx4(q, scale, s["wq"], s["ws"], dtype=dtype)
    y, scale, h, rms = ro.rowops_add_rmsnorm_fwd(s["x"], s["gamma"], residual=s["residual"], rng=s["rng"], p=s["p"],
                                                 eps=EPS, quantize=s["quantize"] or None)
    return (y, h, rms) if scale is None else (y, scale, h, rms)


def run(state):
    return _calls(state) if own else _plain(state)


# ----------------------------------------------------------- work and exact results

def work(case):
    kind, b = case["kind"], BYTES[case["dtype"]]
    if kind == "mx4":
        m, e, n, k = case["slots"], case["experts"], case["out"], case["in"]
        hit = e * (1.0 - (1.0 - 1.0 / e) ** m) if e > 1 else 1.0  # experts that get a row, where they are alike
        weights = hit * n * k * (b if case["requantize"] else 17 / 32)
        return {"bytes": m * (k + n) * b + weights + 4 * (e + 1), "flops": 2.0 * m * n * k}
    values, h = case["rows"] * case["cols"], BYTES[case["stream"]]
    if kind == "dropout":
        return {"bytes": values * (b + h * (2 if case["residual"] else 1)) + 16, "flops": 2 * values}
    if kind == "norm_bwd":
        # without dropout and with one type, both gradients are one
        dx = 0 if case["p"] == 0 and case["dtype"] == case["stream"] else b
        return {"bytes": values * (b + 3 * h + dx) + case["rows"] * 4 + case["cols"] * 8, "flops": 10 * values}
    if kind == "layer":
        return {"bytes": values * (b + 2 * h) + case["cols"] * 4 + case["out"] * (case["cols"] * 17 / 32 + case["rows"] * b),
                "flops": 2.0 * values * case["out"]}
    out = 1 + 4 / 128 if case["quantize"] else b
    return {"bytes": values * (b + 2 * h + out) + case["rows"] * 4 + case["cols"] * 4, "flops": 6 * values}


def _kept(rng, rows, cols, p):
    """Truth values (rows, cols): the generator from its definition, its products from 16-bit halves."""
    per = (cols + 7) // 8
    seed, offset = [v % 2 ** 64 for v in rng.tolist()]

    def product(x, m):
        """(high, low) 32 bits of x * m."""
        x0, x1, m0, m1 = x % 65536, x // 65536, m % 65536, m // 65536
        middle = x0 * m1 + x1 * m0 + x0 * m0 // 65536
        return x1 * m1 + middle // 65536, middle % 65536 * 65536 + x0 * m0 % 65536

    at = torch.arange(rows * per, device=rng.device)
    counter = [at % 2 ** 32, at // 2 ** 32, torch.full_like(at, offset % 2 ** 32), torch.full_like(at, offset // 2 ** 32)]
    for r in range(10):
        key = (seed % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32
        high0, low0 = product(counter[0], 0xD2511F53)
        high1, low1 = product(counter[2], 0xCD9E8D57)
        counter = [high1 ^ counter[1] ^ key[0], low1, high0 ^ counter[3] ^ key[1], low0]
    out = torch.empty(rows, per, 8, dtype=torch.bool, device=rng.device)
    for i in range(8):
        u = counter[i // 2] // (65536 if i % 2 else 1) % 65536
        out[:, :, i] = (u >= round(p * 65536)).reshape(rows, per)
    return out.reshape(rows, per * 8)[:, :cols]


def _dropped64(x, s):
    t = round(s["p"] * 65536)
    if t == 0:
        return x.double()
    return torch.where(_kept(s["rng"], *x.shape, s["p"]), x.double() * 65536 / (65536 - t), 0.0)


def _nearest(v, values):
    """The nearest of the rising values (ties to the one of even place) for v >= 0, the last for what lies behind it."""
    between = torch.tensor([(a + b) / 2 for a, b in zip(values, values[1:])], dtype=torch.float64, device=v.device)
    at = torch.searchsorted(between, v.contiguous())
    tie = (at < len(between)) & (v == between[at.clamp(max=len(between) - 1)])
    at = torch.where(tie & (at % 2 == 1), at + 1, at)
    return torch.tensor(values, dtype=torch.float64, device=v.device)[at]


def _mx4_64(x):
    """What x (fp64) stands for when it is quantised, a column of blocks at a time."""
    out = torch.empty_like(x)
    for c in range(0, x.shape[-1], 32):
        block = x[..., c:c + 32]
        most = block.abs().amax(dim=-1, keepdim=True)
        unit = torch.exp2((torch.floor(torch.log2(most.clamp(min=2.0 ** -140))) - 2).clamp(min=-127))
        out[..., c:c + 32] = torch.sign(block) * _nearest((block / unit).abs(), [0, 0.5, 1, 1.5, 2, 3, 4, 6]) * unit
    return out


def _e4m3_64(y):
    """(values, scales) of y (fp64), a block of 128 columns at a time."""
    grid = [m / 512 for m in range(8)] + [2.0 ** e * (1 + m / 8) for e in range(-6, 9) for m in range(8)][:-1]
    q, scale = torch.empty_like(y), torch.empty(y.shape[0], -(-y.shape[1] // 128), dtype=torch.float64, device=y.device)
    for b in range(scale.shape[1]):
        block = y[:, b * 128:b * 128 + 128]
        most = block.abs().amax(dim=1).clamp(min=2.0 ** -100)
        scale[:, b] = most / 448
        q[:, b * 128:b * 128 + 128] = torch.sign(block) * _nearest((block * 448 / most[:, None]).abs(), grid)
    return q, scale


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "mx4":
        if case["slots"] * case["in"] * case["out"] * 2.0 > 5e12:
            return None
        x = _mx4_64(s["x"].double())
        w = _mx4_64(s["w"].double())
        y = torch.zeros(case["slots"], case["out"], dtype=torch.float64, device="cuda")
        bounds = s["offsets"].tolist()
        for e in range(case["experts"]):
            y[bounds[e]:bounds[e + 1]] = x[bounds[e]:bounds[e + 1]] @ w[e].T
        return y
    if kind == "dropout":
        y = _dropped64(s["x"], s)
        return y if s["residual"] is None else s["residual"].double() + y
    gamma = s["gamma"].double()
    if kind == "norm_bwd":
        dy, h, rms = s["dy"].double(), s["h"].double(), s["row_rms"].double()[:, None]
        g = dy * gamma
        dh = s["dh"].double() + g / rms - h * (g * h).sum(1, keepdim=True) / (case["cols"] * rms ** 3)
        return _dropped64(dh, s), dh, (dy * h / rms).sum(0)
    h = s["residual"].double() + _dropped64(s["x"], s)
    rms = ((h * h).sum(1) / case["cols"] + EPS) ** 0.5
    y = gamma * h / rms[:, None]
    if kind == "layer":
        code = torch.empty(case["out"], -(-case["cols"] // 2) * 2, dtype=torch.int64, device="cuda")
        code[:, 0::2], code[:, 1::2] = s["wq"][0] % 16, s["wq"][0] // 16
        e, m, sign = code // 2 % 4, code % 2 / 2.0, 1.0 - 2.0 * (code // 8)  # e2m1: a sign, two bits, one bit
        w = sign * torch.where(e == 0, m, (1.0 + m) * 2.0 ** (e - 1).double())
        for c in range(s["ws"].shape[-1]):
            w[:, 32 * c:32 * c + 32] *= 2.0 ** (s["ws"][0, :, c:c + 1].double() - 127)
        return h, _mx4_64(y) @ w.double()[:, :case["cols"]].T
    return (*_e4m3_64(y), h, rms) if case["quantize"] else (y, h, rms)
