"""Plain 64-bit forms (numpy) of dropout, the residual's addition with its norm, and
microscaled 4-bit values, written from their formulas."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def philox(key, counter):
    """Philox4x32-10 of counters (n, 4) under key (2,): (n, 4), all uint64 below 2^32."""
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    a, b, c, d = (np.asarray(v, np.uint64).copy() for v in np.asarray(counter, np.uint64).T)
    k, l = (int(v) for v in key)
    for _ in range(10):
        m, n = a * np.uint64(0xD2511F53), c * np.uint64(0xCD9E8D57)
        a, b, c, d = (n >> half) ^ b ^ np.uint64(k), n & low, (m >> half) ^ d ^ np.uint64(l), m & low
        k, l = (k + 0x9E3779B9) % 2 ** 32, (l + 0xBB67AE85) % 2 ** 32
    return np.stack([a, b, c, d], 1)


def kept(rng, rows, cols, p):
    """Truth values (rows, cols): what dropout keeps."""
    per = -(-cols // 8)
    key, offset = (int(v) % 2 ** 64 for v in rng)
    j = np.arange(rows * per, dtype=np.uint64)
    counter = np.stack([j & np.uint64(0xFFFFFFFF), j >> np.uint64(32), np.full_like(j, offset % 2 ** 32),
                        np.full_like(j, offset >> 32)], 1)
    words = philox((key % 2 ** 32, key >> 32), counter)
    halves = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], 2).reshape(rows, per * 8)
    return halves[:, :cols] >= threshold(p)


def threshold(p):
    return int(np.rint(np.float64(np.float32(p)) * 65536))


def drop(x, rng, p):
    t = threshold(p)
    if t in (0, 65536):
        return x * (t == 0)
    return np.where(kept(rng, *x.shape, p), x * (65536.0 / (65536 - t)), 0.0)


def add_norm(x, residual, gamma, rng, p, eps):
    """(h, rms, y)"""
    h = drop(x, rng, p) + (0.0 if residual is None else residual)
    rms = np.sqrt((h * h).mean(1) + eps)
    return h, rms, gamma * h / rms[:, None]


def add_norm_bwd(dy, gamma, h, rms, dh, rng, p):
    """(dx, dresidual, dgamma)"""
    n = h / rms[:, None]
    g = dy * gamma
    t = (g - n * (g * n).mean(1, keepdims=True)) / rms[:, None] + (0.0 if dh is None else dh)
    return drop(t, rng, p), t, (dy * n).sum(0)


def nearest_e2m1(v):
    """Nearest e2m1 value, ties to the even code, 6 for what lies above."""
    m = np.abs(v)
    step = np.where(m < 2, 0.5, np.where(m < 4, 1.0, 2.0))
    return np.copysign(np.minimum(np.rint(m / step) * step, 6.0), v)


def quantize_mx4(x):
    """(values, scale codes) of blocks of 32 columns."""
    x = np.asarray(x, np.float64)
    cols = x.shape[-1]
    q, code = np.zeros_like(x), np.zeros((*x.shape[:-1], -(-cols // 32)), np.int64)
    for b in range(code.shape[-1]):
        block = x[..., 32 * b:32 * b + 32]
        fine = np.isfinite(block).all(-1)
        a = np.abs(np.where(np.isfinite(block), block, 0.0)).max(-1)
        e = np.where(a > 0, np.frexp(a)[1] - 1 - 2, -127)
        e = np.maximum(e, -127)
        code[..., b] = np.where(fine, e + 127, 255)
        q[..., 32 * b:32 * b + 32] = np.where(fine[..., None], nearest_e2m1(np.where(fine[..., None], block, 0.0) * np.exp2(-e.astype(np.float64))[..., None]), 0.0)
    return q, code


def unpack_mx4(packed, cols):
    """e2m1 values of bytes (..., ceil(cols / 2))."""
    packed = np.asarray(packed, np.int64)
    code = np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)[..., :cols]
    return np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]


def spread_mx4(code, cols):
    """The scale of each column (NaN for code 255)."""
    code = np.asarray(code, np.float64)
    s = np.where(code == 255, np.nan, np.exp2(code - 127))
    return np.repeat(s, 32, axis=-1)[..., :cols]
