"""Plain 64-bit forms of the expert operators (numpy), written from their formulas."""
import numpy as np


def plan(indices, values, experts):
    """(offsets, order, slot) by a loop over the pairs."""
    rows, k = indices.shape
    lists = [[] for _ in range(experts)]
    for p, i in enumerate(indices.reshape(-1)):
        if 0 <= i < experts and (values is None or values.reshape(-1)[p] != 0):
            lists[int(i)].append(p)
    offsets = np.cumsum([0] + [len(x) for x in lists]).astype(np.int32)
    order = np.full(rows * k, -1, np.int32)
    flat = [p for x in lists for p in x]
    order[:len(flat)] = flat
    slot = np.full(rows * k, -1, np.int32)
    slot[flat] = np.arange(len(flat))
    return offsets, order, slot.reshape(rows, k)


def _there(slot, slots):
    return [(t, j, s) for t, row in enumerate(slot) for j, s in enumerate(row) if 0 <= s < slots]


def combine(y, slot, weights):
    out = np.zeros((slot.shape[0], y.shape[1]))
    for t, j, s in _there(slot, len(y)):
        out[t] += (1.0 if weights is None else np.float64(weights[t, j])) * y[s]
    return out


def combine_magnitude(y, slot, weights):
    return combine(np.abs(y), slot, None if weights is None else np.abs(weights))


def combine_bwd(dout, y, slot, weights, dy):
    """dy (a copy, with the rows that a slot names replaced) and dweights."""
    dy, dw = dy.astype(np.float64).copy(), np.zeros(slot.shape)
    for t, j, s in _there(slot, len(y)):
        dy[s] = np.float64(weights[t, j]) * dout[t]
        dw[t, j] = np.dot(dout[t], y[s])
    return dy, dw


def groups(offsets, slots):
    if offsets is None:
        return [(0, slots)]
    return [(offsets[e], offsets[e + 1]) for e in range(len(offsets) - 1)]


def matmul(x, w, offsets):
    """Rows that no expert has are NaN.  w: (experts, out, in)."""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    for e, (a, b) in enumerate(groups(offsets, len(x))):
        y[a:b] = x[a:b] @ w[e].T
    return y


def wgrad(dy, x, offsets):
    return np.stack([dy[a:b].T @ x[a:b] for a, b in groups(offsets, len(x))])


def e4m3(v):
    """Nearest e4m3 value, ties to even; magnitudes up to 448."""
    exponent = np.maximum(np.frexp(v)[1] - 1, -6)
    step = np.exp2(exponent - 3.0)
    return np.rint(v / step) * step


def quantize(x, block_rows):
    """(values, scale) of the last two dimensions' blocks; non-finite entries become NaN."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape[-2:]
    q = np.empty_like(x)
    scale = np.empty((*x.shape[:-2], -(-rows // block_rows), -(-cols // 128)))
    for index in np.ndindex(*scale.shape):
        *b, r, c = index
        at = (*b, slice(r * block_rows, (r + 1) * block_rows), slice(c * 128, (c + 1) * 128))
        block = x[at]
        fine = np.isfinite(block)
        a = max(np.max(np.abs(block[fine]), initial=0.0), 2.0 ** -100)
        scale[index] = a / 448.0
        q[at] = np.where(fine, e4m3(np.where(fine, block, 0.0) * 448.0 / a), np.nan)
    return q, scale


def spread(scale, block_rows, rows, cols):
    s = np.repeat(scale, block_rows, axis=-2)[..., :rows, :]
    return np.repeat(s, 128, axis=-1)[..., :cols]
