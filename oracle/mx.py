"""MXFP4 and the experts' routing, from their definitions, in float64.

MXFP4 (OCP Microscaling Formats): 32 consecutive values of a row share an E8M0
byte s (scale 2^(s - 127), 255 = NaN); an element is one of the e2m1 values
+-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, two a byte, the first in the low nibble.
"""

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx_pack(w):
    """w float32 [rows, K] -> (codes uint8 [rows, nb, 16], scales uint8 [rows, nb],
    whether every value is finite)."""
    w = np.asarray(w, dtype=np.float32)
    rows, K = w.shape
    nb = -(-K // 32)
    v = np.zeros((rows, nb * 32))
    v[:, :K] = w
    v = v.reshape(rows, nb, 32)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[:, :, None], 0.0, v)
    top = np.abs(v).max(axis=2)
    _, ex = np.frexp(top)                              # top = f 2^ex, 0.5 <= f < 1
    s = np.where(top > 0, np.clip(ex - 1 - 2 + 127, 0, 254), 0)
    a = np.abs(v) * 2.0 ** (127.0 - s)[:, :, None]
    d = np.abs(a[..., None] - E2M1)
    near = d == d.min(axis=-1, keepdims=True)          # one value, or the two around a tie
    even = near & (np.arange(8) % 2 == 0)
    c = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    c = c | np.where(np.signbit(v), 8, 0)
    c = np.where(bad[:, :, None], 0, c).astype(np.uint8)
    s = np.where(bad, 255, s).astype(np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), s, not bad.any()


def mx_unpack(codes, scales, K):
    """The values of a package, float64 [..., K]."""
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(codes.shape[:-1] + (32,))
    v = np.where(c > 7, -1.0, 1.0) * E2M1[c & 7]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127.0))
    v = v * s[..., None]
    return v.reshape(codes.shape[:-2] + (-1,))[..., :K]


def moe_route(ids, E):
    """counts [E], offsets [E + 1], order [M * top_k] of expert ids [M, top_k]."""
    flat = np.asarray(ids).reshape(-1)
    lists = [np.nonzero(flat == e)[0] for e in range(E)]
    rest = np.nonzero((flat < 0) | (flat >= E))[0]
    counts = np.array([len(l) for l in lists], dtype=np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return counts, offsets, np.concatenate(lists + [rest]).astype(np.int32)


def moe_balance(z, counts, mask=None):
    """(loss, weights [E], p [M, E]) of float64 logits; p is 0 for masked
    tokens and for rows of -inf."""
    z = np.asarray(z, dtype=np.float64)
    M, E = z.shape
    keep = np.ones(M, bool) if mask is None else np.asarray(mask) != 0
    T, n = int(keep.sum()), int(np.sum(counts))
    w = np.asarray(counts, dtype=np.float64) * E / (T * n) if T and n else np.zeros(E)
    p = np.zeros((M, E))
    live = keep & ~np.all(z == -np.inf, axis=1)
    e = np.exp(z[live] - z[live].max(axis=1, keepdims=True))
    p[live] = e / e.sum(axis=1, keepdims=True)
    return float((p * w).sum()), w, p


def moe_balance_grad(z, counts, mask=None):
    """dloss/dz, float64 [M, E]."""
    _, w, p = moe_balance(z, counts, mask)
    return p * (w - (p * w).sum(axis=1, keepdims=True))
