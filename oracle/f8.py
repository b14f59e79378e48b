"""e4m3 packages and their products, the norm that packs, the router's choice and the
combination of the experts' rows, from their definitions, in float64.

e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; largest 448, no infinities,
0x7f and 0xff are NaN.  A package has blocks of 128 columns with an fp32 scale for
each block_rows rows.
"""

import numpy as np


def _e4m3():
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c > 127, -v, v)


E4M3 = _e4m3()


def f8_encode(v):
    """The codes of the e4m3 values nearest to v, |v| <= 448, ties to the even code."""
    grid = E4M3[:127]                                  # 0 .. 448, rising with the code
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)     # grid[hi - 1] < a <= grid[hi]
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (c + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def f8_pack(w, block_rows):
    """w float32 [rows, K] -> (codes uint8 [rows, nb, 128], scales float32
    [ceil(rows / block_rows), nb], whether every value is finite)."""
    w = np.asarray(w, dtype=np.float32)
    rows, K = w.shape
    nb, nr = -(-K // 128), -(-rows // block_rows)
    v = np.zeros((nr * block_rows, nb * 128))
    v[:rows, :K] = w
    v = v.reshape(nr, block_rows, nb, 128)
    bad = ~np.isfinite(v).all(axis=(1, 3))
    v = np.where(bad[:, None, :, None], 0.0, v)
    top = np.abs(v).max(axis=(1, 3))
    s = 2.0 ** np.maximum(np.ceil(np.log2(np.maximum(top, 2.0 ** -149) / 448)), -126)
    s = np.where((s > 2.0 ** -126) & (top <= 448 * s / 2), s / 2, s)        # log2's own rounding
    s = np.where(top > 448 * s, s * 2, s)
    c = np.where(bad[:, None, :, None], 0, f8_encode(v / s[:, None, :, None]))
    s = np.where(bad, np.nan, s).astype(np.float32)
    return c.reshape(nr * block_rows, nb, 128)[:rows].astype(np.uint8), s, not bad.any()


def f8_unpack(codes, scales, K, block_rows):
    """The values of a package [rows, nb, 128], float64 [rows, K]."""
    rows = codes.shape[0]
    s = np.repeat(scales.astype(np.float64), block_rows, axis=0)[:rows]
    return (E4M3[codes] * s[:, :, None]).reshape(rows, -1)[:, :K]


def f8_matmul(x, w, bias=None):
    """(y, sum of magnitudes) for decoded float64 x [M, K] and w [N, K]."""
    y, B = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        y, B = y + bias, B + np.abs(bias)
    return y, B


def f8_norm(x, residual, weight, eps, store):
    """(h, y): the sum, rounded by `store` (float64 -> stored values), and its norm in
    fp32, each as float32 values."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    h = store(h).astype(np.float64)
    f = (1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)).astype(np.float32)
    y = h.astype(np.float32) * f
    return h.astype(np.float32), y * np.asarray(weight, dtype=np.float32)


def gate_scores(z, score):
    z = np.asarray(z, dtype=np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-z))
    with np.errstate(invalid="ignore"):
        e = np.exp(z - z.max(axis=1, keepdims=True))
        return e / e.sum(axis=1, keepdims=True)


def _first(values, open_):
    """Index of the largest value among the open ones (NaN above all, ties to the lowest)."""
    at = np.nonzero(open_)[0]
    if len(at) == 0:
        return -1
    v = values[at]
    nan = np.nonzero(np.isnan(v))[0]
    return int(at[nan[0]] if len(nan) else at[np.argmax(v)])


def moe_gate(z, top_k, score="softmax", bias=None, n_groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0,
             mask=None):
    """(ids int32 [M, top_k], weights float64 [M, top_k])."""
    z = np.asarray(z, dtype=np.float64)
    M, E = z.shape
    size = E // n_groups
    ids, w = np.full((M, top_k), -1, np.int32), np.zeros((M, top_k))
    for t in range(M):
        if mask is not None and not mask[t]:
            continue
        there = z[t] != -np.inf
        if bias is not None:
            there &= bias != -np.inf
        if not there.any():
            continue
        p = gate_scores(z[t:t + 1], score)[0]
        c = z[t] if bias is None else p + bias
        if n_groups > 1:
            of = np.where(there, p if bias is None and group_top > 1 else c, -np.inf)
            rank = np.sort(of.reshape(n_groups, size), axis=1)[:, ::-1][:, :min(group_top, size)]    # NaN first
            total = rank.sum(axis=1)
            total = np.where(np.isnan(of.reshape(n_groups, size)).any(axis=1), np.nan, total)
            left = np.ones(n_groups, bool)
            keep = np.zeros(n_groups, bool)
            for _ in range(top_groups):
                g = _first(total, left)
                left[g], keep[g] = False, True
            there &= np.repeat(keep, size)
        for j in range(top_k):
            e = _first(c, there)
            if e < 0:
                break
            ids[t, j], there[e] = e, False
        on = ids[t] >= 0
        zj = z[t, ids[t][on]]
        if not on.any():
            continue
        if score == "softmax":
            if renorm:
                e = np.exp(zj - zj.max())
                w[t, on] = e / e.sum()
            else:
                w[t, on] = p[ids[t][on]]
        else:
            # log p = -log(1 + e^-z); a common factor leaves the quotients
            with np.errstate(over="ignore"):
                lp = -np.logaddexp(0.0, -zj)
            w[t, on] = np.exp(lp - lp.max()) / np.exp(lp - lp.max()).sum() if renorm else np.exp(lp)
    return ids, w * scale


def moe_gate_grad(z, ids, dw, score="softmax", renorm=True, scale=1.0):
    """dlogits float64 [M, E], by the chain rule through the scores."""
    z = np.asarray(z, dtype=np.float64)
    M, E = z.shape
    out = np.zeros((M, E))
    for t in range(M):
        on = (ids[t] >= 0) & (ids[t] < E)
        if not on.any():
            continue
        e, d = ids[t][on], np.asarray(dw[t], dtype=np.float64)[on]
        zj = z[t, e]
        if renorm:
            lp = zj if score == "softmax" else -np.logaddexp(0.0, -zj)
            q = np.exp(lp - lp.max())
            q /= q.sum()
            g = scale * q * (d - (q * d).sum())                 # by log p
            if score == "sigmoid":
                g = g * np.exp(-np.logaddexp(0.0, zj))          # 1 - p
            np.add.at(out[t], e, g)
        elif score == "sigmoid":
            np.add.at(out[t], e, scale * d * np.exp(-np.logaddexp(0.0, -zj) - np.logaddexp(0.0, zj)))
        else:
            p, g = gate_scores(z[t:t + 1], "softmax")[0], np.zeros(E)
            np.add.at(g, e, scale * d)
            out[t] = p * (g - (p * g).sum())
    return out


def moe_combine(y, ids, w, E, add=None):
    """(out, sum of magnitudes) float64 [M, N]."""
    on = ((ids >= 0) & (ids < E))[:, :, None]
    terms = np.where(on, np.where(on, y, 0.0) * np.where(on, w[:, :, None], 0.0), 0.0)
    out, B = terms.sum(axis=1), np.abs(terms).sum(axis=1)
    return (out, B) if add is None else (out + add, B + np.abs(add))


def moe_combine_grad(y, ids, w, E, dout):
    """(dy, dweights, sum of magnitudes of dweights), float64."""
    on = (ids >= 0) & (ids < E)
    yy, ww = np.where(on[:, :, None], y, 0.0), np.where(on, w, 0.0)
    return (ww[:, :, None] * dout[:, None, :], np.einsum("tjn,tn->tj", yy, dout),
            np.einsum("tjn,tn->tj", np.abs(yy), np.abs(dout)))
