"""The router's choice, the combination of the experts' rows and their gradients on the GPU
against the float64 oracle.

Choices match exactly.  A weight is a quotient of exponentials: with d the spread of the
token's finite logits (sigmoid: their largest magnitude) exp is off by d 2^-24 and its own few
units, sums by their depth, the division and products by a unit each:
    r = (d + 32) 2^-23 of itself.
A gradient is a weight (and 1 - p) times a difference dw_j - mean; the mean over
approximate weights is off by r times the differences, and taken off twice by r^2 times
the largest:
    r (3 |d_j| + 3 sum_i q_i |d_i| + 4 r max |dw|) of the weight, and half a step of its type.
A combined row has top_k fused additions (2^-24 each of the sum of magnitudes), a
dweight the additions of N products, in any order at most N + 16.
"""

import numpy as np
import pytest

import oracle
from test_gpu_f8 import rows_apart
from test_gpu_mx import DEV, bf16_of, bf16_values, dev, guarded, host, intact, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dmm():
    import decode_matmul_amd
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return decode_matmul_amd


def typed(a, bf):
    return bf16_values(a) if bf else a.astype(np.float32)


def spread(z, score):
    live = np.where(np.isfinite(z), z, np.nan)
    if not np.isfinite(z).any(axis=1).all():
        live = np.where(np.isfinite(z).any(axis=1)[:, None], live, 0.0)
    d = np.nanmax(np.abs(live), axis=1) if score == "sigmoid" else np.nanmax(live, axis=1) - np.nanmin(live, axis=1)
    return (d + 32) * 2.0 ** -23


def gate(dmm, z, top_k, dtype, bias=None, mask=None, pad=3, **kw):
    M = z.shape[0]
    wi, ids = guarded(M * top_k, torch.int32)
    ww, w = guarded(M * top_k, torch.float32)
    dmm.moe_gate(rows_apart(z, dtype, pad), ids.view(M, top_k), w.view(M, top_k),
                 bias=None if bias is None else dev(bias), token_mask=None if mask is None else dev(mask), **kw)
    assert intact(wi) and intact(ww)
    return host(ids).reshape(M, top_k), host(w).reshape(M, top_k)


# M, E, top_k, n_groups, top_groups, group_top
GATE = [(1, 1, 1, 1, 1, 1), (1, 8, 2, 1, 1, 1), (3, 7, 7, 1, 1, 1), (16, 64, 8, 1, 1, 1), (5, 60, 4, 4, 2, 2),
        (100, 65, 6, 5, 3, 1), (33, 128, 8, 1, 1, 1), (16, 256, 8, 8, 4, 2), (70, 256, 8, 8, 4, 1), (9, 512, 32, 64, 8, 2),
        (20, 512, 8, 1, 1, 1), (64, 160, 6, 8, 3, 1), (40, 64, 3, 64, 5, 2), (7, 300, 9, 3, 1, 2), (1000, 16, 2, 1, 1, 1),
        (513, 128, 8, 4, 4, 2), (50, 96, 32, 2, 2, 2), (25, 8, 8, 2, 2, 2), (31, 32, 1, 1, 1, 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
@pytest.mark.parametrize("M,E,top_k,n_groups,top_groups,group_top", GATE, ids=["x".join(map(str, g)) for g in GATE])
def test_gate(dmm, M, E, top_k, n_groups, top_groups, group_top, biased, score, dtype):
    say(f"moe_gate M={M} E={E} top_k={top_k} groups={n_groups},{top_groups},{group_top} {biased} {score} {dtype}")
    rng = np.random.default_rng(M * 5 + E)
    z = typed(rng.standard_normal((M, E)) * 2, dtype == torch.bfloat16)
    if M > 4:
        z[1] = z[1, 0]                                              # all equal
        z[2, ::2] = -np.inf                                         # half of them are not there
        z[3] = -np.inf                                              # nor any
        z[4] = np.round(z[4])                                       # many ties
    bias = None
    if biased:
        bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
        bias[rng.random(E) < 0.2] = 0
        if E > 4:
            bias[E // 2] = -np.inf
    mask = (rng.random(M) < 0.8).astype(np.uint8) if M > 8 else None
    for renorm, scale in ((True, 2.5), (False, 1.0)):
        kw = dict(score=score, n_groups=n_groups, top_groups=top_groups, group_top=group_top, renorm=renorm, scale=scale)
        ids, w = gate(dmm, z, top_k, dtype, bias, mask, **kw)
        rids, rw = oracle.moe_gate(z, top_k, score, bias, n_groups, top_groups, group_top, renorm, scale, mask)
        assert np.array_equal(ids, rids)
        assert (np.abs(w - rw) <= spread(z, score)[:, None] * np.abs(rw)).all()


# More choices than lanes the experts fill; groups of no whole lanes, of one lane, of lanes that do not fit a wave.
FORMS = [(65, 64, 8, 1, 1, 1), (40, 64, 31, 1, 1, 1), (10, 48, 16, 1, 1, 1), (30, 8, 8, 1, 1, 1), (64, 160, 6, 8, 3, 2),
         (40, 64, 8, 16, 4, 2), (12, 64, 8, 32, 8, 2), (10, 24, 8, 3, 2, 1), (21, 63, 8, 7, 4, 2), (33, 500, 8, 5, 2, 2),
         (9, 510, 20, 6, 3, 1), (17, 36, 12, 4, 2, 2)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
@pytest.mark.parametrize("M,E,top_k,n_groups,top_groups,group_top", FORMS, ids=["x".join(map(str, g)) for g in FORMS])
def test_gate_forms(dmm, M, E, top_k, n_groups, top_groups, group_top, biased, score, dtype):
    test_gate(dmm, M, E, top_k, n_groups, top_groups, group_top, biased, score, dtype)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n_groups,group_top", [(1, 1), (4, 2)])
@pytest.mark.parametrize("E", [16, 64, 128, 256])
def test_gate_next_to_borders(dmm, E, n_groups, group_top, score):
    """Scores a few units of fp32 apart, that rounding to fp32 puts in the wrong order or
    makes equal: the order is float64's."""
    say(f"moe_gate borders E={E} {score} {n_groups}")
    rng = np.random.default_rng(E)
    M, top_k = 400, 6
    base = rng.standard_normal((M, 1))
    z = (base + rng.integers(-3, 4, (M, E)) * 2.0 ** -22).astype(np.float32)
    bias = (rng.integers(-2, 3, E) * 2.0 ** -25).astype(np.float32)
    for b in (None, bias, np.float32(1.0) - oracle.gate_scores(z[:1], score)[0].astype(np.float32)):
        kw = dict(score=score, n_groups=n_groups, top_groups=max(1, n_groups // 2), group_top=group_top)
        ids, _ = gate(dmm, z, top_k, torch.float32, b, **kw)
        rids, _ = oracle.moe_gate(z, top_k, bias=b, **kw)
        assert np.array_equal(ids, rids)


def test_gate_of_many_tokens(dmm):
    """A whole batch, each kind of score: the choices of a stable sort in float64 on the CPU."""
    say("moe_gate of many tokens")
    rng = np.random.default_rng(0)
    for M, E, k, bf in ((20000, 128, 8, True), (5000, 256, 8, False), (20001, 64, 6, False)):
        z = typed(rng.standard_normal((M, E)), bf)
        bias = (rng.standard_normal(E) * 0.05).astype(np.float32)
        for score in ("softmax", "sigmoid"):
            for b in (None, bias):
                ids, _ = gate(dmm, z, k, torch.bfloat16 if bf else torch.float32, b, score=score, pad=0)
                c = z.astype(np.float64) if b is None else oracle.gate_scores(z, score) + b.astype(np.float64)
                assert np.array_equal(ids, np.argsort(-c, axis=1, kind="stable")[:, :k])


def test_gate_of_infinities_and_nan(dmm):
    """NaN ranks above all; +inf and NaN make a softmax's weights NaN; zeros of both signs tie."""
    say("moe_gate infinities and NaN")
    inf, nan = np.inf, np.nan
    z = np.array([[0, 1, nan, 2], [nan, 1, nan, 2], [0, inf, 3, 2], [-0.0, 0.0, -0.0, 0.0], [-inf, -inf, 5, -inf],
                  [88, -88, 200, -200], [3e38, -3e38, 1, 2]], np.float32)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            for bias in (None, np.array([0, 0, 0, 0.5], np.float32), np.array([nan, 0, inf, -inf], np.float32)):
                ids, w = gate(dmm, z, 3, torch.float32, bias, score=score, renorm=renorm)
                with np.errstate(all="ignore"):
                    rids, rw = oracle.moe_gate(z, 3, score, bias, renorm=renorm)
                assert np.array_equal(ids, rids)
                assert np.array_equal(np.isnan(w), np.isnan(rw))
                fine = ~np.isnan(rw)
                # spread of up to 6e38: exp is 0 or 1 there; below 2^-126 a weight may be 0
                tol = np.minimum(spread(np.clip(z, -300, 300), score), 1)[:, None] * np.abs(rw) + 2.0 ** -126
                assert (np.abs(w - rw)[fine] <= tol[fine]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("M,E,top_k", [(1, 1, 1), (1, 8, 2), (7, 7, 7), (16, 64, 8), (33, 65, 6), (300, 128, 8),
                                       (20, 256, 8), (9, 512, 32), (100, 20, 20), (65, 130, 9)])
def test_gate_grad(dmm, M, E, top_k, renorm, score, dtype):
    say(f"moe_gate_grad M={M} E={E} top_k={top_k} {renorm} {score} {dtype}")
    rng = np.random.default_rng(M + E)
    bf = dtype == torch.bfloat16
    z = typed(rng.standard_normal((M, E)) * 3, bf)
    z[rng.random((M, E)) < 0.05] = -np.inf
    if M > 3:
        z[2, 0] = 30
        z[3] = -40
    z = typed(z, bf)
    ids, _ = oracle.moe_gate(z, top_k, score)
    if M > 6:
        ids[5] = -1
        ids[6, 0] = E                                               # of no expert
        ids[4, top_k - 1] = ids[4, 0]                               # the same one twice
    dw = rng.standard_normal((M, top_k)).astype(np.float32)
    given = dw.copy()
    given[(ids < 0) | (ids >= E)] = np.nan                          # not read
    zz = z.copy()
    if M > 6:
        zz[5] = np.nan                                              # nor is a row without an expert
    whole, g = guarded(M * E, dtype)
    dmm.moe_gate_grad(rows_apart(zz, dtype, 3), dev(ids), dev(given), g.view(M, E), score=score, renorm=renorm, scale=1.5)
    got = host(g).reshape(M, E).astype(np.float64)
    ref = oracle.moe_gate_grad(z, ids, dw, score, renorm, 1.5)
    assert intact(whole)
    tol = grad_tolerance(z, ids, dw, score, renorm, 1.5) + (2.0 ** -8 if bf else 2.0 ** -24) * np.abs(ref) + 2.0 ** -126
    assert (np.abs(got - ref) <= tol).all()
    if M > 6:
        assert not got[5].any()


def grad_tolerance(z, ids, dw, score, renorm, scale):
    M, E = z.shape
    r, tol = spread(z, score), np.zeros((M, E))
    for t in range(M):
        on = (ids[t] >= 0) & (ids[t] < E)
        if not on.any():
            continue
        e, d = ids[t][on], dw[t][on].astype(np.float64)
        if renorm or score == "sigmoid":
            lp = z[t, e].astype(np.float64) if score == "softmax" else -np.logaddexp(0.0, -z[t, e].astype(np.float64))
            q = np.exp(lp - (lp.max() if renorm else 0))
            rest = 1.0 if score == "softmax" else np.exp(-np.logaddexp(0.0, z[t, e].astype(np.float64)))
            if renorm:
                q /= q.sum()
                c = np.abs(d - (q * d).sum())
                off = r[t] * (3 * c + 3 * (q * c).sum() + 4 * r[t] * np.abs(d).max())
            else:
                off = r[t] * np.abs(d)
            np.add.at(tol[t], e, scale * q * rest * off)
        else:
            p, g = oracle.gate_scores(z[t:t + 1], "softmax")[0], np.zeros(E)
            np.add.at(g, e, scale * d)
            c = np.abs(g - (p * g).sum())
            tol[t] = p * r[t] * (3 * c + 3 * (p * c).sum() + 4 * r[t] * np.abs(g).max())
    return tol


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("gap", [0, 6, 12, 17])
def test_gate_grad_of_a_sure_choice(dmm, gap, renorm, score):
    """One logit `gap` ahead of 63 others: the gradients of the rest, and of the one, keep
    their digits (the tolerance is relative to the differences, not to the mean)."""
    say(f"moe_gate_grad gap={gap} {score} {renorm}")
    z = np.zeros((4, 64), np.float32)
    z[:, 9] = gap
    ids, _ = oracle.moe_gate(z, 4, score)
    dw = np.tile(np.array([[1.0, -2.0, 0.5, 3.0]], np.float32), (4, 1))
    g = torch.zeros((4, 64), device=DEV)
    dmm.moe_gate_grad(dev(z), dev(ids), dev(dw), g, score=score, renorm=renorm)
    ref = oracle.moe_gate_grad(z, ids, dw, score, renorm)
    tol = grad_tolerance(z, ids, dw, score, renorm, 1.0) + 2.0 ** -24 * np.abs(ref)
    assert (np.abs(host(g) - ref) <= tol).all()
    assert (np.abs(host(g) - ref) <= 1e-3 * np.abs(ref)).all() or gap > 12


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_grad_by_differences(dmm, renorm, score):
    """Central differences of the GPU's own weights (the choice holds still: the steps are
    smaller than the gaps).  h = 2^-7: truncation h^2 / 6 of the third derivative (below 6
    sum |dw|), the weights' rounding r sum |dw w| / h."""
    say(f"moe_gate differences {score} {renorm}")
    rng = np.random.default_rng(3)
    M, E, k, h = 3, 6, 3, 2.0 ** -7
    z = np.stack([rng.permutation(E) for _ in range(M)]).astype(np.float32) * 0.5
    dw = rng.standard_normal((M, k)).astype(np.float32)

    def f(a):
        ids, w = gate(dmm, a.astype(np.float32), k, torch.float32, score=score, renorm=renorm)
        return ids, (w.astype(np.float64) * dw).sum()

    ids, _ = f(z)
    g = torch.zeros((M, E), device=DEV)
    dmm.moe_gate_grad(dev(z), dev(ids), dev(dw), g, score=score, renorm=renorm)
    g = host(g)
    r = spread(z, score).max()
    for t in range(M):
        for e in range(E):
            up, dn = z.copy(), z.copy()
            up[t, e] += h
            dn[t, e] -= h
            (iu, fu), (idn, fd) = f(up), f(dn)
            assert np.array_equal(iu, ids) and np.array_equal(idn, ids)
            assert abs((fu - fd) / (2 * h) - g[t, e]) <= h * h * np.abs(dw).sum() + r * np.abs(dw).sum() / h


# --------------------------------------------------------------- combination

COMBINE = [(1, 1, 1), (1, 2, 64), (3, 8, 100), (16, 8, 4096), (33, 3, 257), (5, 2, 2049), (2, 32, 1000), (300, 4, 512),
           (7, 1, 8192), (4, 6, 20001)]


@pytest.mark.parametrize("yt", [torch.float32, torch.bfloat16], ids=["yf32", "ybf16"])
@pytest.mark.parametrize("ot", [torch.float32, torch.bfloat16], ids=["of32", "obf16"])
@pytest.mark.parametrize("M,top_k,N", COMBINE, ids=["x".join(map(str, c)) for c in COMBINE])
def test_combine_and_gradient(dmm, M, top_k, N, yt, ot):
    say(f"moe_combine M={M} top_k={top_k} N={N} {yt} {ot}")
    rng = np.random.default_rng(M + top_k + N)
    E = 16
    ids = rng.integers(0, E, (M, top_k)).astype(np.int32)
    ids[rng.random((M, top_k)) < 0.2] = -1
    if M > 2:
        ids[1], ids[2, 0] = -1, E                                   # a token of no expert
    on = (ids >= 0) & (ids < E)
    y = typed(rng.standard_normal((M, top_k, N)).reshape(M * top_k, N), yt == torch.bfloat16).reshape(M, top_k, N)
    w = rng.standard_normal((M, top_k)).astype(np.float32)
    y[~on], w[~on] = np.nan, np.inf                                 # whatever is there
    add, dout = (typed(rng.standard_normal((M, N)), ot == torch.bfloat16) for _ in range(2))

    def of(a, dtype):
        return bf16_of(a.reshape(-1, a.shape[-1])).reshape(a.shape) if dtype == torch.bfloat16 else dev(a)

    Y, I, W = of(y, yt), dev(ids), dev(w)
    step = 2.0 ** -8 if ot == torch.bfloat16 else 0.0
    for a in (None, add):
        whole, out = guarded(M * N, ot)
        if a is not None and N % 2:                                 # in place
            out.copy_(of(a, ot).view(-1))
            dmm.moe_combine(Y, I, W, E, out.view(M, N), add=out.view(M, N))
        else:
            dmm.moe_combine(Y, I, W, E, out.view(M, N), add=None if a is None else of(a, ot))
        ref, B = oracle.moe_combine(y.astype(np.float64), ids, w.astype(np.float64), E, a)
        assert (np.abs(host(out).reshape(M, N) - ref) <= (top_k + 1) * 2.0 ** -24 * B + step * np.abs(ref)).all()
        assert intact(whole)
    whole, dy = guarded(M * top_k * N, yt)
    dw = torch.full((M, top_k), 7.0, device=DEV)
    dmm.moe_combine_grad(Y, I, W, E, of(dout, ot), dy.view(M, top_k, N), dw)
    rdy, rdw, B = oracle.moe_combine_grad(y.astype(np.float64), ids, w.astype(np.float64), E, dout.astype(np.float64))
    got = host(dy).reshape(M, top_k, N)
    assert (np.abs(got - rdy) <= (2.0 ** -8 if yt == torch.bfloat16 else 2.0 ** -24) * np.abs(rdy) * (1 + 2.0 ** -20)).all()
    assert (np.abs(host(dw) - rdw) <= (N + 16) * 2.0 ** -24 * B).all()
    assert intact(whole) and not got[~on].any() and not host(dw)[~on].any()
    # in place of y
    again = Y.clone()
    dw2 = torch.full((M, top_k), 7.0, device=DEV)
    dmm.moe_combine_grad(again, I, W, E, of(dout, ot), again, dw2)
    assert torch.equal(again.view(-1), dy) and torch.equal(dw2, dw)


def test_combine_of_nothing(dmm):
    say("moe_combine of nothing")
    y, ids, w = torch.zeros((3, 2, 0), device=DEV), torch.zeros((3, 2), dtype=torch.int32, device=DEV), torch.ones((3, 2), device=DEV)
    dmm.moe_combine(y, ids, w, 4, torch.zeros((3, 0), device=DEV))
    dw = torch.full((3, 2), 7.0, device=DEV)
    dmm.moe_combine_grad(y, ids, w, 4, torch.zeros((3, 0), device=DEV), y, dw)
    assert not host(dw).any()
    dmm.moe_combine(torch.zeros((0, 2, 5), device=DEV), ids[:0], w[:0], 4, torch.zeros((0, 5), device=DEV))
