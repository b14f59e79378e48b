"""The experts' routing, the balance loss and the grouped MXFP4 product on the
GPU against the float64 oracle.

Lists and counts are whole numbers and match exactly; products carry the
tolerance of tests/test_gpu_mx.py.  For the loss, p = exp(z - top) / sum: the
difference is off by 2^-24 of its size d, so exp by d 2^-24 and its own few
units, the sums by their depth (at most 8 + 6 additions) and the division and
product by a unit each: p is within (d + 32) 2^-23 of itself, and so is
sum_e w_e p_e of nonnegative terms.  The gradient p (w - s) is then off by at
most (d + 32) 2^-23 p (|w| + 2 s), and half a step of its type.
"""

import numpy as np
import pytest

import oracle
import workloads
from test_gpu_mx import DEV, activations, assert_close, bf16_of, bf16_values, dev, guarded, host, intact, packed, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dmm():
    import decode_matmul_amd
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return decode_matmul_amd


def route(dmm, ids, E):
    M, top_k = ids.shape
    counts, offsets, order = (torch.full((n,), -7, dtype=torch.int32, device=DEV) for n in (E, E + 1, M * top_k))
    n = dmm.moe_route_workspace_bytes(M, top_k, E)
    ws = torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV) if n else None
    dmm.moe_route(dev(ids), E, counts, offsets, order, workspace=ws)
    return counts, offsets, order


# ------------------------------------------------------------------- routing

ROUTE = [(1, 1, 1), (1, 8, 64), (16, 8, 64), (3, 5, 2), (64, 1, 7), (333, 3, 60), (512, 8, 512), (513, 8, 64),
         (1000, 7, 128), (5000, 8, 511), (70001, 4, 33), (1, 1, 512), (65536, 8, 128)]


@pytest.mark.parametrize("M,top_k,E", ROUTE, ids=["x".join(map(str, r)) for r in ROUTE])
def test_route(dmm, M, top_k, E):
    say(f"moe_route M={M} top_k={top_k} E={E}")
    rng = np.random.default_rng(M + E)
    ids = rng.integers(-1, E + 1, (M, top_k)).astype(np.int32)      # -1 and E belong to no expert
    ids[rng.random((M, top_k)) < 0.3] = E // 2                      # one busy expert
    if M > 4:
        ids[2] = np.iinfo(np.int32).max
        ids[3] = np.iinfo(np.int32).min
    got = route(dmm, ids, E)
    for g, r in zip(got, oracle.moe_route(ids, E)):
        assert np.array_equal(host(g), r)


@pytest.mark.parametrize("fill", [0, 5, -1])
@pytest.mark.parametrize("M", [0, 1, 4096, 9000])
def test_route_of_one_value(dmm, M, fill):
    say(f"moe_route M={M} all {fill}")
    ids = np.full((M, 1), fill, np.int32)
    for g, r in zip(route(dmm, ids, 6), oracle.moe_route(ids, 6)):
        assert np.array_equal(host(g), r)


# ------------------------------------------------------------------- balance


def balance_tolerances(z, w, p):
    live = np.where(np.isfinite(z), z, np.nan)
    with np.errstate(all="ignore"):
        d = np.nan_to_num(np.nanmax(live, axis=1) - np.nanmin(live, axis=1)) if z.size else np.zeros(0)
    rel = (d + 32) * 2.0 ** -23
    s = (p * w).sum(axis=1)
    return (rel * s).sum() + 2.0 ** -24 * s.sum(), rel[:, None] * p * (np.abs(w) + 2 * s[:, None])


BALANCE = [(1, 1), (1, 2), (1, 64), (7, 3), (16, 64), (100, 65), (65, 60), (300, 128), (1000, 256), (33, 257),
           (50, 512), (5000, 8), (64, 100)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("M,E", BALANCE, ids=["x".join(map(str, r)) for r in BALANCE])
def test_balance(dmm, M, E, masked, dtype):
    say(f"moe_balance M={M} E={E} masked={masked} {dtype}")
    rng = np.random.default_rng(M * 3 + E)
    z = bf16_values((rng.standard_normal((M, E)) * 3).astype(np.float32))
    z[rng.random((M, E)) < 0.05] = -np.inf
    if M > 3:
        z[2] = -np.inf
        z[3] = -3e4
        z[3, 0] = 3e4
        z = bf16_values(z)
    mask = (rng.random(M) < 0.7).astype(np.uint8) if masked else None
    counts = rng.integers(0, 50, E).astype(np.int32)
    loss_ref, w, p = oracle.moe_balance(z, counts, mask)
    grad_ref = oracle.moe_balance_grad(z, counts, mask) * 0.75
    tol, gtol = balance_tolerances(z, w, p)
    zz = z.copy()
    if masked:
        zz[mask == 0] = np.nan                                      # whatever masked rows hold
    if dtype == torch.bfloat16:
        Z = bf16_of(zz, pad=3)
    else:
        Z = torch.full((M, E + 3), float("nan"), device=DEV)[:, :E]
        Z.copy_(dev(zz))
    Mk = None if mask is None else dev(mask)
    loss, weights = torch.full((1,), -1.0, device=DEV), torch.full((E,), -1.0, device=DEV)
    ws = torch.full((dmm.moe_balance_workspace_bytes(M, E),), 0x5A, dtype=torch.uint8, device=DEV)
    dmm.moe_balance(Z, dev(counts), loss, weights, token_mask=Mk, workspace=ws)
    assert np.allclose(host(weights), w, rtol=2.0 ** -23, atol=0)
    assert abs(host(loss)[0] - loss_ref) <= tol, (host(loss)[0], loss_ref, tol)
    whole, g = guarded(M * E, dtype)
    dmm.moe_balance_grad(Z, weights, torch.tensor([0.75], device=DEV), g.view(M, E), token_mask=Mk)
    got = host(g).reshape(M, E).astype(np.float64)
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    assert (np.abs(got - grad_ref) <= gtol + step * np.abs(grad_ref)).all()
    assert intact(whole)
    if masked:
        assert not got[mask == 0].any()


def test_balance_gradient_by_differences(dmm):
    """Central differences of the GPU's own loss: with h = 2^-6 the truncation is
    h^2 / 6 of the third derivative, at most p |w| 2 (below 3e-4 each of the
    largest weight), and the two losses' rounding is tol / h."""
    say("moe_balance differences")
    rng = np.random.default_rng(1)
    M, E, h = 4, 6, 2.0 ** -6
    z = np.round(rng.standard_normal((M, E)) * 64) / 64
    counts = dev(np.array([9, 0, 1, 2, 3, 1], np.int32))
    _, w, p = oracle.moe_balance(z, host(counts))
    tol, _ = balance_tolerances(z, w, p)
    loss, weights = torch.zeros(1, device=DEV), torch.zeros(E, device=DEV)
    ws = torch.zeros(dmm.moe_balance_workspace_bytes(M, E), dtype=torch.uint8, device=DEV)

    def f(a):
        dmm.moe_balance(dev(a.astype(np.float32)), counts, loss, weights, workspace=ws)
        return float(host(loss)[0])

    f(z)
    g = torch.zeros((M, E), device=DEV)
    dmm.moe_balance_grad(dev(z.astype(np.float32)), weights, torch.ones(1, device=DEV), g)
    g = host(g)
    for t in range(M):
        for e in range(E):
            up, dn = z.copy(), z.copy()
            up[t, e] += h
            dn[t, e] -= h
            assert abs((f(up) - f(dn)) / (2 * h) - g[t, e]) <= h * h / 6 * 2 * w.max() + tol / h


def test_balance_of_nothing(dmm):
    """No tokens, all masked, no slots: loss and gradients 0; a NaN logit of a
    token that takes part is not hidden."""
    say("moe_balance of nothing")
    ws = torch.zeros(64, dtype=torch.uint8, device=DEV)
    loss, w = torch.full((1,), 5.0, device=DEV), torch.full((4,), 5.0, device=DEV)
    one, zero = torch.ones(4, dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    for z, counts, mask in ((torch.zeros((0, 4), device=DEV), one, None),
                            (torch.full((3, 4), float("nan"), device=DEV), one,
                             torch.zeros(3, dtype=torch.uint8, device=DEV)),
                            (torch.zeros((3, 4), device=DEV), zero, None)):
        loss.fill_(5)
        dmm.moe_balance(z, counts, loss, w, token_mask=mask, workspace=ws)
        assert host(loss)[0] == 0 and not host(w).any()
        g = torch.full_like(z, 5.0)
        dmm.moe_balance_grad(z, w, torch.ones(1, device=DEV), g, token_mask=mask)
        assert not host(g).any()
    z = torch.zeros((3, 4), device=DEV)
    z[1, 2] = float("nan")
    dmm.moe_balance(z, one, loss, w, workspace=ws)
    assert np.isnan(host(loss)[0])


# ------------------------------------------------------------------- experts

# M, N, K, E, top_k, bias, busy: every slot of a third of the tokens goes to one expert
EXPERTS = [(1, 16, 32, 1, 1, False, False), (1, 50, 100, 8, 2, True, False), (16, 96, 512, 64, 8, False, False),
           (5, 33, 129, 4, 3, True, True), (40, 130, 320, 6, 2, True, True), (130, 64, 1000, 3, 2, False, True),
           (300, 270, 384, 5, 4, True, True), (600, 256, 160, 16, 2, False, False), (64, 20, 4128, 2, 1, False, False),
           (257, 257, 64, 2, 2, True, True)]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,E,top_k,bias,busy", EXPERTS, ids=["x".join(map(str, e[:5])) for e in EXPERTS])
def test_experts(dmm, M, N, K, E, top_k, bias, busy, out):
    say(f"mx_matmul_experts M={M} N={N} K={K} E={E} top_k={top_k} bias={bias} {out}")
    rng = np.random.default_rng(M + N + K)
    x = activations(rng, M, K)
    c, s = packed(rng, E * N, K)
    b = rng.standard_normal((E, N)).astype(np.float32) if bias else None
    ids = rng.integers(0, E, (M, top_k)).astype(np.int32)           # the same expert twice is possible
    if busy:
        ids[: M // 3] = E - 1
    ids[rng.random((M, top_k)) < 0.1] = -1
    w = oracle.mx_unpack(c, s, K).reshape(E, N, K)
    counts, offsets, order = route(dmm, ids, E)
    whole, y = guarded(M * top_k * N, out)
    dmm.mx_matmul_experts(bf16_of(x, 8), dev(c), dev(s), N, y, E, offsets, order, top_k,
                          bias=None if b is None else dev(b))
    got = host(y).reshape(M, top_k, N)
    assert intact(whole)
    assert np.isnan(got[ids < 0]).all()
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        ref, B = oracle.matmul_ref(workloads.bf16_bits(x)[t], w[e], None if b is None else b[e])
        assert_close(got[t, j], ref, B, K, out, f"expert {e}")


def test_experts_skip_bad_lists(dmm):
    """Offsets and slots out of range are skipped; rows listed nowhere stay as they were."""
    say("mx_matmul_experts with bad lists")
    M, N, K, E = 6, 40, 96, 3
    rng = np.random.default_rng(2)
    x = activations(rng, M, K)
    c, s = packed(rng, E * N, K)
    w = oracle.mx_unpack(c, s, K).reshape(E, N, K)
    order = np.array([0, -5, 1, 6, 1 << 30, 2], np.int32)
    offsets = np.array([-3, 2, 4, 900], np.int32)                   # 0: slots 0, -5; 1: 1, 6; 2: 2^30, 2
    whole, y = guarded(M * N, torch.float32)
    y.fill_(3.0)
    dmm.mx_matmul_experts(bf16_of(x), dev(c), dev(s), N, y, E, dev(offsets), dev(order), 1)
    got = host(y).reshape(M, N)
    for t, e in ((0, 0), (1, 1), (2, 2)):
        ref, B = oracle.matmul_ref(workloads.bf16_bits(x)[t:t + 1], w[e])
        assert_close(got[t:t + 1], ref, B, K, torch.float32, f"slot {t}")
    assert (got[3:] == 3).all() and intact(whole)


@pytest.mark.parametrize("M,K", [(60, 96), (200, 40), (200, 320)])
def test_tiled_experts_skip_bad_lists(dmm, M, K):
    """The same with enough slots for the tiles."""
    say(f"mx_matmul_experts with bad lists M={M} K={K}")
    N, E = 140, 3
    rng = np.random.default_rng(M + K)
    x = activations(rng, M, K)
    c, s = packed(rng, E * N, K)
    w = oracle.mx_unpack(c, s, K).reshape(E, N, K)
    order = rng.permutation(M).astype(np.int32)
    bad = rng.random(M) < 0.2
    order[bad] = rng.choice(np.array([-1, -7, M, M + 1, 2**31 - 1, -2**31], np.int64), bad.sum()).astype(np.int32)
    offsets = np.array([-3, M // 2, M // 2 + 9, 2 * M], np.int32)
    whole, y = guarded(M * N, torch.float32)
    y.fill_(3.0)
    dmm.mx_matmul_experts(bf16_of(x), dev(c), dev(s), N, y, E, dev(offsets), dev(order), 1)
    got = host(y).reshape(M, N)
    for e, at in enumerate((np.arange(M // 2), np.arange(M // 2, M // 2 + 9), np.arange(M // 2 + 9, M))):
        t = order[at[~bad[at]]]
        ref, B = oracle.matmul_ref(workloads.bf16_bits(x)[t], w[e])
        assert_close(got[t], ref, B, K, torch.float32, f"expert {e}")
    left = np.ones(M, bool)
    left[order[~bad]] = False
    assert (got[left] == 3).all() and intact(whole)


@pytest.mark.parametrize("M,E,valid", [(300, 5, 0), (512, 1, 448), (512, 1, 512), (700, 3, 1), (90, 2, 64)])
def test_padded_batches(dmm, M, E, valid):
    """Batches whose tail (or all) is padding: its rows are NaN, the others right."""
    say(f"padded batch M={M} E={E} valid={valid}")
    N, K = 520, 64
    rng = np.random.default_rng(M + valid)
    x = activations(rng, M, K)
    c, s = packed(rng, E * N, K)
    w = oracle.mx_unpack(c, s, K).reshape(E, N, K)
    ids = rng.integers(0, E, (M, 1)).astype(np.int32)
    ids[valid:] = -1
    counts, offsets, order = route(dmm, ids, E)
    whole, y = guarded(M * N, torch.bfloat16)
    dmm.mx_matmul_experts(bf16_of(x), dev(c), dev(s), N, y, E, offsets, order, 1)
    got = host(y).reshape(M, N)
    assert intact(whole) and np.isnan(got[valid:]).all()
    for e in range(E):
        t = np.nonzero(ids[:, 0] == e)[0]
        if len(t):
            ref, B = oracle.matmul_ref(workloads.bf16_bits(x)[t], w[e])
            assert_close(got[t], ref, B, K, torch.bfloat16, f"expert {e}")


def test_layer_together(dmm):
    """A whole expert layer: routing, balance loss and gradient, both of the
    experts' products (the second with activations of its own for each slot)
    and a shared expert on MXFP4 activations, eagerly and replayed."""
    say("expert layer")
    rng = np.random.default_rng(9)
    M, K, N, E, top_k = 33, 256, 160, 8, 2
    c1, s1 = packed(rng, E * N, K, spread=1)
    c2, s2 = packed(rng, E * K, N, spread=1)
    c3, s3 = packed(rng, N, K, spread=1)
    D = [dev(a) for a in (c1, s1, c2, s2, c3, s3)]
    X = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    Z = torch.zeros((M, E), device=DEV)
    ids = torch.zeros((M, top_k), dtype=torch.int32, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    counts, offsets, order = torch.zeros(E, **i32), torch.zeros(E + 1, **i32), torch.zeros(M * top_k, **i32)
    loss, weights, g = torch.zeros(1, device=DEV), torch.zeros(E, device=DEV), torch.zeros((M, E), device=DEV)
    one = torch.ones(1, device=DEV)
    up = torch.zeros((M, top_k, N), dtype=torch.bfloat16, device=DEV)
    down = torch.zeros((M, top_k, K), device=DEV)
    shared = torch.zeros((M, N), device=DEV)
    xc, xs = (torch.zeros(sh, dtype=torch.uint8, device=DEV) for sh in dmm.mx_shape(M, K))
    ws = torch.zeros(dmm.moe_balance_workspace_bytes(M, E), dtype=torch.uint8, device=DEV)
    outs = (counts, offsets, order, loss, g, up, down, shared)

    def step():
        dmm.moe_route(ids, E, counts, offsets, order)
        dmm.moe_balance(Z, counts, loss, weights, workspace=ws)
        dmm.moe_balance_grad(Z, weights, one, g)
        dmm.mx_matmul_experts(X, D[0], D[1], N, up, E, offsets, order, top_k)
        dmm.mx_matmul_experts(up.view(M * top_k, N), D[2], D[3], K, down, E, offsets, order, 1)
        dmm.mx_pack(X, xc, xs)
        dmm.mx_matmul_mx(xc, xs, M, K, D[4], D[5], N, shared)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        x = activations(rng, M, K)
        z = rng.standard_normal((M, E)).astype(np.float32)
        chosen = np.argsort(-z, axis=1)[:, :top_k].astype(np.int32)
        X.copy_(bf16_of(x))
        Z.copy_(dev(z))
        ids.copy_(dev(chosen))
        step()
        eager = [host(t.clone()) for t in outs]
        for t in outs:
            t.zero_()
        graph.replay()
        for t, e in zip(outs, eager):
            assert np.array_equal(host(t), e)
        for a, r in zip(eager, oracle.moe_route(chosen, E)):
            assert np.array_equal(a, r)
        l, w, p = oracle.moe_balance(z, eager[0])
        tol, gtol = balance_tolerances(z, w, p)
        ref = oracle.moe_balance_grad(z, eager[0])
        assert abs(eager[3][0] - l) <= tol and (np.abs(eager[4] - ref) <= gtol + 2.0 ** -24 * np.abs(ref)).all()
        w1, w2 = oracle.mx_unpack(c1, s1, K).reshape(E, N, K), oracle.mx_unpack(c2, s2, N).reshape(E, K, N)
        for t in range(M):
            for j in range(top_k):
                e = chosen[t, j]
                r, B = oracle.matmul_ref(workloads.bf16_bits(x[t:t + 1]), w1[e])
                assert_close(eager[5][t, j][None], r, B, K, torch.bfloat16, "up")
                r, B = oracle.matmul_ref(workloads.bf16_bits(eager[5][t, j][None]), w2[e])
                assert_close(eager[6][t, j][None], r, B, N, torch.float32, "down")
        xq = oracle.mx_unpack(*oracle.mx_pack(x)[:2], K)
        w3 = oracle.mx_unpack(c3, s3, K)
        assert_close(eager[7], xq @ w3.T, np.abs(xq) @ np.abs(w3).T, K, torch.float32, "shared")


@pytest.mark.parametrize("E", [2, 3, 64, 100, 512])
@pytest.mark.parametrize("gap", [0, 4, 8, 12, 14, 16, 18, 20, 24])
def test_gradient_of_confident_tokens(dmm, E, gap):
    """A token whose top logit leads by `gap`: w_e - s is then small against w and
    s themselves.  With the terms centred, d_j = w_j - s for the computed s = s* + h,
    |h| <= rel s*, and the result p_e (d_e - sum_j p_j d_j), h drops out but for
    its product with the error of p: off by at most 2 rel p_e (D_e + sum_j p_j D_j
    + 2 rel s*), D_j = |w_j - s*|, with rel = (d + 32) 2^-23 of a probability."""
    say(f"moe_balance_grad of confident tokens E={E} gap={gap}")
    rng = np.random.default_rng(E + gap)
    M = 96
    z = bf16_values(rng.standard_normal((M, E)).astype(np.float32))
    top = rng.integers(0, E, M)
    z[np.arange(M), top] = z.max(axis=1) + gap
    z = bf16_values(z)
    w = (rng.integers(0, 60, E) / 97.0).astype(np.float32)
    p = np.exp(z.astype(np.float64) - z.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    s = (p * w).sum(axis=1, keepdims=True)
    D = np.abs(w - s)
    # w - s itself cancels in 64 bits too late to matter: 2^-53 against 1e-9
    ref = p * (w - s)
    rel = ((z.max(axis=1) - z.min(axis=1) + 32) * 2.0 ** -23)[:, None]
    tol = 2 * rel * p * (D + (p * D).sum(axis=1, keepdims=True) + 2 * rel * s)
    for dtype, step in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)):
        Z = dev(z) if dtype == torch.float32 else bf16_of(z)
        g = torch.empty((M, E), dtype=dtype, device=DEV)
        dmm.moe_balance_grad(Z, dev(w), torch.ones(1, device=DEV), g)
        off = np.abs(host(g).astype(np.float64) - ref)
        assert (off <= tol + step * np.abs(ref)).all(), (off / (tol + step * np.abs(ref))).max()
