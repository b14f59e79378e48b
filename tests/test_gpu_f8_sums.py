"""A bf16 y of the e4m3 products is the fp32 y rounded, however many tokens there are; short_sums, which
the caller asks for, is the e4m3 matrix instruction with its own bound D (tests/test_gpu_f8.py)."""

import numpy as np
import pytest

import oracle
from test_gpu_f8 import EXPERTS, MATMUL, assert_close, dropped, random_package
from test_gpu_f8_forms import FORMS, LISTS, LONG_LISTS
from test_gpu_mx import DEV, dev, guarded, host, intact, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def dmm():
    import decode_matmul_amd
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return decode_matmul_amd


# with sums that round: every form of many tokens
ROUNDING = [(16, 256, 512), (17, 130, 384), (33, 64, 2048), (100, 257, 129), (128, 128, 4096), (40, 8300, 200),
            (600, 700, 1111), (930, 930, 4096), (1500, 2100, 700), (4100, 2990, 256), (4096, 3104, 640)]


@pytest.mark.parametrize("M,N,K", ROUNDING, ids=["x".join(map(str, f)) for f in ROUNDING])
def test_bf16_is_fp32_rounded(dmm, M, N, K):
    say(f"f8_matmul bf16 y is the fp32 y rounded M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K)
    xc, xs, _ = random_package(rng, M, K, 1)
    wc, ws, _ = random_package(rng, N, K, 128)
    a = (dev(xc), dev(xs), M, K, dev(wc), dev(ws), N)
    bias = dev(rng.standard_normal(N).astype(np.float32))
    y, z = torch.empty((M, N), device=DEV), torch.empty((M, N), dtype=BF16, device=DEV)
    dmm.f8_matmul(*a, y, bias=bias)
    dmm.f8_matmul(*a, z, bias=bias)
    assert torch.equal(y.to(BF16), z)


def experts_call(dmm, rng, M, N, K, E, top_k, exact):
    xc, xs, x = random_package(rng, M, K, 1, exact=exact)
    made = [random_package(rng, N, K, 128, exact=exact) for _ in range(E)]
    ids = np.minimum((rng.random((M, top_k)) ** 2 * (E + 0.5)).astype(np.int32), E)         # E: of no expert
    _, offsets, order = oracle.moe_route(ids, E)
    wc, ws = dev(np.stack([m[0] for m in made])), dev(np.stack([m[1] for m in made]))

    def call(y, **kw):
        dmm.f8_matmul_experts(dev(xc), dev(xs), M, K, wc, ws, N, y, E, dev(offsets), dev(order), top_k, **kw)

    return call, ids, x, [m[2] for m in made]


@pytest.mark.parametrize("M,N,K,E,top_k", LISTS, ids=["x".join(map(str, f)) for f in LISTS])
def test_bf16_of_the_experts_is_fp32_rounded(dmm, M, N, K, E, top_k):
    say(f"f8_matmul_experts bf16 y is the fp32 y rounded M={M} N={N} K={K} E={E} top_k={top_k}")
    call, ids, _, _ = experts_call(dmm, np.random.default_rng(M + N + K), M, N, K, E, top_k, False)
    y, z = (torch.empty((M, top_k, N), dtype=t, device=DEV) for t in (torch.float32, BF16))
    call(y)
    call(z)
    on = dev((ids < E).astype(np.uint8)).bool()
    assert torch.equal(y.to(BF16)[on], z[on]) and z[~on].isnan().all()


# ------------------------------------------------------------- short sums


@pytest.mark.parametrize("M,N,K", FORMS, ids=["x".join(map(str, f)) for f in FORMS])
def test_short_sums_of_whole_numbers(dmm, M, N, K):
    """Whole numbers up to 4 times scales 1 and 2: products are whole and at most 64, so nothing lies 13 bits
    below the largest of eight, and sums below 2^24 are exact."""
    say(f"f8_matmul short sums, exact M={M} N={N} K={K}")
    rng = np.random.default_rng(M + 2 * N + 3 * K)
    xc, xs, x = random_package(rng, M, K, 1, exact=True)
    wc, ws, w = random_package(rng, N, K, 128, exact=True)
    bias = rng.integers(-9, 10, N).astype(np.float32)
    ref = torch.from_numpy((x @ w.T + bias).astype(np.float32)).to(BF16).float().numpy()
    whole, y = guarded(M * N, BF16)
    dmm.f8_matmul(dev(xc), dev(xs), M, K, dev(wc), dev(ws), N, y, bias=dev(bias), short_sums=True)
    assert np.array_equal(host(y).reshape(M, N), ref) and intact(whole)


@pytest.mark.parametrize("M,N,K", MATMUL, ids=["x".join(map(str, m)) for m in MATMUL])
def test_short_sums_within_their_bound(dmm, M, N, K):
    """The fp32 bound, D beside it for more than 16 tokens, and the same bits twice."""
    say(f"f8_matmul short sums M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K)
    xc, xs, x = random_package(rng, M, K, 1)
    wc, ws, w = random_package(rng, N, K, 128)
    a = (dev(xc), dev(xs), M, K, dev(wc), dev(ws), N)
    whole, y = guarded(M * N, BF16)
    dmm.f8_matmul(*a, y, short_sums=True)
    ref, B = oracle.f8_matmul(x, w)
    assert_close(host(y).reshape(M, N), ref, B, K, BF16, "y", dropped(x, w) * (1 + 2.0 ** -8) if M > 16 else 0)
    again = torch.empty_like(y)
    dmm.f8_matmul(*a, again, short_sums=True)
    assert torch.equal(again, y) and intact(whole)


@pytest.mark.parametrize("M,N,K,E,top_k", LISTS + LONG_LISTS, ids=["x".join(map(str, f)) for f in LISTS + LONG_LISTS])
def test_short_sums_of_lists(dmm, M, N, K, E, top_k):
    say(f"f8_matmul_experts short sums, exact M={M} N={N} K={K} E={E} top_k={top_k}")
    call, ids, x, ws = experts_call(dmm, np.random.default_rng(M + N + K), M, N, K, E, top_k, True)
    whole, y = guarded(M * top_k * N, BF16)
    call(y, short_sums=True)
    got = host(y).reshape(M, top_k, N)
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if len(t):
            ref = torch.from_numpy((x[t] @ ws[e].T).astype(np.float32)).to(BF16).float().numpy()
            assert np.array_equal(got[t, j], ref), f"expert {e}"
    assert np.isnan(got[ids == E]).all() and intact(whole)


@pytest.mark.parametrize("M,N,K,E,top_k,bias,busy", EXPERTS, ids=["x".join(map(str, e[:5])) for e in EXPERTS])
def test_short_sums_of_the_experts_within_their_bound(dmm, M, N, K, E, top_k, bias, busy):
    say(f"f8_matmul_experts short sums M={M} N={N} K={K} E={E} top_k={top_k}")
    call, ids, x, ws = experts_call(dmm, np.random.default_rng(M + N + K), M, N, K, E, top_k, False)
    y = torch.empty((M, top_k, N), dtype=BF16, device=DEV)
    call(y, short_sums=True)
    got = host(y)
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if len(t):
            ref, B = oracle.f8_matmul(x[t], ws[e])
            D = dropped(x[t], ws[e]) * (1 + 2.0 ** -8) if M * top_k >= 8 * E else 0
            assert_close(got[t, j], ref, B, K, BF16, f"expert {e}", D)


def test_short_sums_of_any_alignment(dmm):
    """y at an address of its type only, and rows that are no whole pieces."""
    say("f8_matmul short sums, y of any alignment")
    rng = np.random.default_rng(0)
    for M, N, K in ((50, 72, 300), (900, 904, 130), (1500, 2104, 130), (4100, 2992, 130)):
        xc, xs, x = random_package(rng, M, K, 1, exact=True)
        wc, ws, w = random_package(rng, N, K, 128, exact=True)
        ref = torch.from_numpy((x @ w.T).astype(np.float32)).to(BF16).float().numpy()
        y = torch.full((M * N + 9,), 7.0, dtype=BF16, device=DEV)
        dmm.f8_matmul(dev(xc), dev(xs), M, K, dev(wc), dev(ws), N, y[1:1 + M * N], short_sums=True)
        got = host(y)
        assert np.array_equal(got[1:1 + M * N].reshape(M, N), ref) and got[0] == 7 and (got[1 + M * N:] == 7).all()


def test_short_sums_keep_nan_and_nothing(dmm):
    """K = 0 leaves the bias; a NaN code or scale takes its row or column."""
    say("f8_matmul short sums of nothing and NaN")
    M, N, K = 300, 200, 300
    rng = np.random.default_rng(1)
    bias = rng.standard_normal(N).astype(np.float32)
    y = torch.full((M, N), 7.0, dtype=BF16, device=DEV)
    e, f = torch.empty(0, dtype=torch.uint8, device=DEV), torch.empty(0, device=DEV)
    dmm.f8_matmul(e, f, M, 0, e, f, N, y, bias=dev(bias), short_sums=True)
    assert torch.equal(y, dev(bias).to(BF16).expand(M, N))
    xc, xs, _ = random_package(rng, M, K, 1)
    wc, ws, _ = random_package(rng, N, K, 128)
    wc[7, 1, 3], ws[1, 2], xs[5, 0] = 0xff, np.nan, np.nan
    dmm.f8_matmul(dev(xc), dev(xs), M, K, dev(wc), dev(ws), N, y, short_sums=True)
    bad = np.zeros((M, N), bool)
    bad[:, 7], bad[:, 128:], bad[5] = True, True, True
    assert np.array_equal(np.isnan(host(y)), bad)


@pytest.mark.parametrize("short_sums", [False, True], ids=["fp32 sums", "short sums"])
def test_captured_and_on_two_streams(dmm, short_sums):
    """Products of both kinds captured once and replayed on other inputs, while another stream multiplies
    too: the bits of an eager pass."""
    say(f"f8 products captured, short_sums={short_sums}")
    rng = np.random.default_rng(3)
    M, N, K, E, top_k = 300, 520, 900, 4, 2
    cs, ss = dmm.f8_shape(M, K)
    xc, xs = torch.empty(cs, dtype=torch.uint8, device=DEV), torch.empty(ss, device=DEV)
    made = [random_package(rng, N, K, 128) for _ in range(E)]
    wc, ws = dev(np.stack([m[0] for m in made])), dev(np.stack([m[1] for m in made]))
    _, offsets, order = (dev(v) for v in oracle.moe_route(rng.integers(0, E, (M, top_k)).astype(np.int32), E))

    def products(y, rows):
        dmm.f8_matmul(xc, xs, M, K, wc[0], ws[0], N, y, short_sums=short_sums)
        dmm.f8_matmul_experts(xc, xs, M, K, wc, ws, N, rows, E, offsets, order, top_k, short_sums=short_sums)

    def results():
        return torch.zeros((M, N), dtype=BF16, device=DEV), torch.zeros((M, top_k, N), dtype=BF16, device=DEV)

    captured, eager, beside = results(), results(), results()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    dmm.f8_pack(torch.randn((M, K), device=DEV), xc, xs)
    torch.cuda.synchronize()
    with torch.cuda.stream(one):
        products(*captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=one):
        products(*captured)
    for i in range(4):
        dmm.f8_pack(torch.randn((M, K), device=DEV), xc, xs)
        products(*eager)
        torch.cuda.synchronize()
        with torch.cuda.stream(one):
            graph.replay()
        with torch.cuda.stream(two):
            products(*beside)
        torch.cuda.synchronize()
        for got in (captured, beside):
            assert all(torch.equal(a, b) for a, b in zip(got, eager)), i
