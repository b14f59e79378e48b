"""MXFP4 products at the borders of the format: codes behind the last column,
and the smallest and largest scales."""

import numpy as np
import pytest

import oracle
from test_gpu_mx import DEV, bf16_of, dev, dmm, guarded, host, intact, packed, say  # noqa: F401  (dmm: fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def cut_blocks(rng, rows, K, scale):
    """A package whose last, cut block has this scale byte, the largest codes
    behind K and at most 1.5 before it; and the same with zeros behind K."""
    nb = -(-K // 32)
    c = rng.integers(0, 16, (rows, nb * 32)).astype(np.uint8)
    c[:, (nb - 1) * 32:K] &= 0xB                                    # finite with scale byte 254 too
    s = (127 + rng.integers(-3, 4, (rows, nb))).astype(np.uint8)
    s[:, -1] = scale
    c[:, K:] = 7 + 8 * rng.integers(0, 2, c[:, K:].shape)
    zero = c.copy()
    zero[:, K:] = 0
    join = lambda a: a.reshape(rows, nb, 32)[..., 0::2] | (a.reshape(rows, nb, 32)[..., 1::2] << 4)
    return join(c), join(zero), s


# tokens and rows of W: every streaming form's and every tile's way of cutting the last block
CUT = [(1, 33), (3, 40), (7, 40), (16, 70), (40, 100), (130, 2100), (500, 4100), (700, 4300), (1030, 12500)]
CUTS = [(M, N, K, scale) for M, N in CUT for K in (1, 31, 45, 497, 1100) for scale in (130, 253, 254)
        if M <= 40 or (scale > 130 and K not in (1, 31))]


@pytest.mark.parametrize("M,N,K,scale", CUTS, ids=["x".join(map(str, c)) for c in CUTS])
def test_codes_past_the_last_column(dmm, M, N, K, scale):
    """They take no part, whatever they and their scale stand for: the bits are
    those with zeros in their place, and finite."""
    say(f"codes past K: M={M} N={N} K={K} scale={scale}")
    rng = np.random.default_rng(M + N + K + scale)
    c, zero, s = cut_blocks(rng, N, K, scale)
    x = (rng.integers(-4, 5, (M, K)) * 2.0 ** -20).astype(np.float32)
    y, z = torch.empty((2, M, N), device=DEV)
    dmm.mx_matmul(bf16_of(x), dev(c), dev(s), N, y)
    dmm.mx_matmul(bf16_of(x), dev(zero), dev(s), N, z)
    assert np.isfinite(host(y)).all() and torch.equal(y, z)
    # with both operands packed, one of them has zeros there
    xc, xz, xs = cut_blocks(rng, M, K, scale)
    s[:, -1] = 100
    xq = torch.empty((2, M, N), device=DEV)
    dmm.mx_matmul_mx(dev(xc), dev(xs), M, K, dev(zero), dev(s), N, xq[0])
    dmm.mx_matmul_mx(dev(xz), dev(xs), M, K, dev(c), dev(s), N, xq[1])
    assert np.isfinite(host(xq)).all() and torch.equal(xq[0], xq[1])


@pytest.mark.parametrize("M,K", [(3, 45), (3, 497), (40, 45), (40, 1003), (300, 331)])
def test_experts_codes_past_the_last_column(dmm, M, K):
    say(f"experts' codes past K: M={M} K={K}")
    N, E = 300, 3
    rng = np.random.default_rng(M + K)
    c, zero, s = cut_blocks(rng, E * N, K, 254)
    x = (rng.integers(-4, 5, (M, K)) * 2.0 ** -20).astype(np.float32)
    ids = dev(rng.integers(0, E, (M, 1)).astype(np.int32))
    counts, offsets, order = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (E, E + 1, M))
    dmm.moe_route(ids, E, counts, offsets, order)
    y, z = torch.empty((2, M, N), device=DEV)
    dmm.mx_matmul_experts(bf16_of(x), dev(c), dev(s), N, y, E, offsets, order, 1)
    dmm.mx_matmul_experts(bf16_of(x), dev(zero), dev(s), N, z, E, offsets, order, 1)
    assert np.isfinite(host(y)).all() and torch.equal(y, z)


@pytest.mark.parametrize("M,N", [(1, 37), (7, 60), (20, 37), (300, 4100), (700, 4300)])
def test_smallest_scales(dmm, M, N):
    """Weights down to 2^-128, most of them subnormal in bf16: x = 2^k e_j reads
    each exactly, as a normal fp32 value for k = 40 and a subnormal one for k = 0."""
    say(f"smallest scales M={M} N={N}")
    K = 320
    rng = np.random.default_rng(M)
    c, _ = packed(rng, N, K)
    s = rng.integers(0, 4, (N, K // 32)).astype(np.uint8)
    w = oracle.mx_unpack(c, s, K)
    ks = rng.integers(0, K, M)
    for k in (40, 0):
        x = np.zeros((M, K), np.float32)
        x[np.arange(M), ks] = 2.0 ** k
        ref = (w[:, ks].T * 2.0 ** k).astype(np.float32)
        y = torch.empty((M, N), device=DEV)
        dmm.mx_matmul(bf16_of(x), dev(c), dev(s), N, y)
        assert np.array_equal(host(y), ref), f"bf16, k = {k}"
        xc, xs, _ = oracle.mx_pack(x)
        dmm.mx_matmul_mx(dev(xc), dev(xs), M, K, dev(c), dev(s), N, y)
        assert np.array_equal(host(y), ref), f"MXFP4, k = {k}"


def test_call_on_the_current_stream(dmm):
    say("stream handles")
    side = torch.cuda.Stream()
    for stream in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(stream):
            assert dmm._raw_stream(0) == torch.cuda.current_stream(0).cuda_stream == stream.cuda_stream
