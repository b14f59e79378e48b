"""MXFP4 quantization and products on the GPU against the float64 oracle.

Quantization and decoding match bit for bit.  For products the operands are
exact and each is exact in fp32, so only the K additions round: an addition
(of a matrix instruction that truncates as well) is off by at most 2^-23 of
the largest partial sum, itself at most B = sum |x w_hat| + |bias|, and a few
more join the waves' sums and the bias:
    |y - y_ref| <= (K + 16) 2^-23 B   (+ 2^-8 |y| for the rounding to bf16).
Where every product is a whole multiple of one unit and sums stay below 2^24
of it, no addition rounds and the results are equal.
"""

import numpy as np
import pytest

import oracle
import workloads

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def say(msg):
    print(f"[case] {msg}", flush=True)


@pytest.fixture(scope="module")
def dmm():
    import decode_matmul_amd
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return decode_matmul_amd


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def bf16_of(a, pad=0, fill=np.nan):
    """Device bf16 [M, K] holding a (fp32 values exact in bf16), its rows K + pad
    apart with `fill` between them."""
    M, K = a.shape
    w = np.full((M, K + pad), fill, np.float32)
    w[:, :K] = a
    return dev(workloads.bf16_bits(w).view(np.int16)).view(torch.bfloat16)[:, :K]


def bf16_values(a):
    return oracle.bf16_bits_to_f64(workloads.bf16_bits(a)).astype(np.float32)


def packed(rng, rows, K, spread=3):
    """A random package: scales 2^-spread .. 2^spread around 1, padding codes 0."""
    nb = -(-K // 32)
    c = rng.integers(0, 16, (rows, nb * 32)).astype(np.uint8)
    c[:, K:] = 0
    s = (127 + rng.integers(-spread, spread + 1, (rows, nb))).astype(np.uint8)
    c = c.reshape(rows, nb, 32)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


def guarded(n, dtype):
    """A buffer of n elements within a larger one, to see writes past its ends."""
    whole = torch.full((n + 512,), 7.0, dtype=dtype, device=DEV)
    return whole, whole[256:256 + n]


def intact(whole):
    w = host(whole)
    return (w[:256] == 7).all() and (w[-256:] == 7).all()


def assert_close(y, ref, B, K, dtype, what):
    tol = (K + 16) * 2.0 ** -23 * B + (2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 0)
    off = np.abs(y.astype(np.float64) - ref)
    assert (off <= tol).all(), f"{what}: off by {(off / np.maximum(tol, 1e-300)).max():.3g} of the tolerance"


# ------------------------------------------------------------------ quantize

PACK = [(1, 1), (1, 32), (3, 31), (5, 33), (2, 64), (257, 100), (16, 4096), (129, 1000), (1, 100000), (300, 7)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,K", PACK)
def test_pack_and_unpack_are_exact(dmm, rows, K, dtype):
    say(f"mx_pack {rows}x{K} {dtype}")
    rng = np.random.default_rng(rows * 1000 + K)
    w = (rng.standard_normal((rows, K)) * 10.0 ** rng.uniform(-6, 6, (rows, 1))).astype(np.float32)
    w[:, ::7] = np.round(w[:, ::7])
    if rows > 2:
        w[1] = 0
        w[2, :] = rng.integers(-12, 13, K) * 0.25                   # ties
    if dtype == torch.bfloat16:
        w = bf16_values(w)
        W = bf16_of(w, pad=5)
    else:
        W = torch.full((rows, K + 3), float("nan"), device=DEV)[:, :K]
        W.copy_(dev(w))
    cs, ss = dmm.mx_shape(rows, K)
    codes = torch.full(cs, 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full(ss, 0xA5, dtype=torch.uint8, device=DEV)
    st = torch.full((1,), 99, dtype=torch.int32, device=DEV)
    dmm.mx_pack(W, codes, scales, status=st)
    c, s, fine = oracle.mx_pack(w)
    assert fine and int(host(st)[0]) == 0
    assert np.array_equal(host(scales), s) and np.array_equal(host(codes), c)
    for out in (torch.float32, torch.bfloat16):
        whole, y = guarded(rows * K, out)
        dmm.mx_unpack(codes, scales, rows, K, y, status=st)
        assert np.array_equal(host(y).reshape(rows, K), oracle.mx_unpack(c, s, K).astype(np.float32))
        assert intact(whole) and int(host(st)[0]) == 0


def test_pack_of_extreme_blocks(dmm):
    """Zeros of both signs, subnormals, the largest values, each scale's border;
    then blocks that are not finite."""
    say("mx_pack extreme blocks")
    rng = np.random.default_rng(0)
    w = np.zeros((300, 64), np.float32)
    w[1, 3] = -0.0
    w[2, :32] = 2.0 ** -149
    w[3, 1] = -(2.0 ** -126)
    w[4, :] = np.finfo(np.float32).max
    w[5, :2] = [6.99, 7.0]
    for i in range(6, 260):                                         # each binade, just below and at its border
        top = np.float32(2.0) ** np.float32(i - 132)
        w[i, :32] = rng.uniform(-1, 1, 32).astype(np.float32) * top
        w[i, 5] = np.nextafter(top, np.float32(0))
        w[i, 32:] = rng.uniform(-1, 1, 32).astype(np.float32) * top
        w[i, 40] = top
    w = np.where(np.isfinite(w), w, 0).astype(np.float32)
    W = dev(w)
    cs, ss = dmm.mx_shape(300, 64)
    codes, scales = torch.empty(cs, dtype=torch.uint8, device=DEV), torch.empty(ss, dtype=torch.uint8, device=DEV)
    dmm.mx_pack(W, codes, scales)
    c, s, _ = oracle.mx_pack(w)
    assert np.array_equal(host(scales), s) and np.array_equal(host(codes), c)
    for bad in (np.nan, np.inf, -np.inf):
        w[270, 33] = bad
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        dmm.mx_pack(dev(w), codes, scales, status=st)
        c, s, fine = oracle.mx_pack(w)
        assert not fine and int(host(st)[0]) == dmm.TQ_DATA_RANGE
        assert np.array_equal(host(scales), s) and np.array_equal(host(codes), c)
        y = torch.empty((300, 64), device=DEV)
        dmm.mx_unpack(codes, scales, 300, 64, y, status=st)
        assert int(host(st)[0]) == dmm.TQ_DATA_RANGE
        got = host(y)
        assert np.isnan(got[270, 32:]).all() and np.isfinite(np.delete(got, 270, 0)).all()


def test_unpack_of_every_scale_and_padding(dmm):
    say("mx_unpack every scale")
    c = np.tile(np.arange(16, dtype=np.uint8) * 17, (256, 1, 1))
    s = np.arange(256, dtype=np.uint8).reshape(256, 1)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    with np.errstate(over="ignore"):
        ref = oracle.mx_unpack(c, s, 32).astype(np.float32)
    for out in (torch.float32, torch.bfloat16):
        y = torch.empty((256, 32), dtype=out, device=DEV)
        dmm.mx_unpack(dev(c), dev(s), 256, 32, y, status=st)
        assert np.array_equal(host(y), ref, equal_nan=True)
        assert int(host(st)[0]) == dmm.TQ_DATA_RANGE
    for K, at, flag in ((31, 15, True), (31, 14, False), (9, 4, True), (1, 0, True), (24, 12, True), (24, 11, False)):
        c = np.zeros((2, 1, 16), np.uint8)
        c[1, 0, at] = 0x10                                          # the byte's second code
        y = torch.empty((2, K), device=DEV)
        dmm.mx_unpack(dev(c), dev(np.full((2, 1), 127, np.uint8)), 2, K, y, status=st)
        assert int(host(st)[0]) == (dmm.TQ_DATA_PADDING if flag else 0), (K, at)


# ------------------------------------------------------------------ products

# M, N, K, gap between x's rows, bias
SHAPES = [
    (1, 1, 1, 0, False), (1, 16, 32, 0, True), (1, 17, 33, 0, False), (2, 15, 31, 1, True), (1, 64, 4096, 0, False),
    (3, 100, 127, 0, True), (4, 48, 128, 8, False), (5, 33, 129, 3, True), (16, 80, 512, 0, False),
    (17, 16, 96, 0, True), (16, 130, 1056, 16, False), (31, 257, 160, 0, True), (33, 64, 1000, 24, False),
    (64, 100, 256, 0, True), (65, 300, 1023, 1, False), (127, 129, 320, 0, True), (128, 256, 512, 8, False),
    (129, 513, 2048, 0, True), (200, 77, 4100, 4, False), (255, 256, 64, 0, False), (257, 511, 384, 0, True),
    (300, 1001, 1000, 24, True), (513, 260, 1184, 0, False), (1, 7, 9000, 0, True),
    # enough tiles for the larger ones
    (700, 4300, 330, 0, True), (650, 4404, 1155, 3, False), (1030, 12500, 264, 0, True), (1027, 12403, 577, 1, False),
    # more than a few tokens of short rows
    (40, 50, 1, 0, True), (70, 300, 31, 1, False), (130, 260, 63, 0, True), (300, 257, 255, 0, False),
    (64, 128, 225, 7, True), (650, 4404, 130, 6, False), (1030, 12500, 200, 0, True), (1030, 12500, 64, 0, False),
    # small tiles dealt over K to groups of waves, several rounds of them and what is left
    (20, 4000, 6000, 0, True), (129, 2100, 2600, 3, False), (40, 7000, 1500, 8, True), (64, 512, 8192, 0, False),
    (300, 1000, 2048, 1, True),
]
IDS = ["x".join(map(str, s[:3])) for s in SHAPES]


def activations(rng, M, K):
    x = bf16_values(rng.standard_normal((M, K)).astype(np.float32))
    x[rng.random((M, K)) < 0.01] *= 64
    return x


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,pad,bias", SHAPES, ids=IDS)
def test_matmul(dmm, M, N, K, pad, bias, out):
    say(f"mx_matmul M={M} N={N} K={K} pad={pad} bias={bias} {out}")
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    x = activations(rng, M, K)
    c, s = packed(rng, N, K)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    ref, B = oracle.matmul_ref(workloads.bf16_bits(x), oracle.mx_unpack(c, s, K), b)
    if K % 32:                                                      # codes past K take no part
        q = c.reshape(N, -1)
        q[:, (K + 1) // 2:] |= 0xE7 if (K + 1) // 2 < q.shape[1] else 0
        q[:, (K % 32 and K - 1) // 2 + 0] |= 0x70 if K % 2 else 0
        c = q.reshape(c.shape)
    whole, y = guarded(M * N, out)
    dmm.mx_matmul(bf16_of(x, pad), dev(c), dev(s), N, y, bias=None if b is None else dev(b))
    assert_close(host(y).reshape(M, N), ref, B, K, out, f"{M}x{N}x{K}")
    assert intact(whole)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,pad,bias", SHAPES, ids=IDS)
def test_matmul_mx(dmm, M, N, K, pad, bias, out):
    say(f"mx_matmul_mx M={M} N={N} K={K} bias={bias} {out}")
    rng = np.random.default_rng(M * 5 + N + K)
    xc, xs = packed(rng, M, K)
    c, s = packed(rng, N, K)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    x, w = oracle.mx_unpack(xc, xs, K), oracle.mx_unpack(c, s, K)
    ref, B = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias:
        ref, B = ref + b, B + np.abs(b)
    whole, y = guarded(M * N, out)
    dmm.mx_matmul_mx(dev(xc), dev(xs), M, K, dev(c), dev(s), N, y, bias=None if b is None else dev(b))
    assert_close(host(y).reshape(M, N), ref, B, K, out, f"{M}x{N}x{K}")
    assert intact(whole)


@pytest.mark.parametrize("M,N,K", [(1, 40, 8192), (16, 33, 4096), (100, 300, 2080), (700, 270, 1030)])
def test_whole_numbers_are_exact(dmm, M, N, K):
    """x in -8 .. 8, scales 1 and weights multiples of 1/2: sums stay below
    8 * 6 * 8192 = 2^18.6, in units of 1/2 (with x in MXFP4, of 1/4)."""
    say(f"whole numbers {M}x{N}x{K}")
    rng = np.random.default_rng(K)
    x = rng.integers(-8, 9, (M, K)).astype(np.float32)
    c, s = packed(rng, N, K, spread=0)
    y = torch.empty((M, N), device=DEV)
    dmm.mx_matmul(bf16_of(x), dev(c), dev(s), N, y)
    assert np.array_equal(host(y), (x.astype(np.float64) @ oracle.mx_unpack(c, s, K).T).astype(np.float32))
    xc, xs = packed(rng, M, K, spread=0)
    dmm.mx_matmul_mx(dev(xc), dev(xs), M, K, dev(c), dev(s), N, y)
    ref = oracle.mx_unpack(xc, xs, K) @ oracle.mx_unpack(c, s, K).T
    assert np.array_equal(host(y), ref.astype(np.float32))


@pytest.mark.parametrize("M", [1, 20, 300])
def test_one_hot_reads_every_weight(dmm, M):
    """x = e_k reads column k exactly, over the whole range of scales."""
    say(f"one-hot M={M}")
    K, N = 320, 37
    rng = np.random.default_rng(M)
    c, _ = packed(rng, N, K)
    s = rng.integers(3, 252, (N, 10)).astype(np.uint8)
    w = oracle.mx_unpack(c, s, K)
    ks = rng.integers(0, K, M)
    x = np.zeros((M, K), np.float32)
    x[np.arange(M), ks] = 1
    y = torch.empty((M, N), device=DEV)
    dmm.mx_matmul(bf16_of(x), dev(c), dev(s), N, y)
    assert np.array_equal(host(y), w[:, ks].T.astype(np.float32))
    xc, xs, _ = oracle.mx_pack(x)
    dmm.mx_matmul_mx(dev(xc), dev(xs), M, K, dev(c), dev(s), N, y)
    assert np.array_equal(host(y), w[:, ks].T.astype(np.float32))


@pytest.mark.parametrize("M", [1, 16, 200])
def test_nan_blocks_and_infinities(dmm, M):
    """A NaN block of W makes its column NaN, one of x its row; an infinity in
    x reaches its own row alone."""
    say(f"NaN blocks M={M}")
    K, N = 200, 50
    rng = np.random.default_rng(M)
    x = activations(rng, M, K)
    c, s = packed(rng, N, K)
    s[7, 6] = 255
    s[49, 0] = 255
    xi = x.copy()
    xi[M - 1, 3] = np.inf
    y = torch.empty((M, N), device=DEV)
    dmm.mx_matmul(bf16_of(xi), dev(c), dev(s), N, y)
    got = host(y)
    assert np.isnan(got[:, [7, 49]]).all()
    rest = np.delete(got, [7, 49], 1)
    assert np.isfinite(rest[:M - 1]).all() and not np.isfinite(rest[M - 1]).any()
    xc, xs, _ = oracle.mx_pack(x)
    xs[M // 2, 2] = 255
    dmm.mx_matmul_mx(dev(xc), dev(xs), M, K, dev(c), dev(s), N, y)
    got = host(y)
    assert np.isnan(got[:, [7, 49]]).all() and np.isnan(got[M // 2]).all()
    assert np.isfinite(np.delete(np.delete(got, M // 2, 0), [7, 49], 1)).all()


def test_empty_sums(dmm):
    say("K = 0 and empty sizes")
    y = torch.full((3, 5), 9.0, device=DEV)
    c, s = torch.empty((5, 0, 16), dtype=torch.uint8, device=DEV), torch.empty((5, 0), dtype=torch.uint8, device=DEV)
    x = torch.empty((3, 0), dtype=torch.bfloat16, device=DEV)
    dmm.mx_matmul(x, c, s, 5, y, bias=torch.arange(5.0, device=DEV))
    assert np.array_equal(host(y), np.tile(np.arange(5, dtype=np.float32), (3, 1)))
    dmm.mx_matmul(x, c, s, 5, y)
    assert not host(y).any()
    y.fill_(9.0)
    dmm.mx_matmul_mx(torch.empty((3, 0, 16), dtype=torch.uint8, device=DEV),
                     torch.empty((3, 0), dtype=torch.uint8, device=DEV), 3, 0, c, s, 5, y)
    assert not host(y).any()
    many = torch.full((70, 5), 9.0, device=DEV)
    dmm.mx_matmul(torch.empty((70, 0), dtype=torch.bfloat16, device=DEV), c, s, 5, many, bias=torch.arange(5.0, device=DEV))
    assert np.array_equal(host(many), np.tile(np.arange(5, dtype=np.float32), (70, 1)))
    dmm.mx_matmul_mx(torch.empty((70, 0, 16), dtype=torch.uint8, device=DEV),
                     torch.empty((70, 0), dtype=torch.uint8, device=DEV), 70, 0, c, s, 5, many)
    assert not host(many).any()
    dmm.mx_matmul(x[:0], c, s, 5, y[:0])
    dmm.mx_pack(torch.empty((0, 5), device=DEV), torch.empty((0, 1, 16), dtype=torch.uint8, device=DEV),
                torch.empty((0, 1), dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("M", [3, 150, 300])
def test_activations_at_any_offset(dmm, M):
    """x starting 1, 3 and 8 elements into its buffer gives the same bits as
    its aligned copy wherever the same kernel runs, and the bound everywhere."""
    say(f"offsets M={M}")
    K, N = 512, 130
    rng = np.random.default_rng(M)
    x = activations(rng, M, K)
    c, s = packed(rng, N, K)
    ref, B = oracle.matmul_ref(workloads.bf16_bits(x), oracle.mx_unpack(c, s, K))
    for off in (1, 3, 8):
        buf = torch.full((M * K + off,), float("nan"), dtype=torch.bfloat16, device=DEV)
        xo = buf[off:].view(M, K)
        xo.copy_(bf16_of(x))
        y = torch.empty((M, N), device=DEV)
        dmm.mx_matmul(xo, dev(c), dev(s), N, y)
        assert_close(host(y), ref, B, K, torch.float32, f"offset {off}")


@pytest.mark.parametrize("M", [1, 4, 16, 33, 130])
@pytest.mark.parametrize("K", [512, 1024, 8704, 700])
def test_scales_at_any_offset(dmm, M, K):
    """Scale bytes that start anywhere give the same bits as aligned ones."""
    say(f"scales' offsets M={M} K={K}")
    N, nb = 70, -(-K // 32)
    rng = np.random.default_rng(M + K)
    x = activations(rng, M, K)
    c, s = packed(rng, N, K)
    X, C = bf16_of(x), dev(c)
    xc, xs = packed(rng, M, K)
    XC = dev(xc)
    first = {}
    for off in (0, 1, 8, 15):
        S, XS = (torch.full((n * nb + off,), 200, dtype=torch.uint8, device=DEV)[off:].view(n, nb) for n in (N, M))
        S.copy_(dev(s))
        XS.copy_(dev(xs))
        y = torch.empty((2, M, N), device=DEV)
        dmm.mx_matmul(X, C, S, N, y[0])
        dmm.mx_matmul_mx(XC, XS, M, K, C, S, N, y[1])
        got = host(y)
        if off == 0:
            ref, B = oracle.matmul_ref(workloads.bf16_bits(x), oracle.mx_unpack(c, s, K))
            assert_close(got[0], ref, B, K, torch.float32, "aligned")
            first = got
        assert np.array_equal(got, first), off


@pytest.mark.parametrize("M", [2, 60])
def test_far_rows(dmm, M):
    """Rows of x a long way apart: offsets past 2^31 bytes, x's rows past
    what the tiles' 32-bit offsets take."""
    say(f"far rows M={M}")
    K, N, ld = 64, 40, 9000001
    rng = np.random.default_rng(M)
    x = activations(rng, M, K)
    c, s = packed(rng, N, K)
    ref, B = oracle.matmul_ref(workloads.bf16_bits(x), oracle.mx_unpack(c, s, K))
    for step in (ld, 60000000 if M == 2 else 30000000):
        buf = torch.full(((M - 1) * step + K,), float("nan"), dtype=torch.bfloat16, device=DEV)
        xo = buf.as_strided((M, K), (step, 1))
        xo.copy_(bf16_of(x))
        y = torch.empty((M, N), device=DEV)
        dmm.mx_matmul(xo, dev(c), dev(s), N, y)
        assert_close(host(y), ref, B, K, torch.float32, f"rows {step} apart")
        xc, xs = (torch.zeros(sh, dtype=torch.uint8, device=DEV) for sh in dmm.mx_shape(M, K))
        dmm.mx_pack(xo, xc, xs)
        pc, ps = oracle.mx_pack(x)[:2]
        assert np.array_equal(xc.cpu().numpy(), pc) and np.array_equal(xs.cpu().numpy(), ps)


def test_two_streams_at_once(dmm):
    """Calls on two streams, each with its own tensors, that may run together."""
    say("two streams")
    rng = np.random.default_rng(8)
    jobs = []
    for M, N, K in ((5, 4000, 2048), (300, 1000, 1024)):
        x = activations(rng, M, K)
        c, s = packed(rng, N, K)
        jobs.append((bf16_of(x), dev(c), dev(s), N, torch.empty((M, N), device=DEV), torch.cuda.Stream()))
    alone = []
    for X, C, S, N, y, _ in jobs:
        dmm.mx_matmul(X, C, S, N, y)
        alone.append(host(y))
        y.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for X, C, S, N, y, stream in jobs:
            with torch.cuda.stream(stream):
                dmm.mx_matmul(X, C, S, N, y)
    torch.cuda.synchronize()
    for (_, _, _, _, y, _), a in zip(jobs, alone):
        assert np.array_equal(host(y), a)


def test_large_offsets(dmm):
    """Rows whose codes lie past 2^31 bytes, and outputs past 2^31 elements' bytes."""
    say("large offsets")
    N, K = 140000, 32768                                            # 2.3 GB of codes
    rng = np.random.default_rng(3)
    codes = torch.zeros((N, K // 32, 16), dtype=torch.uint8, device=DEV)
    scales = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
    c, s = packed(rng, 64, K, spread=0)
    codes[-64:] = dev(c)
    x = rng.integers(-4, 5, (20, K)).astype(np.float32)
    ref = (x.astype(np.float64) @ oracle.mx_unpack(c, s, K).T).astype(np.float32)
    for M in (1, 20):
        y = torch.full((M, N), 5.0, device=DEV)
        dmm.mx_matmul(bf16_of(x[:M]), codes, scales, N, y)
        assert np.array_equal(host(y[:, -64:]), ref[:M]) and not host(y[:, :1000]).any()


def test_another_stream_and_repeats(dmm):
    """On a side stream, behind work of the current one; twice the same bits."""
    say("side stream")
    rng = np.random.default_rng(5)
    x = activations(rng, 40, 640)
    c, s = packed(rng, 96, 640)
    X, C, S = bf16_of(x), dev(c), dev(s)
    ys = [torch.empty((40, 96), device=DEV) for _ in range(3)]
    dmm.mx_matmul(X, C, S, 96, ys[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dmm.mx_matmul(X, C, S, 96, ys[1])
        dmm.mx_matmul(X, C, S, 96, ys[2])
    torch.cuda.current_stream().wait_stream(side)
    assert np.array_equal(host(ys[0]), host(ys[1])) and np.array_equal(host(ys[0]), host(ys[2]))


def test_bf16_linear_with_quantised_activations_replayed(dmm):
    """pack + product captured once and replayed on new inputs, with eager work between."""
    say("captured linear")
    rng = np.random.default_rng(6)
    M, N, K = 24, 200, 544
    c, s = packed(rng, N, K)
    C, S = dev(c), dev(s)
    X = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    xc, xs = (torch.zeros(sh, dtype=torch.uint8, device=DEV) for sh in dmm.mx_shape(M, K))
    y, st = torch.zeros((M, N), device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)

    def step(y):
        dmm.mx_pack(X, xc, xs, status=st)
        dmm.mx_matmul_mx(xc, xs, M, K, C, S, N, y)

    step(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(y)
    for i in range(4):
        X.copy_(bf16_of(activations(rng, M, K)))
        eager = torch.zeros_like(y)
        step(eager)
        y.zero_()
        graph.replay()
        assert np.array_equal(host(y), host(eager)) and int(host(st)[0]) == 0
