"""e4m3 blocks, the router's choice and the combination without a GPU: the oracle against
values worked out by hand, and what the entry points and their binding refuse before any
launch."""

import ctypes

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
dmm = pytest.importorskip("decode_matmul_amd")
lib = dmm.raw()

NULL, SHAPE, UNSUPPORTED, DTYPE, ALIGN = 1, 2, 3, 4, 5
FAKE = ctypes.c_void_p(0x10000)          # never dereferenced: every call below fails first
ODD = ctypes.c_void_p(0x10001)
EVEN = ctypes.c_void_p(0x10002)
HALF = ctypes.c_void_p(0x10008)          # 8-byte aligned
BIG = 1 << 31


# ---------------------------------------------------------------- the oracle


def test_e4m3_against_torch():
    """Every code, and rounding of values around every grid point and midpoint."""
    c = torch.arange(256, dtype=torch.int16).to(torch.uint8)
    v = c.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(oracle.E4M3)) and np.array_equal(v[~np.isnan(v)], oracle.E4M3[~np.isnan(v)])
    grid = oracle.E4M3[:127]
    mid = (grid[1:] + grid[:-1]) / 2
    points = np.concatenate([grid, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    points = np.concatenate([points, -points]).astype(np.float32)
    want = torch.from_numpy(points).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.f8_encode(points.astype(np.float64)), want)


def test_pack_by_hand():
    """448 itself needs scale 1, the next fp32 value scale 2; an empty block the least scale."""
    w = np.zeros((3, 130), np.float32)
    w[0, :3] = [448, -1, 0.0009765625]                  # 2^-10: half of the least subnormal, to 0
    w[0, 129] = 0.001953125
    w[1, 5] = np.nextafter(np.float32(448), np.float32(500))
    codes, scales, fine = oracle.f8_pack(w, 1)
    assert fine and scales[:, 0].tolist() == [1, 2, 2.0 ** -126]
    assert scales[0, 1] == 2.0 ** -17                   # 2^-9 / 448 = 2^-17 / 1.75 ... 2^-17.8
    assert codes[0, 0, :3].tolist() == [0x7e, 0xb8, 0]
    assert codes[1, 0, 5] == 0x76                       # 224
    v = oracle.f8_unpack(codes, scales, 130, 1)
    assert v.shape == (3, 130) and v[0, 0] == 448 and v[0, 129] == w[0, 129] and v[1, 5] == 448
    codes, scales, fine = oracle.f8_pack(w, 128)
    assert scales.shape == (1, 2) and scales[0, 0] == 2 and codes[0, 0, 1] == 0xb0
    w[2, 7] = np.inf
    codes, scales, fine = oracle.f8_pack(w, 1)
    assert not fine and np.isnan(scales[2, 0]) and not codes[2].any() and scales[2, 1] == 2.0 ** -126


def test_pack_rule():
    """The least power of two: a block's largest code lies in (224, 448], or at the least scale below."""
    rng = np.random.default_rng(0)
    w = (rng.standard_normal((64, 128)) * 10.0 ** rng.uniform(-44, 38, (64, 1))).astype(np.float32)
    codes, scales, _ = oracle.f8_pack(w, 1)
    top = np.abs(w).max(axis=1).astype(np.float64) / scales[:, 0]
    assert (top <= 448).all() and ((top > 224) | (scales[:, 0] == np.float32(2.0 ** -126))).all()


def test_norm_by_hand():
    h, y = oracle.f8_norm([[3.0, 4.0]], [[0.0, 0.0]], [1.0, 2.0], 0.0, lambda v: v.astype(np.float32))
    assert np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=2.0 ** -22) and h.tolist() == [[3, 4]]


def test_gate_by_hand():
    z = np.log([[1.0, 4.0, 2.0, 1.0]])
    ids, w = oracle.moe_gate(z, 2)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[2 / 3, 1 / 3]])
    ids, w = oracle.moe_gate(z, 2, renorm=False, scale=2.0)
    assert np.allclose(w, [[1.0, 0.5]])
    ids, _ = oracle.moe_gate(np.zeros((1, 4)), 3)                       # ties: lowest first
    assert ids.tolist() == [[0, 1, 2]]
    # a bias chooses, the weights do not see it
    ids, w = oracle.moe_gate(np.zeros((1, 4)), 2, "sigmoid", bias=np.array([0, 0, 0.1, 0.2]), renorm=False)
    assert ids.tolist() == [[3, 2]] and w.tolist() == [[0.5, 0.5]]
    # groups {0, 1} and {2, 3}: by the best one the second, by the two best the first
    z = np.array([[2.0, 1.9, 2.1, -5.0]])
    assert oracle.moe_gate(z, 2, n_groups=2)[0].tolist() == [[2, 3]]
    assert oracle.moe_gate(z, 2, "sigmoid", n_groups=2, group_top=2)[0].tolist() == [[0, 1]]
    z = np.array([[-np.inf, 1.0, np.nan, -np.inf]])
    ids, w = oracle.moe_gate(z, 3, "sigmoid")
    assert ids.tolist() == [[2, 1, -1]] and np.isnan(w[0, :2]).all() and w[0, 2] == 0
    assert oracle.moe_gate(z, 1, mask=[0])[0].tolist() == [[-1]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_by_differences(score, renorm):
    """Central differences with h = 1e-5 of the weights of fixed ids: truncation h^2 / 6
    of the third derivative (below 6 scale max|dw|), rounding 1e-15 / h."""
    rng = np.random.default_rng(1)
    M, E, k, h = 5, 7, 3, 1e-5
    z, dw = rng.standard_normal((M, E)) * 2, rng.standard_normal((M, k))
    ids, _ = oracle.moe_gate(z, k, score, renorm=renorm)
    ids[2, 1], ids[3] = -1, -1

    def f(z):
        p = oracle.gate_scores(z, score)
        w = np.where(ids >= 0, np.take_along_axis(p, np.maximum(ids, 0), 1), 0)
        if renorm:
            w = w / np.maximum(w.sum(axis=1, keepdims=True), 1e-300)
        return 1.5 * (w * dw).sum()

    g = oracle.moe_gate_grad(z, ids, dw, score, renorm, 1.5)
    for t in range(M):
        for e in range(E):
            up, dn = z.copy(), z.copy()
            up[t, e] += h
            dn[t, e] -= h
            assert abs((f(up) - f(dn)) / (2 * h) - g[t, e]) < 1e-8
    assert not g[3].any()


def test_combine_by_hand():
    y = np.array([[[1.0, 2.0], [np.nan, np.nan], [3.0, 4.0]]])
    ids, w = np.array([[0, -1, 1]]), np.array([[0.5, np.nan, 2.0]])
    out, _ = oracle.moe_combine(y, ids, w, 2, np.array([[10.0, 20.0]]))
    assert out.tolist() == [[16.5, 29.0]]
    dy, dw, _ = oracle.moe_combine_grad(y, ids, w, 2, np.array([[1.0, -1.0]]))
    assert dy.tolist() == [[[0.5, -0.5], [0, 0], [2, -2]]] and dw.tolist() == [[-1, 0, -1]]


# ------------------------------------------------------------------ refusals


def refused(f, ok, cases):
    for i, v, want in cases:
        a = list(ok)
        a[i] = v
        assert f(*a) == want, (i, v)


def test_f8_pack_refusals():
    ok = [FAKE, 0, 4, 64, 64, 1, FAKE, FAKE, None, None]
    refused(lib.f8_pack, ok, ((0, None, NULL), (6, None, NULL), (7, None, NULL), (1, 2, DTYPE), (2, -1, SHAPE),
                              (2, BIG, SHAPE), (3, 1 << 23, SHAPE), (4, 63, SHAPE), (5, 2, UNSUPPORTED),
                              (5, 0, UNSUPPORTED), (0, ODD, ALIGN), (6, HALF, ALIGN), (7, EVEN, ALIGN), (8, ODD, ALIGN),
                              (2, 1 << 29, SHAPE), (2, 0, 0), (3, 0, 0)))
    assert lib.f8_pack(FAKE, 1, ((1 << 28) - 16) // 2, 129, 129, 1, FAKE, FAKE, None, None) == SHAPE


def test_f8_unpack_refusals():
    ok = [FAKE, FAKE, 4, 64, 128, FAKE, 1, None, None]
    refused(lib.f8_unpack, ok, ((0, None, NULL), (1, None, NULL), (5, None, NULL), (6, 3, DTYPE), (2, -1, SHAPE),
                                (3, -1, SHAPE), (4, 64, UNSUPPORTED), (5, ODD, ALIGN), (0, HALF, ALIGN),
                                (1, EVEN, ALIGN), (7, ODD, ALIGN), (2, 1 << 29, SHAPE), (2, 0, 0)))


def test_f8_norm_pack_refusals():
    ok = [FAKE, 1, 4, 64, 64, FAKE, 64, FAKE, 1, 1e-6, FAKE, 64, FAKE, 64, FAKE, FAKE, None, None]
    refused(lib.f8_norm_pack, ok, (
        (0, None, NULL), (7, None, NULL), (14, None, NULL), (15, None, NULL), (1, 2, DTYPE), (8, 2, DTYPE),
        (2, -1, SHAPE), (3, -1, SHAPE), (3, 1 << 23, SHAPE), (2, 1 << 22, SHAPE), (4, 63, SHAPE), (6, 63, SHAPE),
        (11, 63, SHAPE), (13, 63, SHAPE), (9, -1e-9, SHAPE), (9, float("nan"), SHAPE), (0, ODD, ALIGN), (5, ODD, ALIGN),
        (7, ODD, ALIGN), (10, ODD, ALIGN), (12, ODD, ALIGN), (14, HALF, ALIGN), (15, EVEN, ALIGN), (16, ODD, ALIGN),
        (2, 0, 0), (3, 0, 0)))


def test_f8_matmul_refusals():
    ok = [FAKE, FAKE, 4, 64, FAKE, FAKE, 16, FAKE, FAKE, 0, None]
    refused(lib.f8_matmul, ok, (
        (0, None, NULL), (1, None, NULL), (4, None, NULL), (5, None, NULL), (8, None, NULL), (2, -1, SHAPE),
        (2, BIG, SHAPE), (3, -1, SHAPE), (3, 1 << 23, SHAPE), (6, -1, SHAPE), (6, BIG, SHAPE), (9, 2, DTYPE),
        (0, HALF, ALIGN), (1, EVEN, ALIGN), (4, HALF, ALIGN), (5, EVEN, ALIGN), (7, ODD, ALIGN), (8, EVEN, ALIGN),
        (2, 0, 0), (6, 0, 0)))
    assert lib.f8_matmul(FAKE, FAKE, BIG - 1, 64, FAKE, FAKE, BIG - 1, None, FAKE, 0, None) == SHAPE    # grid


def test_f8_matmul_experts_refusals():
    ok = [FAKE, FAKE, 4, 64, FAKE, FAKE, 16, 8, FAKE, FAKE, FAKE, 2, FAKE, 0, None]
    refused(lib.f8_matmul_experts, ok, (
        (0, None, NULL), (1, None, NULL), (4, None, NULL), (5, None, NULL), (9, None, NULL), (10, None, NULL),
        (12, None, NULL), (7, 0, SHAPE), (11, 0, SHAPE), (2, 1 << 30, SHAPE), (2, -1, SHAPE), (13, 9, DTYPE),
        (4, HALF, ALIGN), (9, ODD, ALIGN), (10, ODD, ALIGN), (12, ODD, ALIGN), (2, 0, 0)))
    for E in (BIG - 1, 1 << 25):
        for N in (129, 300):
            assert lib.f8_matmul_experts(FAKE, FAKE, 4, 64, FAKE, FAKE, N, E, None, FAKE, FAKE, 2, FAKE, 0, None) == SHAPE


def test_moe_gate_refusals():
    ok = [FAKE, 0, 4, 64, 64, None, None, 0, 1, 1, 1, 8, 1, 1.0, FAKE, FAKE, None]
    refused(lib.moe_gate, ok, (
        (0, None, NULL), (14, None, NULL), (15, None, NULL), (1, 2, DTYPE), (2, -1, SHAPE), (2, BIG, SHAPE),
        (3, 0, SHAPE), (3, 513, UNSUPPORTED), (4, 63, SHAPE), (7, 2, UNSUPPORTED), (8, 0, SHAPE), (8, 3, SHAPE),
        (8, 65, UNSUPPORTED), (9, 0, SHAPE), (9, 2, SHAPE), (10, 0, UNSUPPORTED), (10, 3, UNSUPPORTED), (11, 0, SHAPE),
        (11, 33, UNSUPPORTED), (0, ODD, ALIGN), (6, ODD, ALIGN), (14, ODD, ALIGN), (15, EVEN, ALIGN), (2, 0, 0)))
    grouped = list(ok)
    grouped[8], grouped[9] = 16, 1                      # 4 experts take part
    assert lib.moe_gate(*grouped) == SHAPE
    assert lib.moe_gate(FAKE, 1, 1 << 26, 512, 512, None, None, 0, 1, 1, 1, 8, 1, 1.0, FAKE, FAKE, None) == SHAPE


def test_moe_gate_grad_refusals():
    ok = [FAKE, 1, 100, 8, 8, FAKE, FAKE, 0, 2, 1, 1.0, FAKE, None]
    refused(lib.moe_gate_grad, ok, (
        (0, None, NULL), (5, None, NULL), (6, None, NULL), (11, None, NULL), (1, 5, DTYPE), (2, -1, SHAPE),
        (3, 0, SHAPE), (3, 600, UNSUPPORTED), (4, 7, SHAPE), (7, -1, UNSUPPORTED), (8, 0, SHAPE), (8, 33, UNSUPPORTED),
        (0, ODD, ALIGN), (5, ODD, ALIGN), (6, ODD, ALIGN), (11, ODD, ALIGN), (2, 0, 0)))
    assert lib.moe_gate_grad(FAKE, 1, BIG - 1, 512, 512, FAKE, FAKE, 0, 2, 1, 1.0, FAKE, None) == SHAPE


def test_moe_combine_refusals():
    ok = [FAKE, 1, 4, 2, 64, FAKE, FAKE, 8, FAKE, FAKE, 1, None]
    refused(lib.moe_combine, ok, (
        (0, None, NULL), (5, None, NULL), (6, None, NULL), (9, None, NULL), (1, 2, DTYPE), (10, 2, DTYPE),
        (2, -1, SHAPE), (2, 1 << 30, SHAPE), (3, 0, SHAPE), (4, -1, SHAPE), (4, BIG, SHAPE), (7, 0, SHAPE),
        (0, ODD, ALIGN), (5, ODD, ALIGN), (6, ODD, ALIGN), (8, ODD, ALIGN), (9, ODD, ALIGN), (2, 0, 0), (4, 0, 0)))
    assert lib.moe_combine(FAKE, 1, (1 << 30) - 1, 1, 1 << 20, FAKE, FAKE, 8, None, FAKE, 1, None) == SHAPE


def test_moe_combine_grad_refusals():
    ok = [FAKE, 1, 4, 2, 64, FAKE, FAKE, 8, FAKE, 1, FAKE, FAKE, None]
    refused(lib.moe_combine_grad, ok, (
        (0, None, NULL), (5, None, NULL), (6, None, NULL), (8, None, NULL), (10, None, NULL), (11, None, NULL),
        (1, 2, DTYPE), (9, 2, DTYPE), (2, -1, SHAPE), (2, 1 << 30, SHAPE), (3, 0, SHAPE), (4, -1, SHAPE), (7, 0, SHAPE),
        (2, 1 << 24, SHAPE), (0, ODD, ALIGN), (8, ODD, ALIGN), (10, ODD, ALIGN), (11, ODD, ALIGN), (2, 0, 0)))


def test_binding_refuses_wrong_tensors():
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    x = torch.zeros(2, 200, dtype=bf)
    (cs, ss), (ws, wss) = dmm.f8_shape(2, 200), dmm.f8_shape(130, 200, 128)
    assert (cs, ss, ws, wss) == ((2, 2, 128), (2, 2), (130, 2, 128), (2, 2))
    c, s, w, t, y = torch.zeros(cs, dtype=u8), torch.zeros(ss), torch.zeros(ws, dtype=u8), torch.zeros(wss), \
        torch.zeros(2, 130)
    gate = (torch.zeros(2, 8), torch.zeros(2, 2, dtype=i32), torch.zeros(2, 2))
    rows = (torch.zeros(2, 2, 5), torch.zeros(2, 2, dtype=i32), torch.zeros(2, 2), 8)
    for error, call in (
            (TypeError, lambda: dmm.f8_pack(x.half(), c, s)),
            (ValueError, lambda: dmm.f8_pack(x, c[:1], s)),
            (ValueError, lambda: dmm.f8_pack(x, c, s, block_rows=128)),
            (ValueError, lambda: dmm.f8_pack(x[:1].expand(2, 200), c, s)),
            (TypeError, lambda: dmm.f8_pack(x, c.float(), s)),
            (TypeError, lambda: dmm.f8_unpack(c, s, 2, 200, x.half())),
            (TypeError, lambda: dmm.f8_norm_pack(x, torch.zeros(200).half(), c, s, 1e-6)),
            (ValueError, lambda: dmm.f8_norm_pack(x, torch.zeros(199), c, s, 1e-6)),
            (TypeError, lambda: dmm.f8_norm_pack(x, torch.zeros(200), c, s, 1e-6, residual=x.float())),
            (ValueError, lambda: dmm.f8_norm_pack(x, torch.zeros(200), c, s, 1e-6, h_out=x[:1])),
            (ValueError, lambda: dmm.f8_matmul(c, s, 2, 200, w[:129], t, 130, y)),
            (ValueError, lambda: dmm.f8_matmul(c, s, 2, 200, w, t[:1], 130, y)),
            (TypeError, lambda: dmm.f8_matmul(c, s.to(bf), 2, 200, w, t, 130, y)),
            (ValueError, lambda: dmm.f8_matmul(c, s, 2, 200, w, t, 130, y)),            # not on a GPU
            (ValueError, lambda: dmm.f8_matmul_experts(c, s, 2, 200, w, t, 65, y, 2, torch.zeros(2, dtype=i32),
                                                       torch.zeros(2, dtype=i32), 1)),
            (ValueError, lambda: dmm.moe_gate(*gate, score="relu")),
            (ValueError, lambda: dmm.moe_gate(gate[0], gate[1], torch.zeros(2, 3))),
            (TypeError, lambda: dmm.moe_gate(gate[0], gate[1].long(), gate[2])),
            (ValueError, lambda: dmm.moe_gate(*gate, bias=torch.zeros(7))),
            (ValueError, lambda: dmm.moe_gate_grad(gate[0], gate[1], gate[2], torch.zeros(2, 7))),
            (TypeError, lambda: dmm.moe_gate_grad(gate[0], gate[1], gate[2], torch.zeros(2, 8, dtype=bf))),
            (ValueError, lambda: dmm.moe_combine(*rows, torch.zeros(2, 4))),
            (TypeError, lambda: dmm.moe_combine(*rows, torch.zeros(2, 5), add=torch.zeros(2, 5, dtype=bf))),
            (TypeError, lambda: dmm.moe_combine(*rows, torch.zeros(2, 5).half())),
            (TypeError, lambda: dmm.moe_combine_grad(*rows, torch.zeros(2, 5), rows[0].to(bf), rows[2]))):
        with pytest.raises(error):
            call()
