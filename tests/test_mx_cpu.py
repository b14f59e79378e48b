"""MXFP4 and routing without a GPU: the oracle against values worked out by
hand, and what the entry points and their binding refuse before any launch."""

import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
dmm = pytest.importorskip("decode_matmul_amd")
lib = dmm.raw()

NULL, SHAPE, UNSUPPORTED, DTYPE, ALIGN = 1, 2, 3, 4, 5
FAKE = ctypes.c_void_p(0x10000)          # never dereferenced: every call below fails first
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10008)          # 8-byte aligned
BIG = 1 << 31


# ---------------------------------------------------------------- the oracle


def test_pack_by_hand():
    """max 6.5 -> scale 1; ties to the even code, 6.5 saturates, signs kept."""
    w = np.zeros((1, 34), np.float32)
    w[0, :12] = [6.5, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.1, -0.75, 5.1, 0.26]
    w[0, 32:] = [-3 * 2.0 ** -20, 2.0 ** -20]             # max 1.5 * 2^-19 -> scale 2^-21
    codes, scales, fine = oracle.mx_pack(w)
    assert fine and scales.tolist() == [[127, 106]]
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(2, 32)
    assert nib[0, :12].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 7, 1]
    assert nib[1, :3].tolist() == [15, 4, 0]
    v = oracle.mx_unpack(codes, scales, 34)
    assert v[0, 0] == 6 and v[0, 9] == -1 and v[0, 32] == -6 * 2.0 ** -21 and v[0, 33] == 2.0 ** -20


def test_pack_scale_range():
    """Zero, subnormal and the largest blocks, and blocks that are not finite."""
    w = np.zeros((6, 32), np.float32)
    w[1, 0] = 2.0 ** -149
    w[2, 0] = 2.0 ** -126
    w[3, 0] = np.finfo(np.float32).max
    w[4, 0] = np.inf
    w[5, 31] = np.nan
    codes, scales, fine = oracle.mx_pack(w)
    assert not fine and scales[:, 0].tolist() == [0, 0, 0, 252, 255, 255]
    assert codes[0].max() == 0 and codes[1].max() == 0 and codes[2, 0, 0] == 4      # 2 * 2^-127
    assert codes[3, 0, 0] == 7 and codes[4:].max() == 0
    assert np.isnan(oracle.mx_unpack(codes, scales, 32)[4:]).all()


def test_unpack_of_every_code():
    codes = np.arange(16, dtype=np.uint8).reshape(1, 1, 16)     # low nibble c, high nibble 0
    v = oracle.mx_unpack(codes, np.array([[128]], np.uint8), 32)[0]
    assert v[0::2].tolist() == [0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12]
    assert not v[1::2].any()


def test_route_by_hand():
    counts, offsets, order = oracle.moe_route([[2, 0], [-1, 2], [2, 3]], 3)
    assert counts.tolist() == [1, 0, 3] and offsets.tolist() == [0, 1, 1, 4]
    assert order.tolist() == [1, 0, 3, 4, 2, 5]


def test_balance_by_hand():
    """An even router has loss 1 and no gradient; all slots on one of E experts
    and p = (3/4, 1/4) give 2 * 3/4."""
    loss, w, _ = oracle.moe_balance(np.zeros((5, 4)), [3, 3, 3, 3])
    assert abs(loss - 1) < 1e-15 and np.allclose(w, 0.2)
    assert np.abs(oracle.moe_balance_grad(np.zeros((5, 4)), [3, 3, 3, 3])).max() < 1e-17
    z = np.log([[3.0, 1.0]])
    loss, _, _ = oracle.moe_balance(z, [7, 0])
    assert abs(loss - 1.5) < 1e-15
    assert np.allclose(oracle.moe_balance_grad(z, [7, 0]), [[3 / 8, -3 / 8]])
    assert oracle.moe_balance(z, [0, 0])[0] == 0 and oracle.moe_balance(z, [1, 1], [0])[0] == 0


def test_balance_gradient_by_differences():
    """Central differences with h = 1e-4: truncation h^2 / 6 of the third
    derivative (below 2 max w, w < E / T), rounding 1e-16 / h."""
    rng = np.random.default_rng(0)
    z = rng.standard_normal((6, 5))
    z[2, 1] = -np.inf
    z[4] = -np.inf
    counts, mask = [4, 0, 1, 2, 3], [1, 1, 1, 0, 1, 1]
    g = oracle.moe_balance_grad(z, counts, mask)
    h = 1e-4
    for t in range(6):
        for e in range(5):
            if z[t, e] == -np.inf:
                assert g[t, e] == 0
                continue
            up, dn = z.copy(), z.copy()
            up[t, e] += h
            dn[t, e] -= h
            d = (oracle.moe_balance(up, counts, mask)[0] - oracle.moe_balance(dn, counts, mask)[0]) / (2 * h)
            assert abs(d - g[t, e]) < 1e-8
    assert not g[3].any() and not g[4].any()


# ------------------------------------------------------------------ refusals


def changed(ok, i, v):
    a = list(ok)
    a[i] = v
    return a


def test_mx_pack_refusals():
    f, ok = lib.mx_pack, [FAKE, 0, 4, 64, 64, FAKE, FAKE, None, None]
    for i, v, want in ((0, None, NULL), (5, None, NULL), (6, None, NULL), (1, 2, DTYPE), (2, -1, SHAPE),
                       (2, BIG, SHAPE), (3, BIG, SHAPE), (4, 63, SHAPE), (0, ODD, ALIGN), (5, HALF, ALIGN),
                       (7, ODD, ALIGN)):
        assert f(*changed(ok, i, v)) == want, (i, v)
    assert f(FAKE, 0, BIG - 1, BIG - 1, BIG - 1, FAKE, FAKE, None, None) == SHAPE       # grid
    assert f(*changed(ok, 2, 0)) == 0 and f(*changed(ok, 3, 0)) == 0                    # nothing to do


def test_mx_unpack_refusals():
    f, ok = lib.mx_unpack, [FAKE, FAKE, 4, 64, FAKE, 1, None, None]
    for i, v, want in ((0, None, NULL), (1, None, NULL), (4, None, NULL), (5, 3, DTYPE), (2, -1, SHAPE),
                       (3, -1, SHAPE), (4, ODD, ALIGN), (0, HALF, ALIGN), (6, ODD, ALIGN)):
        assert f(*changed(ok, i, v)) == want, (i, v)
    assert f(*changed(ok, 2, 0)) == 0


def test_mx_matmul_refusals():
    f, ok = lib.mx_matmul, [FAKE, 4, 64, 64, FAKE, FAKE, 16, FAKE, FAKE, 0, None]
    for i, v, want in ((0, None, NULL), (4, None, NULL), (5, None, NULL), (8, None, NULL), (1, -1, SHAPE),
                       (2, -1, SHAPE), (6, -1, SHAPE), (1, BIG, SHAPE), (3, 63, SHAPE), (9, 2, DTYPE),
                       (0, ODD, ALIGN), (4, HALF, ALIGN), (7, ODD, ALIGN), (8, ctypes.c_void_p(0x10002), ALIGN)):
        assert f(*changed(ok, i, v)) == want, (i, v)
    assert f(FAKE, BIG - 1, 64, 64, FAKE, FAKE, BIG - 1, None, FAKE, 0, None) == SHAPE  # grid
    assert f(*changed(ok, 1, 0)) == 0 and f(*changed(ok, 6, 0)) == 0


def test_mx_matmul_mx_refusals():
    f, ok = lib.mx_matmul_mx, [FAKE, FAKE, 4, 64, FAKE, FAKE, 16, FAKE, FAKE, 1, None]
    for i, v, want in ((0, None, NULL), (1, None, NULL), (4, None, NULL), (5, None, NULL), (8, None, NULL),
                       (2, -1, SHAPE), (3, BIG, SHAPE), (6, -1, SHAPE), (9, -1, DTYPE), (0, HALF, ALIGN),
                       (4, HALF, ALIGN), (8, ODD, ALIGN)):
        assert f(*changed(ok, i, v)) == want, (i, v)
    assert f(*changed(ok, 2, 0)) == 0


def test_mx_matmul_experts_refusals():
    f = lib.mx_matmul_experts
    ok = [FAKE, 4, 64, 64, FAKE, FAKE, 16, 8, FAKE, FAKE, FAKE, 2, FAKE, 0, None]
    for i, v, want in ((0, None, NULL), (4, None, NULL), (9, None, NULL), (10, None, NULL), (12, None, NULL),
                       (7, 0, SHAPE), (11, 0, SHAPE), (1, 1 << 30, SHAPE), (1, -1, SHAPE), (3, 10, SHAPE),
                       (13, 9, DTYPE), (4, HALF, ALIGN), (9, ODD, ALIGN), (10, ODD, ALIGN), (12, ODD, ALIGN)):
        assert f(*changed(ok, i, v)) == want, (i, v)
    assert f(*changed(ok, 1, 0)) == 0


def test_moe_route_refusals():
    f, ok = lib.moe_route, [FAKE, 4, 2, 8, FAKE, FAKE, FAKE, None, 0, None]
    for i, v, want in ((0, None, NULL), (4, None, NULL), (5, None, NULL), (6, None, NULL), (1, -1, SHAPE),
                       (2, 0, SHAPE), (3, 0, SHAPE), (3, 513, UNSUPPORTED), (1, 1 << 30, SHAPE),
                       (0, ODD, ALIGN), (6, ODD, ALIGN)):
        assert f(*changed(ok, i, v)) == want, (i, v)
    need = lib.moe_route_workspace_bytes(1 << 16, 8, 64)
    big = [FAKE, 1 << 16, 8, 64, FAKE, FAKE, FAKE, FAKE, need - 1, None]
    assert need > 0 and f(*big) == SHAPE
    assert f(*changed(big, 7, None)) == NULL and f(*changed(big, 7, ODD)) == ALIGN
    assert lib.moe_route_workspace_bytes(16, 8, 64) == 0
    assert lib.moe_route_workspace_bytes(-1, 8, 64) == -1 and lib.moe_route_workspace_bytes(1, 8, 513) == -1


def test_moe_balance_refusals():
    need = lib.moe_balance_workspace_bytes(1 << 16, 8)
    assert need > 0 and lib.moe_balance_workspace_bytes(16, 64) == 0
    f, ok = lib.moe_balance, [FAKE, 0, 1 << 16, 8, 8, None, FAKE, FAKE, FAKE, FAKE, need, None]
    for i, v, want in ((0, None, NULL), (6, None, NULL), (7, None, NULL), (8, None, NULL), (9, None, NULL),
                       (1, 5, DTYPE), (2, -1, SHAPE), (3, 0, SHAPE), (3, 600, UNSUPPORTED), (4, 7, SHAPE),
                       (10, need - 1, SHAPE), (0, ODD, ALIGN), (9, ctypes.c_void_p(0x10004), ALIGN)):
        assert f(*changed(ok, i, v)) == want, (i, v)
    assert lib.moe_balance_workspace_bytes(-1, 8) == -1


def test_moe_balance_grad_refusals():
    f, ok = lib.moe_balance_grad, [FAKE, 1, 100, 8, 8, None, FAKE, FAKE, FAKE, None]
    for i, v, want in ((0, None, NULL), (6, None, NULL), (7, None, NULL), (8, None, NULL), (1, 5, DTYPE),
                       (2, -1, SHAPE), (3, 0, SHAPE), (3, 600, UNSUPPORTED), (4, 7, SHAPE), (0, ODD, ALIGN),
                       (8, ODD, ALIGN)):
        assert f(*changed(ok, i, v)) == want, (i, v)
    assert f(*changed(ok, 2, 0)) == 0


def test_binding_refuses_wrong_tensors():
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    x, c, s, y = torch.zeros(2, 64, dtype=bf), torch.zeros(16, 2, 16, dtype=u8), torch.zeros(16, 2, dtype=u8), \
        torch.zeros(2, 16)
    with pytest.raises(TypeError):
        dmm.mx_matmul(x.float(), c, s, 16, y)
    with pytest.raises(ValueError):
        dmm.mx_matmul(x, c[:15], s, 16, y)
    with pytest.raises(ValueError):
        dmm.mx_matmul(x[:1].expand(2, 64), c, s, 16, y)          # rows on top of each other
    with pytest.raises(ValueError):
        dmm.mx_matmul(torch.zeros(64, 2, dtype=bf).t(), c, s, 16, y)
    with pytest.raises(ValueError):
        dmm.mx_matmul(x, c, s, 16, y[:1])
    with pytest.raises(ValueError):
        dmm.mx_matmul(x, c, s, 16, y)                            # not on a GPU
    with pytest.raises(TypeError):
        dmm.mx_pack(x.half(), torch.zeros(2, 2, 16, dtype=u8), torch.zeros(2, 2, dtype=u8))
    with pytest.raises(ValueError):
        dmm.mx_pack(x, torch.zeros(2, 2, 16, dtype=u8), torch.zeros(2, 2, dtype=u8))
    with pytest.raises(TypeError):
        dmm.moe_route(torch.zeros(2, 2), 4, torch.zeros(4, dtype=i32), torch.zeros(5, dtype=i32),
                      torch.zeros(4, dtype=i32))
    with pytest.raises(ValueError):
        dmm.moe_route(torch.zeros(2, 2, dtype=i32), 4, torch.zeros(4, dtype=i32), torch.zeros(4, dtype=i32),
                      torch.zeros(4, dtype=i32))
    with pytest.raises(ValueError):
        dmm.moe_balance_grad(torch.zeros(2, 4), torch.zeros(4), torch.zeros(1), torch.zeros(2, 3, dtype=f32))
    with pytest.raises(ValueError):
        dmm.moe_balance_workspace_bytes(1, 0)


def test_moe_balance_largest_batches():
    """2^24 - 1 workgroups are the most: of 1024 / L tokens for the loss, 256 / L for
    the gradient, L = 64 lanes a token of 512 experts, 8 of 64."""
    for E, L in ((512, 64), (257, 64), (64, 8)):
        most = ((1 << 24) - 1) * 1024 // L
        if most < BIG:
            assert lib.moe_balance_workspace_bytes(most, E) == 16 * ((1 << 24) - 1)
            assert lib.moe_balance_workspace_bytes(most + 1, E) == -1
            with pytest.raises(ValueError):
                dmm.moe_balance_workspace_bytes(most + 1, E)
            assert lib.moe_balance(FAKE, 0, most + 1, E, E, None, FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == SHAPE
        assert lib.moe_balance_grad(FAKE, 0, ((1 << 24) - 1) * 256 // L + 1, E, E, None, FAKE, FAKE, FAKE, None) == SHAPE
    assert lib.moe_balance_workspace_bytes(BIG - 1, 8) > 0


def test_most_experts():
    """One workgroup for every 32 rows of W and expert, and for the slots of none."""
    for E in (BIG - 1, 1 << 24):
        for N in (1, 33, 65):
            assert lib.mx_matmul_experts(FAKE, 4, 64, 64, FAKE, FAKE, N, E, None, FAKE, FAKE, 2, FAKE, 0, None) == SHAPE


def test_binding_needs_no_private_function_of_torch():
    """Without them a call takes the current device and stream from the public functions."""
    program = """
import types, torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import decode_matmul_amd as dmm
torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda device: types.SimpleNamespace(cuda_stream=70 + device)
seen = []
dmm._call("test", lambda *a: seen.append(a) or 0, torch.device("cuda", 3), 1, 2)
assert seen == [(1, 2, 73)], seen
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", program], cwd=root, check=True)


def test_largest_packages():
    for K, nb in ((32, 1), (33, 2)):
        assert lib.mx_pack(FAKE, 1, ((1 << 30) - 64) // nb, K, K, FAKE, FAKE, None, None) == SHAPE
        assert lib.mx_unpack(FAKE, FAKE, ((1 << 29) - 32) // nb, K, FAKE, 1, None, None) == SHAPE
