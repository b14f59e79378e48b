"""Every form of the e4m3 products to the last bit, lists, captured graphs, streams and offsets
past 32 bits.

Operands are whole numbers up to 4 in magnitude times scales 1 and 2: every sum is a whole
number below 64 K <= 2^24, which no form rounds, so all of them give the oracle's result.
"""

import numpy as np
import pytest

import oracle
from test_gpu_f8 import assert_close, dropped, random_package
from test_gpu_mx import DEV, dev, guarded, host, intact, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dmm():
    import decode_matmul_amd
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return decode_matmul_amd


# M, N, K by what chooses the form: one token (four or two segments at once), few tokens (three
# or two blocks under way, (1, 8) or (2, 4)), tiles of 32 x 32, 32 x 64, 64 x 64 with four stages
# and two, 128 x 128 and 256 x 256; each with a short K, a cut one, and one of many slabs
FORMS = [(1, 77, 4096), (1, 77, 5120), (1, 77, 5000), (1, 77, 70000), (1, 5, 1), (2, 100, 9000), (8, 100, 130),
         (5, 100, 20001), (3, 8200, 300), (7, 8200, 2300), (16, 100, 700), (11, 100, 9100), (16, 8200, 900),
         (9, 8200, 6500), (13, 8200, 6144),
         (33, 100, 100), (31, 70, 4224), (60, 130, 9000), (100, 65, 640), (17, 33, 5000),
         (40, 8300, 200), (600, 700, 1111), (500, 800, 4100), (64, 8192, 1536),
         (900, 900, 130), (900, 900, 2500), (930, 930, 4096),
         (1100, 1300, 90), (1100, 1300, 900), (1100, 1300, 1100),
         (1500, 2100, 100), (1500, 2100, 700), (2050, 1600, 1300),
         (4100, 2990, 100), (4100, 2990, 256), (3900, 3000, 1030), (4096, 3100, 640)]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", FORMS, ids=["x".join(map(str, f)) for f in FORMS])
def test_dense_forms(dmm, M, N, K, out):
    say(f"f8_matmul form M={M} N={N} K={K} {out}")
    rng = np.random.default_rng(M + 2 * N + 3 * K)
    xc, xs, x = random_package(rng, M, K, 1, exact=True)
    wc, ws, w = random_package(rng, N, K, 128, exact=True)
    bias = rng.integers(-9, 10, N).astype(np.float32)
    ref = torch.from_numpy((x @ w.T + bias).astype(np.float32)).to(out).float().numpy()
    whole, y = guarded(M * N, out)
    dmm.f8_matmul(dev(xc), dev(xs), M, K, dev(wc), dev(ws), N, y, bias=dev(bias))
    assert np.array_equal(host(y).reshape(M, N), ref) and intact(whole)


def test_unaligned_results(dmm):
    """y at an address of its type only, and rows that are no whole pieces."""
    say("f8_matmul y of any alignment")
    rng = np.random.default_rng(0)
    for M, N, K in ((2, 40, 200), (50, 72, 300), (900, 904, 130), (1500, 2104, 130), (4100, 2992, 130)):
        xc, xs, x = random_package(rng, M, K, 1, exact=True)
        wc, ws, w = random_package(rng, N, K, 128, exact=True)
        ref = torch.from_numpy((x @ w.T).astype(np.float32))
        for out in (torch.float32, torch.bfloat16):
            y = torch.full((M * N + 9,), 7.0, dtype=out, device=DEV)
            dmm.f8_matmul(dev(xc), dev(xs), M, K, dev(wc), dev(ws), N, y[1:1 + M * N])
            got = host(y)
            assert np.array_equal(got[1:1 + M * N].reshape(M, N), ref.to(out).float().numpy())
            assert got[0] == 7 and (got[1 + M * N:] == 7).all()


# M, N, K, E, top_k: streaming (few slots), 64 x 128, 128 x 128
LISTS = [(5, 40, 300, 8, 2), (9, 70, 9000, 3, 2), (60, 200, 700, 4, 3), (100, 130, 2000, 7, 4), (300, 300, 100, 5, 2),
         (700, 140, 900, 4, 2), (500, 260, 1300, 3, 3), (1000, 129, 200, 2, 1), (40, 33, 130, 512, 8)]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,E,top_k", LISTS, ids=["x".join(map(str, f)) for f in LISTS])
def test_lists(dmm, M, N, K, E, top_k, out):
    """Uneven lists, experts of none, slots of none, and the same expert twice."""
    say(f"f8_matmul_experts form M={M} N={N} K={K} E={E} top_k={top_k} {out}")
    rng = np.random.default_rng(M + N + K)
    xc, xs, x = random_package(rng, M, K, 1, exact=True)
    made = [random_package(rng, N, K, 128, exact=True) for _ in range(E)]
    ids = np.minimum((rng.random((M, top_k)) ** 2 * (E + 0.5)).astype(np.int32) - 0, E)     # E: of no expert
    ids[M // 2:M // 2 + 3] = 0
    _, offsets, order = oracle.moe_route(ids, E)
    whole, y = guarded(M * top_k * N, out)
    dmm.f8_matmul_experts(dev(xc), dev(xs), M, K, dev(np.stack([m[0] for m in made])),
                          dev(np.stack([m[1] for m in made])), N, y, E, dev(offsets), dev(order), top_k)
    got = host(y).reshape(M, top_k, N)
    assert intact(whole)
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if len(t):
            ref = torch.from_numpy((x[t] @ made[e][2].T).astype(np.float32)).to(out).float().numpy()
            assert np.array_equal(got[t, j], ref), f"expert {e}"
    assert np.isnan(got[ids == E]).all()


# More tiles of an expert than share W, the last group cut; more experts than a workgroup has threads.
LONG_LISTS = [(3000, 300, 130, 2, 2), (2100, 140, 640, 1, 1), (1300, 500, 200, 3, 3), (520, 40, 130, 512, 8),
              (4100, 40, 64, 512, 8)]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,E,top_k", LONG_LISTS, ids=["x".join(map(str, f)) for f in LONG_LISTS])
def test_long_lists(dmm, M, N, K, E, top_k, out):
    test_lists(dmm, M, N, K, E, top_k, out)


def test_second_product_of_the_experts(dmm):
    """Every slot with its own activations: M top_k tokens, top_k 1, the same lists."""
    say("f8_matmul_experts by slots")
    M, N, K, E, top_k = 90, 150, 400, 4, 3
    rng = np.random.default_rng(4)
    xc, xs, x = random_package(rng, M * top_k, K, 1)
    made = [random_package(rng, N, K, 128) for _ in range(E)]
    ids = rng.integers(0, E, (M, top_k)).astype(np.int32)
    _, offsets, order = oracle.moe_route(ids, E)
    y = torch.zeros((M, top_k, N), dtype=torch.bfloat16, device=DEV)
    dmm.f8_matmul_experts(dev(xc), dev(xs), M * top_k, K, dev(np.stack([m[0] for m in made])),
                          dev(np.stack([m[1] for m in made])), N, y, E, dev(offsets), dev(order), 1)
    got = host(y).reshape(-1, N)
    for e in range(E):
        at = np.nonzero(ids.ravel() == e)[0]
        ref, B = oracle.f8_matmul(x[at], made[e][2])
        assert_close(got[at], ref, B, K, torch.bfloat16, f"expert {e}", dropped(x[at], made[e][2]) * (1 + 2.0 ** -8))


def test_scales_at_their_ends(dmm):
    """Scales whose products fp32 still holds, and a zero scale."""
    say("f8_matmul scales at their ends")
    rng = np.random.default_rng(8)
    N, K = 40, 300
    for M in (1, 4, 50):
        xc, xs, _ = random_package(rng, M, K, 1)
        wc, ws, _ = random_package(rng, N, K, 128)
        clean = [c.reshape(c.shape[0], -1).copy() for c in (xc, wc)]
        for c in clean:
            c[:, K:] = 0
        for a, b in ((2.0 ** -126, 1.0), (2.0 ** 60, 2.0 ** 40), (2.0 ** 100, 2.0 ** -120), (0.0, 1.0)):
            xs2, ws2 = (xs * np.float32(a)).astype(np.float32), (ws * np.float32(b)).astype(np.float32)
            if a == 2.0 ** -126:
                xs2 = np.maximum(xs2, np.float32(2.0 ** -126))
                ws2 = np.maximum(ws2, np.float32(1.0))
            x, w = oracle.f8_unpack(clean[0].reshape(xc.shape), xs2, K, 1), oracle.f8_unpack(clean[1].reshape(wc.shape), ws2, K, 128)
            y = torch.full((M, N), 7.0, device=DEV)
            dmm.f8_matmul(dev(xc), dev(xs2), M, K, dev(wc), dev(ws2), N, y)
            ref, B = oracle.f8_matmul(x, w)
            assert_close(host(y), ref, B, K, torch.float32, f"scales {a} {b}")


# ------------------------------------------- graphs, streams, two at once


def layer(dmm, s):
    """One pass through an expert layer on the buffers of s, gradients included."""
    M, E, k, H, K = s["M"], s["E"], s["k"], s["H"], s["K"]
    dmm.f8_norm_pack(s["x"], s["w"], s["xc"], s["xs"], 1e-6, residual=s["res"], h_out=s["h"], y_out=s["y"])
    torch.mm(s["y"].float(), s["router"], out=s["logits"])
    dmm.moe_gate(s["logits"], s["ids"], s["weights"], score="sigmoid", bias=s["bias"], n_groups=4, top_groups=2,
                 group_top=2, scale=2.5)
    dmm.moe_route(s["ids"], E, s["counts"], s["offsets"], s["order"], workspace=s["ws"])
    dmm.f8_matmul_experts(s["xc"], s["xs"], M, K, s["wc"], s["wsc"], H, s["rows"], E, s["offsets"], s["order"], k)
    dmm.moe_combine(s["rows"], s["ids"], s["weights"], E, s["out"], add=s["h"])
    dmm.moe_combine_grad(s["rows"], s["ids"], s["weights"], E, s["dout"], s["drows"], s["dweights"])
    dmm.moe_gate_grad(s["logits"], s["ids"], s["dweights"], s["dlogits"], score="sigmoid", scale=2.5)


def made_layer(dmm, M, seed):
    K = H = 384
    E, k = 16, 4
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=DEV).to(dtype)

    bf = torch.bfloat16
    s = {"M": M, "E": E, "k": k, "H": H, "K": K, "x": randn(M, K, dtype=bf), "res": randn(M, K, dtype=bf),
         "w": 1 + 0.1 * randn(K), "h": torch.empty((M, K), dtype=bf, device=DEV), "bias": 0.05 * randn(E),
         "y": torch.empty((M, K), dtype=bf, device=DEV), "router": randn(K, E) * 0.05,
         "logits": torch.empty((M, E), device=DEV), "ids": torch.empty((M, k), dtype=torch.int32, device=DEV),
         "weights": torch.empty((M, k), device=DEV), "counts": torch.empty(E, dtype=torch.int32, device=DEV),
         "offsets": torch.empty(E + 1, dtype=torch.int32, device=DEV),
         "order": torch.empty(M * k, dtype=torch.int32, device=DEV),
         "rows": torch.empty((M, k, H), dtype=bf, device=DEV), "out": torch.empty((M, H), dtype=bf, device=DEV),
         "dout": randn(M, H, dtype=bf), "drows": torch.empty((M, k, H), dtype=bf, device=DEV),
         "dweights": torch.empty((M, k), device=DEV), "dlogits": torch.empty((M, E), device=DEV)}
    s["ws"] = torch.empty(max(1, dmm.moe_route_workspace_bytes(M, k, E)), dtype=torch.uint8, device=DEV)
    cs, ss = dmm.f8_shape(M, K)
    s["xc"], s["xs"] = torch.empty(cs, dtype=torch.uint8, device=DEV), torch.empty(ss, device=DEV)
    cs, ss = dmm.f8_shape(H, K, 128)
    s["wc"], s["wsc"] = torch.empty((E, *cs), dtype=torch.uint8, device=DEV), torch.empty((E, *ss), device=DEV)
    for e in range(E):
        dmm.f8_pack(randn(H, K) * 0.05, s["wc"][e], s["wsc"][e], 128)
    return s


OUT = ("h", "xc", "xs", "y", "ids", "weights", "order", "rows", "out", "drows", "dweights", "dlogits")


def outputs(s):
    return {n: s[n].view(torch.uint8).clone() if s[n].dtype != torch.uint8 else s[n].clone() for n in OUT}


def same(a, b):
    return [n for n in OUT if not torch.equal(a[n], b[n])]


@pytest.mark.parametrize("M", [1, 16, 200])
def test_expert_layer(dmm, M):
    """The whole pass against the oracle, each step on what the step before gave."""
    say(f"expert layer M={M}")
    s = made_layer(dmm, M, M)
    layer(dmm, s)
    E, k, H, K = s["E"], s["k"], s["H"], s["K"]

    def store(v):
        return torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16).float().numpy()

    h, y = oracle.f8_norm(host(s["x"]) + host(s["res"]), None, host(s["w"]), 1e-6, store)
    assert np.array_equal(host(s["h"]), h) and np.array_equal(host(s["y"]), store(y))
    c, sc, _ = oracle.f8_pack(y, 1)
    assert np.array_equal(host(s["xc"]), c) and np.array_equal(host(s["xs"]), sc)
    z = host(s["logits"])
    ids, w = oracle.moe_gate(z, k, "sigmoid", host(s["bias"]), 4, 2, 2, True, 2.5)
    assert np.array_equal(host(s["ids"]), ids)
    r = (np.abs(z).max(axis=1) + 32)[:, None] * 2.0 ** -23
    assert (np.abs(host(s["weights"]) - w) <= r * w).all()
    for got, ref in zip((s["counts"], s["offsets"], s["order"]), oracle.moe_route(ids, E)):
        assert np.array_equal(host(got), ref)
    rows = host(s["rows"])
    x = oracle.f8_unpack(c, sc, K, 1)
    tiled = M * k >= 8 * E
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if len(t):
            we = oracle.f8_unpack(host(s["wc"])[e], host(s["wsc"])[e], K, 128)
            ref, B = oracle.f8_matmul(x[t], we)
            assert_close(rows[t, j], ref, B, K, torch.bfloat16, f"expert {e}", dropped(x[t], we) * (1 + 2.0 ** -8) if tiled else 0)
    wt = host(s["weights"]).astype(np.float64)
    ref, B = oracle.moe_combine(rows.astype(np.float64), ids, wt, E, h.astype(np.float64))
    assert (np.abs(host(s["out"]) - ref) <= (k + 1) * 2.0 ** -24 * B + 2.0 ** -8 * np.abs(ref)).all()
    dout = host(s["dout"]).astype(np.float64)
    rdy, rdw, B = oracle.moe_combine_grad(rows.astype(np.float64), ids, wt, E, dout)
    assert (np.abs(host(s["drows"]) - rdy) <= 2.0 ** -8 * np.abs(rdy) * (1 + 2.0 ** -20)).all()
    assert (np.abs(host(s["dweights"]) - rdw) <= (H + 16) * 2.0 ** -24 * B).all()
    dw = host(s["dweights"])
    dz = oracle.moe_gate_grad(z, ids, dw, "sigmoid", True, 2.5)
    # r (3 |d| + 3 mean |d| + 4 r max) of the weights, each at most twice the largest |dw| apart
    assert (np.abs(host(s["dlogits"]) - dz) <= 2.5 * r * 14 * np.abs(dw).max(axis=1, keepdims=True) + 2.0 ** -24 * np.abs(dz)).all()


@pytest.mark.parametrize("M", [1, 16, 200])
def test_layer_in_a_graph(dmm, M):
    """Captured once and replayed on other inputs, eager work and synchronizations in between;
    an eager pass over the same inputs gives the same bits."""
    say(f"expert layer in a graph M={M}")
    s, eager = made_layer(dmm, M, 5), made_layer(dmm, M, 5)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        layer(dmm, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        layer(dmm, s)
    for i in range(4):
        for n in ("x", "res", "dout"):
            new = torch.randn((M, s["K"]), device=DEV).to(torch.bfloat16)
            s[n].copy_(new)
            eager[n].copy_(new)
        graph.replay()
        layer(dmm, eager)
        torch.cuda.synchronize()
        assert not same(outputs(s), outputs(eager)), i


def test_two_layers_at_once(dmm):
    """Two streams, each with its own buffers, against one after the other."""
    say("two expert layers at once")
    a, b = made_layer(dmm, 200, 1), made_layer(dmm, 48, 2)
    layer(dmm, a)
    layer(dmm, b)
    torch.cuda.synchronize()
    want = outputs(a), outputs(b)
    for s in (a, b):
        for n in OUT:
            s[n].zero_()
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(one):
            layer(dmm, a)
        with torch.cuda.stream(two):
            layer(dmm, b)
    torch.cuda.synchronize()
    assert not same(outputs(a), want[0]) and not same(outputs(b), want[1])


# --------------------------------------------------- offsets past 32 bits


def test_large_weights(dmm):
    """A package of 4.3 GB: the last rows of W, by a token's kernel, the streaming one and tiles."""
    say("f8_matmul of 4.3 GB")
    N, K = 33000, 131072
    codes = torch.zeros((N, K // 128, 128), dtype=torch.uint8, device=DEV)
    scales = torch.ones((-(-N // 128), K // 128), device=DEV)
    rng = np.random.default_rng(0)
    tail = 300
    wc, ws, w = random_package(rng, tail, K, 128, exact=True)
    ws[:] = 1
    w = oracle.f8_unpack(wc, ws, K, 128)
    codes[N - tail:] = dev(wc)
    for M in (1, 3, 40):
        xc, xs, x = random_package(rng, M, K, 1, exact=True)
        y = torch.full((M, N), 7.0, device=DEV)
        dmm.f8_matmul(dev(xc), dev(xs), M, K, codes, scales, N, y)
        assert np.array_equal(host(y[:, N - tail:]), (x @ w.T).astype(np.float32))
        assert not host(y[:, :N - tail]).any()


def test_large_rows_of_the_experts(dmm):
    """4.3 G values of y: the last tokens, forward and back."""
    say("moe_combine of 8.6 GB")
    M, top_k, N, E = 65600, 8, 8192, 8
    y = torch.zeros((M, top_k, N), dtype=torch.bfloat16, device=DEV)
    ids = torch.randint(0, E, (M, top_k), dtype=torch.int32, device=DEV)
    w = torch.rand((M, top_k), device=DEV)
    y[-2:] = torch.randn((2, top_k, N), device=DEV).to(torch.bfloat16)
    tail = y[-2:].clone()
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    dmm.moe_combine(y, ids, w, E, out)
    t, ww = tail.double().cpu().numpy(), host(w[-2:]).astype(np.float64)
    ref, B = oracle.moe_combine(t, host(ids[-2:]), ww, E)
    assert (np.abs(host(out[-2:]) - ref) <= 9 * 2.0 ** -24 * B + 2.0 ** -8 * np.abs(ref)).all()
    assert not out[:-2].any().item()
    dout = torch.randn((M, N), device=DEV).to(torch.bfloat16)
    dw = torch.full((M, top_k), 7.0, device=DEV)
    dmm.moe_combine_grad(y, ids, w, E, dout, y, dw)                # in place
    rdy, rdw, B = oracle.moe_combine_grad(t, host(ids[-2:]), ww, E, dout[-2:].double().cpu().numpy())
    assert (np.abs(host(y[-2:]) - rdy) <= 2.0 ** -8 * np.abs(rdy) * (1 + 2.0 ** -20)).all()
    assert (np.abs(host(dw[-2:]) - rdw) <= (N + 16) * 2.0 ** -24 * B).all() and not dw[:-2].any().item()
