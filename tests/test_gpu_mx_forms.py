"""Every kernel of the MXFP4 products against sums in 64 bits, to the last bit.

x is whole numbers of -8 .. 8 (in MXFP4: of e2m1 values, scales 1), weights are
e2m1 values times 1/2, 1 or 2 and the bias whole numbers of -50 .. 50.  Every
product is then a whole multiple of 1/4 (1/8), and sums stay below
9000 * 8 * 12 + 50 < 2^20 (the longest rows have 400 products), so that no fp32
addition rounds, in any order: fp32 results are equal, a column left out or
taken twice shows, and bf16 results are the nearest to the sum.
"""

import numpy as np
import pytest

import mx_forms

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module")
def dmm():
    import decode_matmul_amd
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return decode_matmul_amd


def say(msg):
    print(f"[case] {msg}", flush=True)


def seeded(*sizes):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(sum(int(s) * 31 ** i for i, s in enumerate(sizes)))
    return gen


def package(gen, rows, K, spread, offset=0, keep=None):
    """codes, scales (`offset` bytes into their buffer) and the values [rows, K], float64;
    with keep (columns), only those are not 0 and only they are returned."""
    nb = -(-K // 32)
    v = torch.zeros((rows, nb * 32), dtype=torch.uint8, device=DEV)
    if keep is None:
        v[:, :K] = torch.randint(0, 16, (rows, K), dtype=torch.uint8, generator=gen, device=DEV)
    else:
        v[:, keep] = torch.randint(0, 16, (rows, len(keep)), dtype=torch.uint8, generator=gen, device=DEV)
    codes = (v[:, 0::2] | (v[:, 1::2] << 4)).view(rows, nb, 16)
    buf = torch.zeros(rows * nb + offset, dtype=torch.uint8, device=DEV)
    scales = buf[offset:].view(rows, nb)
    scales.copy_(torch.randint(127 - spread, 128 + spread, (rows, nb), dtype=torch.uint8, generator=gen, device=DEV))
    at = torch.arange(K, device=DEV) if keep is None else keep
    grid = torch.tensor(E2M1 + [-e for e in E2M1], dtype=torch.float64, device=DEV)
    return codes, scales, grid[v[:, at].long()] * torch.exp2(scales[:, at // 32].double() - 127)


def whole_numbers(gen, M, K, ld, aligned):
    """bf16 x [M, K], rows ld apart, NaN between them, maybe one element into its buffer."""
    first = 0 if aligned else 1
    buf = torch.full((M * ld + first + 8,), float("nan"), dtype=torch.bfloat16, device=DEV)
    x = buf[first:].as_strided((M, K), (ld, 1), first)
    x.copy_(torch.randint(-8, 9, (M, K), generator=gen, device=DEV).to(torch.bfloat16))
    return x


def output(n, dtype):
    whole = torch.full((n + 512,), 7.0, dtype=dtype, device=DEV)
    return whole, whole[256:256 + n]


def intact(whole):
    return bool((whole[:256] == 7).all() and (whole[-256:] == 7).all())


def bias_of(gen, *shape):
    return torch.randint(-50, 51, shape, generator=gen, device=DEV).float()


@pytest.mark.parametrize("case", mx_forms.DENSE, ids=["x".join(map(str, c)) for c in mx_forms.DENSE])
def test_dense(dmm, case):
    M, N, K, mx, aligned = case
    say(f"{mx_forms.dense_cases_form(*case)} {case}")
    gen = seeded(M, N, K)
    codes, scales, w = package(gen, N, K, 1, 0 if aligned or not mx else 1)
    bias = bias_of(gen, N)
    if mx:
        xc, xs, x = package(gen, M, K, 0, 0 if aligned else 3)
    else:
        X = whole_numbers(gen, M, K, mx_forms._ld(K, aligned), aligned)
        x = X.double()
    ref = torch.matmul(x, w.t().contiguous()) + bias.double()
    for dtype in (torch.float32, torch.bfloat16):
        whole, y = output(M * N, dtype)
        if mx:
            dmm.mx_matmul_mx(xc, xs, M, K, codes, scales, N, y, bias=bias)
        else:
            dmm.mx_matmul(X, codes, scales, N, y, bias=bias)
        assert torch.equal(y.view(M, N), ref.float().to(dtype)) and intact(whole), dtype


def routed(dmm, ids, E):
    M, top_k = ids.shape
    counts, offsets, order = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (E, E + 1, M * top_k))
    nbytes = dmm.moe_route_workspace_bytes(M, top_k, E)
    dmm.moe_route(ids, E, counts, offsets, order,
                  workspace=torch.empty(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None)
    return offsets, order


@pytest.mark.parametrize("case", mx_forms.EXPERTS, ids=["x".join(map(str, c)) for c in mx_forms.EXPERTS])
def test_experts(dmm, case):
    """Uneven lists: a third of the tokens go to one expert, some experts get
    none, some slots have none."""
    M, N, K, E, top_k, direct, aligned = case
    say(f"{mx_forms.experts_cases_form(*case)} {case}")
    gen = seeded(M, N, K, E)
    codes, scales, w = package(gen, E * N, K, 1)
    w = w.view(E, N, K)
    X = whole_numbers(gen, M, K, mx_forms._ld(K, direct), aligned)
    bias = bias_of(gen, E, N)
    ids = torch.randint(0, E, (M, top_k), dtype=torch.int32, generator=gen, device=DEV)
    ids[: M // 3] = E - 1
    ids[ids == E // 2] = 0
    ids[torch.rand((M, top_k), generator=gen, device=DEV) < 0.1] = -1
    offsets, order = routed(dmm, ids, E)
    ref = torch.full((M, top_k, N), float("nan"), dtype=torch.float64, device=DEV)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            ref[t, j] = torch.matmul(X[t].double(), w[e].t().contiguous()) + bias[e].double()
    for dtype in (torch.float32, torch.bfloat16):
        whole, y = output(M * top_k * N, dtype)
        dmm.mx_matmul_experts(X, codes, scales, N, y, E, offsets, order, top_k, bias=bias)
        got = y.view(M, top_k, N)
        assert torch.equal(torch.isnan(got), torch.isnan(ref)) and intact(whole), dtype
        assert torch.equal(got.nan_to_num(0), ref.float().to(dtype).nan_to_num(0)), dtype


@pytest.mark.parametrize("M", [3, 40, 300])
def test_experts_empty_sums(dmm, M):
    """K = 0: the bias alone, and NaN rows where there is no expert."""
    say(f"experts K=0 M={M}")
    E, N = 4, 40
    gen = seeded(M)
    ids = torch.randint(-1, E, (M, 1), dtype=torch.int32, generator=gen, device=DEV)
    offsets, order = routed(dmm, ids, E)
    bias = bias_of(gen, E, N)
    u8 = dict(dtype=torch.uint8, device=DEV)
    for b, rows in ((bias, bias), (None, torch.zeros_like(bias))):
        whole, y = output(M * N, torch.float32)
        dmm.mx_matmul_experts(torch.empty((M, 0), dtype=torch.bfloat16, device=DEV), torch.empty((E * N, 0, 16), **u8),
                              torch.empty((E * N, 0), **u8), N, y, E, offsets, order, 1, bias=b)
        got, e = y.view(M, N), ids[:, 0].long()
        assert torch.equal(got[e >= 0], rows[e[e >= 0]]) and torch.isnan(got[e < 0]).all() and intact(whole)


@pytest.mark.parametrize("case", mx_forms.LONG, ids=["x".join(map(str, c)) for c in mx_forms.LONG])
def test_long_rows(dmm, case):
    """Rows past what the tiles take: 2^23 columns, x not 0 in 400 of them."""
    M, N, K, mx, E = case
    say(f"long rows {case}")
    gen = seeded(M, N, K)
    at = torch.unique(torch.cat((torch.randint(0, K, (392,), generator=gen, device=DEV), torch.arange(K - 8, K, device=DEV))))
    rows = N * max(E, 1)
    codes, scales, w = package(gen, rows, K, 1, keep=at)
    whole, y = output(M * N, torch.float32)
    if mx:
        xc, xs, x = package(gen, M, K, 0, keep=at)
        dmm.mx_matmul_mx(xc, xs, M, K, codes, scales, N, y)
        ref = x @ w.t().contiguous()
    else:
        X = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
        X[:, at] = torch.randint(-8, 9, (M, len(at)), generator=gen, device=DEV).to(torch.bfloat16)
        x = X[:, at].double()
        if E:
            ids = torch.randint(0, E, (M, 1), dtype=torch.int32, generator=gen, device=DEV)
            offsets, order = routed(dmm, ids, E)
            dmm.mx_matmul_experts(X, codes, scales, N, y, E, offsets, order, 1)
            ref = torch.matmul(x[:, None, :], w.view(E, N, -1).transpose(1, 2).contiguous()[ids[:, 0].long()])[:, 0]
        else:
            dmm.mx_matmul(X, codes, scales, N, y)
            ref = x @ w.t().contiguous()
    assert torch.equal(y.view(M, N), ref.float()) and intact(whole)
