"""Tokens that moe_gate takes again in float64, against the float64 oracle."""

import numpy as np
import pytest

import oracle
from test_gpu_gate import gate, spread
from test_gpu_mx import say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dmm():
    import decode_matmul_amd
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return decode_matmul_amd


@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_groups,top_groups", [(64, 8, 3), (256, 8, 4), (128, 16, 5), (24, 3, 2), (512, 4, 2)])
def test_groups_that_alone_ask_for_float64(dmm, E, n_groups, top_groups, score, biased):
    """A group without experts, or with one only, sends its token to float64 from that group's lanes; the token's
    other lanes agree.  The other experts lie where fp32 and float64 order them differently."""
    say(f"moe_gate again E={E} groups={n_groups} {score} {biased}")
    rng = np.random.default_rng(E + n_groups)
    M, top_k, size = 500, 6, E // n_groups
    z = (rng.standard_normal((M, 1)) + rng.integers(-3, 4, (M, E)) * 2.0 ** -22).astype(np.float32)
    for t in range(M):
        g = rng.integers(0, n_groups)
        z[t, g * size + t % 2:(g + 1) * size] = -np.inf
    bias = (rng.integers(-2, 3, E) * 2.0 ** -25).astype(np.float32) if biased else None
    for renorm in (True, False):
        kw = dict(score=score, n_groups=n_groups, top_groups=top_groups, group_top=2, renorm=renorm)
        ids, w = gate(dmm, z, top_k, torch.float32, bias, **kw)
        rids, rw = oracle.moe_gate(z, top_k, bias=bias, **kw)
        assert np.array_equal(ids, rids)
        assert (np.abs(w - rw) <= spread(z, score)[:, None] * np.abs(rw)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_groups,group_top", [(16, 1, 1), (64, 1, 1), (512, 1, 1), (64, 4, 1), (256, 8, 2)])
def test_biases_of_any_magnitude(dmm, E, n_groups, group_top, score):
    """Biases from 2^18 to 2^127 of both signs, equal ones among them: fp32 does not see the scores beside
    them, float64 does up to 2^53, and the margin of near keys, which grows with them, stays below 2^31."""
    say(f"moe_gate large biases E={E} groups={n_groups} {score}")
    rng = np.random.default_rng(E + n_groups)
    M, top_k = 40, 6
    z = rng.standard_normal((M, E)).astype(np.float32)
    for power in (18, 22, 25, 27, 28, 29, 30, 31, 33, 36, 40, 50, 60, 127):
        for sign in (1, -1):
            bias = (sign * 2.0 ** power * (1 - rng.integers(0, 3, E) * 2.0 ** -23)).astype(np.float32)
            kw = dict(score=score, n_groups=n_groups, top_groups=max(1, n_groups // 2), group_top=group_top)
            ids, w = gate(dmm, z, top_k, torch.float32, bias, **kw)
            with np.errstate(over="ignore"):
                rids, rw = oracle.moe_gate(z, top_k, bias=bias, **kw)
            assert np.array_equal(ids, rids), power
            assert (np.abs(w - rw) <= spread(z, score)[:, None] * np.abs(rw)).all()
