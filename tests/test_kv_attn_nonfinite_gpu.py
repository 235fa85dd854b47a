"""Queries that are not finite: a token without positions gives 0 and -inf whatever
its queries hold (padding tokens' are not written), and one with positions gives
NaN in the heads concerned and nowhere else."""
import numpy as np
import pytest

from kv8_cases import KVCase
from oracle import kv8
from test_kv_attn_gpu import _lib, compare, run  # noqa: F401

pytestmark = pytest.mark.gpu

NAN, INF = 0x7FC0, 0x7F80


def spoil(case, tokens):
    """Every head of a third of the tokens, one value in some heads of the others."""
    for n, t in enumerate(tokens):
        if n % 3 == 0:
            case.q[t] = NAN
        else:
            case.q[t, ::3, 7 * n % 512] = [INF, 0xFF80, NAN][n % 3]


QUANTS = pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])


@QUANTS
@pytest.mark.parametrize("B,K,H", [(7, 40, 64), (7, 500, 64), (200, 130, 33), (3, 2048, 128)])
def test_empty_lists(B, K, H, quant):
    case = KVCase(161 + K, [900] * B, [1] * B, 1, H, quant, K=K)
    gone = list(range(1, B, 2))
    case.indices[gone] = -1
    spoil(case, gone)
    compare(case, run(case))


@QUANTS
def test_tokens_that_see_nothing(quant):
    # raw length 1 at ratio 2 has no compressed position; so have a prompt's first
    # queries, and a token that no request covers
    import torch
    for window in (0, 100):
        case = KVCase(162, [1, 600, 3, 0], [1, 1, 3, 0], 2, 64, quant)
        spoil(case, [0, 2])
        compare(case, run(case, window=window), window=window)
    case = KVCase(163, [400, 300], [1, 1], 2, 64, quant)
    case.q[1] = NAN
    o, lse = run(case, err_want=1, cu_seqlens_q=torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda"))
    compare(case, (o, lse), tokens=[0])
    assert not o[1].any() and np.all(np.isneginf(lse[1]))


@QUANTS
@pytest.mark.parametrize("T,K", [(1, 2048), (3, 700), (160, 500)])
def test_lists_with_one_position(T, K, quant):
    """NaN in the heads that have it, although most units hold no position; units
    without positions go to CTAs of their own when the tokens are few."""
    case = KVCase(164 + T, [3000] * T, [1] * T, 1, 64, quant, K=K)
    want = case.q.copy()
    case.indices[:] = -1
    for t in range(T):
        case.indices[t, 0, (t * 97 + K - 1) % K] = t
    case.q[:, ::3, 5] = NAN
    o, lse = run(case)
    assert np.isnan(o[:, ::3]).all() and np.isnan(lse[:, ::3]).all()
    keep = np.arange(64) % 3 != 0
    case.q = want
    o[:, ~keep], lse[:, ~keep] = 0, 0
    for t in range(T):
        js = case.positions(t)
        z = kv8.bf16_to_f64(case.q[t]) @ case.kv(t, js)[0] / np.sqrt(512.0)
        # one position: its value, and its score (512 FP32 terms: 2^-14 of the magnitudes)
        assert np.all(np.abs(o[t][keep] - case.kv(t, js)) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(case.kv(t, js)))
        size = np.abs(kv8.bf16_to_f64(case.q[t])) @ np.abs(case.kv(t, js)[0]) / np.sqrt(512.0)
        assert np.all(np.abs(lse[t] - z)[keep] <= (size * 2.0 ** -13 + 2.0 ** -20 * (1 + np.abs(z)))[keep])


@QUANTS
def test_positions_with_a_whole_query_of_nan(quant):
    case = KVCase(165, [5000, 700, 90], [1, 2, 1], 1, 64, quant)
    case.q[0], case.q[2] = NAN, NAN
    for window in (0, 100):
        o, lse = run(case, window=window)
        for t in (0, 2):
            assert np.isnan(o[t]).all() and np.isnan(lse[t]).all()
        compare(case, (o, lse), tokens=[1, 3], window=window)
