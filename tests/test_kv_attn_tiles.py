"""Row tiles of fewer heads and the launch's plan, in the attention over 8-bit KV
rows: small calls split the heads over more CTAs, and the plan reads the requests
through a copy on the chip while they fit there."""
import numpy as np
import pytest

from kv8_cases import KVCase
from oracle import kv8

SMS = 152


def heads_per_tile(T, H, most, sms):
    ht = 64
    while ht > 16 and (1 if most <= 2 else most) * T * -(-H // (ht // 2)) <= sms:
        ht //= 2
    return ht


def test_tiles_cover_the_heads_and_have_an_sm_per_unit():
    for H in range(1, 129):
        for T in (1, 2, 7, 64, 300):
            for most in (1, 2, 3, 8, 40):
                ht = heads_per_tile(T, H, most, SMS)
                tiles = -(-H // ht)
                seen = [g * ht + r for g in range(tiles) for r in range(64) if r < ht and g * ht + r < H]
                assert seen == list(range(H))
                if ht < 64:
                    assert tiles * T * (1 if most <= 2 else most) <= SMS
    assert heads_per_tile(1, 64, 8, SMS) == 16      # 4 tiles of 8 units
    assert heads_per_tile(64, 32, 2, SMS) == 16     # 128 uncut tiles
    assert heads_per_tile(1, 64, 32, SMS) == 16     # 128 units
    assert heads_per_tile(1, 128, 32, SMS) == 32
    assert heads_per_tile(64, 64, 32, SMS) == 64


def _check(case, window=0):
    from test_kv_attn_gpu import compare, run
    compare(case, run(case, window=window), window=window)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
@pytest.mark.parametrize("T,H,K", [(1, 64, 512), (1, 128, 2048), (1, 100, 500), (3, 40, 1000), (6, 33, 700),
                                   (2, 16, 130), (2, 65, 64), (1, 17, 2000), (9, 128, 65)])
def test_few_tokens_over_lists(T, H, K, quant):
    _check(KVCase(61 + T + H, [4100] * T, [1] * T, 1, H, quant, K=K))


@pytest.mark.gpu
@pytest.mark.parametrize("raw,ql,H,window", [([700, 90], [2, 1], 48, 0), ([2000], [1], 128, 0),
                                             ([500] * 5, [1] * 5, 96, 100), ([333] * 9, [3] * 9, 30, 64)])
def test_few_tokens_over_visible_positions(raw, ql, H, window):
    _check(KVCase(71 + H, raw, ql, 2, H, kv8.INT8), window)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [639, 640, 700, 9999, 10001])
@pytest.mark.parametrize("listed", [False, True], ids=["dense", "listed"])
def test_many_requests(B, listed):
    """More requests than threads, and more than the plan's copy holds. Most have
    neither context nor tokens; the first and the last ones have both."""
    rng = np.random.default_rng(B)
    raw, ql = np.zeros(B, dtype=np.int64), np.zeros(B, dtype=np.int64)
    for b in [0, 1, 638, B - 2, B - 1] + rng.integers(0, B, 12).tolist():
        raw[b], ql[b] = int(rng.integers(3, 300)), int(rng.integers(1, 3))
    case = KVCase(81, raw, ql, 2, 20, kv8.FP8, K=70 if listed else None)
    _check(case)
