"""Lists and windows of whole prompts: more tokens than one launch plans (512), so
that later launches begin at other tokens of the lists, against the float64 oracle
on both sides of every seam and at steps between."""
import pytest

from kv8_cases import KVCase
from oracle import kv8
from test_kv_attn_gpu import _lib, compare, run  # noqa: F401

pytestmark = pytest.mark.gpu


def tokens(T):
    seams = [t for s in range(512, T, 512) for t in (s - 2, s - 1, s, s + 1)]
    return sorted({t for t in (0, 1, T - 2, T - 1, *seams, *range(0, T, 61)) if t < T})


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
@pytest.mark.parametrize("raw,ql,ratio,H,K", [([1500], [1500], 1, 64, 300), ([900, 400, 333], [700, 400, 1], 2, 128, 65),
                                              ([513], [513], 2, 5, 64), ([2100], [2100], 1, 20, 130)])
def test_lists(raw, ql, ratio, H, K, quant):
    case = KVCase(181 + H, raw, ql, ratio, H, quant, K=K)
    # some tokens of every launch list nothing
    case.indices[3::97] = -1
    compare(case, run(case), tokens=tokens(case.T))


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
@pytest.mark.parametrize("raw,ql,ratio,H,window", [([1500], [1500], 1, 64, 128), ([900, 700], [600, 700], 2, 33, 50),
                                                   ([1030], [1030], 1, 128, 300)])
def test_windows(raw, ql, ratio, H, window, quant):
    case = KVCase(191 + H, raw, ql, ratio, H, quant)
    compare(case, run(case, window=window), window=window, tokens=tokens(case.T))
