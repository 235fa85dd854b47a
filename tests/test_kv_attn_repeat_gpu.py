"""The attention over 8-bit KV rows with many units per CTA: the same call gives
the same bits every time, and every token agrees with the float64 oracle. Groups
of softmax warps run at their own pace there, up to a unit apart."""
import numpy as np
import pytest

from kv8_cases import KVCase
from oracle import kv8

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(512.0)

CASES = [
    # name, raw lengths, query lengths, ratio, H, K, code type, tokens checked
    ("listed", [9000] * 16, [4] * 16, 1, 64, 2048, kv8.FP8, range(0, 64, 7)),
    ("dense", [20000, 17001], [24, 17], 2, 64, None, kv8.INT8, range(0, 41, 6)),
    ("few-heads", [15001], [60], 1, 24, None, kv8.FP8, range(0, 60, 9)),
]


@pytest.mark.parametrize("p", CASES, ids=[p[0] for p in CASES])
def test_many_units_per_cta(p):
    import torch

    from sparse_attention_indexer_qli_gb300 import qli
    from test_kv_attn_gpu import compare
    _, raw, ql, ratio, H, K, quant, tokens = p
    case = KVCase(91, raw, ql, ratio, H, quant, K=K)
    kw = case.upload()
    first = None
    for _ in range(25):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = qli.kv_attention(scale=SCALE, err_word=err, **kw)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        if first is None:
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    compare(case, (first[0].float().cpu().numpy().astype(np.float64),
                   first[1].cpu().numpy().astype(np.float64)), tokens=tokens)
