"""A wait of the attention of drafted trees that gives up, on the GPU and without a hang
(see test_kv_attn_timeout_gpu): every output is right or NaN, some are NaN, the call
reports QLI_DEVERR_TIMEOUT, and the next call of the normal build on the same memory is
right."""
import os
import time

import numpy as np
import pytest

from kv8_cases import attention_bounds
from oracle import kv8
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli
from test_kv_tree_gpu import SCALE, TreeCase

pytestmark = pytest.mark.gpu

STALL_DIR = os.path.join(os.path.dirname(libbuild.LIB), "stall")
DEVERR_TIMEOUT = 16


@pytest.fixture(scope="module")
def stall_lib():
    libbuild.build()
    qli.lib()
    return qli.lib(libbuild.build(out_dir=STALL_DIR,
                                  defines=("QLI_WAIT_LIMIT_NS=1000000ull", "QLI_TEST_STALL_EPILOGUE")))


CASES = [
    # name, positions, nodes, H, window
    ("single-few-tiles", [9000], [5], 64, 0),
    ("single-many-tiles", [900] * 12, [6] * 12, 64, 0),
    ("single-whole", [300] * 5, [4] * 5, 64, 100),
    ("groups-few-tiles", [9000], [16], 16, 0),
    ("groups-many-tiles", [1500] * 30, [9] * 30, 16, 0),
    ("groups-whole", [400] * 30, [9] * 30, 16, 100),
]


@pytest.mark.parametrize("p", CASES, ids=[p[0] for p in CASES])
def test_unfinished_outputs_are_nan(stall_lib, monkeypatch, p):
    import torch
    name, raw, nodes, H, window = p
    case = TreeCase(181, raw, nodes, H, kv8.FP8, "tree")
    kw = dict(case.upload(), window=window)
    T = case.T
    out = torch.full((T, H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 5.0, device="cuda")
    # what an earlier call may have left: finite pieces and log-sum-exps
    ws = torch.full((16 << 20,), 1.0, device="cuda").view(torch.uint8)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    with monkeypatch.context() as m:
        m.setattr(qli, "_lib", stall_lib)
        qli.kv_tree_attention(scale=SCALE, out=out, lse=lse, workspace=ws, err_word=err, **kw)
        torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    assert int(err.item()) == DEVERR_TIMEOUT
    o_g, l_g = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    lost = 0
    for t in range(T):
        q, kv = kv8.bf16_to_f64(case.q[t]), case.kv(case.request(t), case.positions(t, window))
        o, l = kv8.attend(q, kv, SCALE)
        do, dl = attention_bounds(q, kv, o, l, SCALE)
        for h in range(H):
            right = np.all(np.abs(o_g[t, h] - o[h]) <= do[h]) and abs(l_g[t, h] - l[h]) <= dl[h]
            gone = np.isnan(o_g[t, h]).all() and np.isnan(l_g[t, h])
            assert right or gone, (t, h)
            lost += int(gone)
    assert 0 < lost and (lost < T * H or "few" in name)
    # the normal build on the same workspace and outputs
    err.zero_()
    again = qli.kv_tree_attention(scale=SCALE, out=out, lse=lse, workspace=ws, err_word=err, **kw)
    want = qli.kv_tree_attention(scale=SCALE, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
