"""A wait of the 8-bit attention that gives up, on the GPU and without a hang: in
a test build of the library (short waits) one CTA's value products are never
issued. Its other warps give up in turn, the call returns and reports
QLI_DEVERR_TIMEOUT, and no output that needs this CTA's work looks like a result:
it is NaN, not what an earlier call left in the workspace or in the output.
The outputs of the other CTAs are right, and so is the next call of the normal
build on the same workspace."""
import os
import time

import numpy as np
import pytest

from kv8_cases import KVCase, attention_bounds
from oracle import kv8
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli

pytestmark = pytest.mark.gpu

# the same build as the one of the indexer's wait test
STALL_DIR = os.path.join(os.path.dirname(libbuild.LIB), "stall")
DEVERR_TIMEOUT = 16
SCALE = 512.0 ** -0.5


@pytest.fixture(scope="module")
def stall_lib():
    libbuild.build()
    qli.lib()
    return qli.lib(libbuild.build(out_dir=STALL_DIR,
                                  defines=("QLI_WAIT_LIMIT_NS=1000000ull", "QLI_TEST_STALL_EPILOGUE")))


CASES = [
    # name, raw lengths, query lengths, K, window, (token, head) that CTA 1 has no part in
    ("cut", [20000, 20000], [1, 1], None, 0, lambda t, h: t == 1),
    ("cut-listed", [3000] * 30, [1] * 30, 2048, 0, lambda t, h: t > 0),
    ("whole", [700] * 3, [1] * 3, None, 100, lambda t, h: (t, h // 16) != (0, 1)),
]


@pytest.mark.parametrize("p", CASES, ids=[p[0] for p in CASES])
def test_unfinished_outputs_are_nan(stall_lib, monkeypatch, p):
    import torch
    _, raw, ql, K, window, apart = p
    case = KVCase(171, raw, ql, 1, 64, kv8.FP8, K=K)
    kw = case.upload()
    if window:
        kw["window"] = window
    T = case.T
    out = torch.full((T, 64, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 64), 5.0, device="cuda")
    # what an earlier call may have left: finite pieces and log-sum-exps
    ws = torch.full((16 << 20,), 1.0, device="cuda").view(torch.uint8)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert ws.numel() >= qli.kv_attention_workspace_bytes(T, 64)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    with monkeypatch.context() as m:
        m.setattr(qli, "_lib", stall_lib)
        qli.kv_attention(scale=SCALE, out=out, lse=lse, workspace=ws, err_word=err, **kw)
        torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    assert int(err.item()) == DEVERR_TIMEOUT
    o_g, l_g = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    lost = 0
    for t in range(T):
        q, kv = kv8.bf16_to_f64(case.q[t]), case.kv(case.request(t), case.positions(t, window))
        o, l = kv8.attend(q, kv, SCALE)
        do, dl = attention_bounds(q, kv, o, l, SCALE)
        for h in range(64):
            right = np.all(np.abs(o_g[t, h] - o[h]) <= do[h]) and abs(l_g[t, h] - l[h]) <= dl[h]
            gone = np.isnan(o_g[t, h]).all() and np.isnan(l_g[t, h])
            assert right if apart(t, h) else gone, (t, h)
            lost += int(gone)
    assert lost
    # the normal build on the same workspace and outputs
    err.zero_()
    again = qli.kv_attention(scale=SCALE, out=out, lse=lse, workspace=ws, err_word=err, **kw)
    want = qli.kv_attention(scale=SCALE, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
