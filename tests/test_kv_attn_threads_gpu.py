"""Calls of the 8-bit attention that several host threads queue on the default
stream at the same time: the same bits as the same calls alone. The sizes differ,
and their row tiles are cut between CTAs, so that every call leaves pieces in its
workspace for a second kernel."""
import threading

import pytest

from kv8_cases import KVCase
from oracle import kv8
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli

pytestmark = pytest.mark.gpu

SCALE = 512.0 ** -0.5


def test_threads_on_the_default_stream():
    import torch
    libbuild.build()
    qli.lib()
    cases = [KVCase(111, [3000, 5000], [2, 2], 1, 64, kv8.FP8), KVCase(112, [4000] * 40, [1] * 40, 2, 64, kv8.INT8, K=700),
             KVCase(113, [9001], [1], 1, 128, kv8.INT8)]
    args = [c.upload() for c in cases]
    want = [tuple(t.clone() for t in qli.kv_attention(scale=SCALE, **kw)) for kw in args]
    torch.cuda.synchronize()
    got, start = [[] for _ in args], threading.Barrier(len(args))

    def body(i):
        start.wait(30)
        for _ in range(60):
            got[i].append(qli.kv_attention(scale=SCALE, **args[i]))

    threads = [threading.Thread(target=body, args=(i,)) for i in range(len(args))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for results, (out, lse) in zip(got, want):
        assert len(results) == 60
        assert all(torch.equal(o, out) and torch.equal(l, lse) for o, l in results)
