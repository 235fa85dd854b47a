"""Workspaces of the attention over 8-bit KV rows when the call gives none: one
kept for the default stream, one for each call on other streams."""
import pytest

from kv8_cases import KVCase
from oracle import kv8

pytestmark = pytest.mark.gpu

SCALE = 512.0 ** -0.5


def _call(case, kw, **more):
    from sparse_attention_indexer_qli_gb300 import qli
    return qli.kv_attention(scale=SCALE, **dict(kw, **more))


def test_default_stream_keeps_one_and_others_do_not_share_it():
    import torch

    from sparse_attention_indexer_qli_gb300 import qli
    torch.zeros(1, device="cuda")
    kept = qli._default_stream_workspace(torch.cuda.current_device())
    assert kept.numel() >= qli.kv_attention_workspace_bytes(4, 64) and kept.data_ptr() % 256 == 0
    case = KVCase(101, [3000, 5000], [2, 2], 1, 64, kv8.FP8)
    kw = case.upload()
    want, want_lse = _call(case, kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    # a call on each stream, side by side, again and again
    for _ in range(20):
        got.append(_call(case, kw))
        with torch.cuda.stream(side):
            got.append(_call(case, kw))
        got.append(_call(case, kw, stream=side))
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # a side stream's calls leave the kept workspace alone
    kept.fill_(0x5A)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _call(case, kw)
    torch.cuda.synchronize()
    assert bool((kept == 0x5A).all())
    _call(case, kw)
    torch.cuda.synchronize()
    assert not bool((kept == 0x5A).all())


def test_a_graph_has_its_own():
    import torch

    from sparse_attention_indexer_qli_gb300 import qli
    case = KVCase(102, [4000], [3], 2, 40, kv8.INT8)
    kw = case.upload()
    want, want_lse = _call(case, kw)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(case, kw, out=out, lse=lse)
    kept = qli._default_stream_workspace(torch.cuda.current_device())
    kept.fill_(0x5A)
    graph.replay()
    torch.cuda.synchronize()
    assert bool((kept == 0x5A).all())
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
