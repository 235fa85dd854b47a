"""Calls of the 8-bit attention on a stream other than the current one, with
memory of their own making, while the current stream is busy with calls of its
own: the same bits as the same calls alone."""
import pytest

from kv8_cases import KVCase
from oracle import kv8
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli

pytestmark = pytest.mark.gpu

SCALE = 512.0 ** -0.5


@pytest.fixture(scope="module")
def calls():
    import torch
    libbuild.build()
    qli.lib()
    args = [KVCase(121, [9000, 5000], [3, 2], 1, 64, kv8.FP8).upload(), KVCase(122, [20000], [40], 1, 64, kv8.INT8).upload()]
    want = [tuple(t.clone() for t in qli.kv_attention(scale=SCALE, **kw)) for kw in args]
    torch.cuda.synchronize()
    return args, want


def _same(got, want):
    return all((g == w).all().item() for g, w in zip(got, want))


def test_two_side_streams_one_of_them_current(calls):
    import torch
    args, want = calls
    here, there = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    with torch.cuda.stream(here):
        for i in range(30):
            # the long call first: its memory is free again at once, and in use for long
            got.append((1, qli.kv_attention(scale=SCALE, **args[1])))
            got.append((0, qli.kv_attention(scale=SCALE, stream=there, **args[0])))
            out, lse = qli.kv_attention(scale=SCALE, stream=there, **args[1])
            got.append((0, qli.merge_attention([qli.kv_attention(scale=SCALE, stream=there, **args[0])[0]],
                                               [want[0][1]], stream=there)))
            del out, lse
    torch.cuda.synchronize()
    for i, g in got:
        # a merge of one part changes nothing: its weight is e^0, and ln 1 is added
        assert torch.equal(g[0], want[i][0]) and torch.equal(g[1], want[i][1])


def test_results_dropped_on_the_current_stream(calls):
    """Results made on another stream, used on the current one after a wait, and
    dropped at once while the use is still pending."""
    import torch
    args, want = calls
    here, there = torch.cuda.Stream(), torch.cuda.Stream()
    busy = torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    copies = []
    with torch.cuda.stream(here):
        for _ in range(20):
            out, lse = qli.kv_attention(scale=SCALE, stream=there, **args[0])
            here.wait_stream(there)
            for _ in range(3):
                busy.add_(1.0)
            copies.append((out.clone(), lse.clone()))
            del out, lse
    torch.cuda.synchronize()
    assert all(_same(c, want[0]) for c in copies)


def test_a_forked_stream_in_a_graph(calls):
    import torch
    args, want = calls
    there = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        there.wait_stream(torch.cuda.current_stream())
        out, lse = qli.kv_attention(scale=SCALE, stream=there, **args[0])
        torch.cuda.current_stream().wait_stream(there)
    other = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        out.zero_()
        other.fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0][0]) and torch.equal(lse, want[0][1])
        assert bool((other == 0x5A).all())
