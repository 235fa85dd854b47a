"""Attention of drafted trees from two host threads at once, each on its own stream or
both on the default one, and from two graphs on two streams: nobody shares memory."""
import threading

import pytest

from oracle import kv8
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    qli.lib()


def _cases():
    from test_kv_tree_gpu import SCALE, TreeCase
    kws = [dict(TreeCase(90 + i, [3000, 900], [8, 5], H, kv8.FP8, "tree").upload(), scale=SCALE)
           for i, H in enumerate((16, 64))]
    return kws, [[t.clone() for t in qli.kv_tree_attention(**kw)] for kw in kws]


@pytest.mark.parametrize("own_streams", [False, True])
def test_two_threads(own_streams):
    import torch
    kws, want = _cases()
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream() if own_streams else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            for _ in range(60):
                got = qli.kv_tree_attention(**kws[i])
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_two_graphs_on_two_streams():
    import torch
    kws, want = _cases()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for kw, s in zip(kws, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(qli.kv_tree_attention(**kw))
        graphs.append(g)
    for _ in range(30):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(got, w))
