"""Who shares the workspace that kv_attention keeps for the default stream: one
call is several kernels, so two host threads that queue calls on that stream side
by side may queue them interleaved, and must not write to one block."""
import threading

import pytest
import torch

from fake_cuda import DEVICE, attention_inputs, fake, on_gpu  # noqa: F401
from sparse_attention_indexer_qli_gb300 import qli


def _in_threads(n, f):
    """f(i) in n threads that are all alive until the last has run."""
    out, all_ran = [None] * n, threading.Barrier(n)

    def body(i):
        out[i] = f(i)
        all_ran.wait(10)

    threads = [threading.Thread(target=body, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return out


def test_host_threads_do_not_share_a_workspace(fake):  # noqa: F811
    def calls(i):
        for _ in range(3):
            qli.kv_attention(**attention_inputs(T=1 + i))

    _in_threads(3, calls)
    used = {}
    for name, (a, workspace, n, stream) in fake.lib.calls:
        assert name == "kv_attention" and stream == 0 and n >= 4096
        used.setdefault(a.T, set()).add(workspace)
    # a thread keeps its own, and no other has it
    assert sorted(used) == [1, 2, 3] and all(len(w) == 1 for w in used.values())
    assert len(set.union(*used.values())) == 3


def test_a_thread_keeps_one_per_device(fake):  # noqa: F811
    kept = _in_threads(1, lambda i: [qli._default_stream_workspace(d) for d in (DEVICE, DEVICE + 1, DEVICE)])[0]
    assert kept[0] is kept[2] and kept[0] is not kept[1]
    assert all(stream is fake.default for stream, _ in fake.made)


def test_a_workspace_has_to_be_as_long_as_it_says(fake):  # noqa: F811
    short = torch.zeros(1, dtype=torch.uint8)
    for ws in (short.expand(1 << 30), torch.zeros(8192, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            qli.kv_attention(workspace=on_gpu(ws), **attention_inputs())
    assert not fake.lib.calls
    qli.kv_attention(workspace=on_gpu(torch.zeros(8192, dtype=torch.uint8)[256:]), **attention_inputs())
    assert fake.lib.calls[0][1][2] == 8192 - 256
