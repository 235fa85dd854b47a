"""Stand-ins for torch's CUDA calls and for the library, so that the binding runs
on the CPU: host tensors that call themselves CUDA tensors, streams that are only
names, an allocator that notes the stream that is current, and a library that
notes the calls it gets. Nothing here reaches a GPU.

The device index is one that no machine has, so that what the binding keeps per
device cannot meet a test on a GPU."""
import contextlib
import threading
import types

import pytest
import torch

from sparse_attention_indexer_qli_gb300 import qli

DEVICE = 97
real_empty = torch.empty


class FakeTensor(torch.Tensor):
    is_cuda = True
    index = DEVICE

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index

    def record_stream(self, stream):
        recorded.append((self.data_ptr(), stream))


class ElsewhereTensor(FakeTensor):
    index = DEVICE + 1


recorded = []                      # (address, stream) of every record_stream


def on_gpu(t, elsewhere=False):
    return t.as_subclass(ElsewhereTensor if elsewhere else FakeTensor)


class FakeStream:
    def __init__(self, name, raw):
        self.name, self.cuda_stream, self.stream_id = name, raw, raw

    def __repr__(self):
        return self.name


class FakeLib:
    """The library's calls: each gives `status` and notes its arguments; a packed
    structure comes back as its mirror."""

    def __init__(self):
        self.calls, self.status = [], 0

    def _note(self, name, *args):
        self.calls.append((name, args))
        return self.status

    def qli_kv_attention(self, a, workspace, n, stream):
        return self._note("kv_attention", qli.KVAttnArgs.from_buffer_copy(a), workspace, n, stream)

    def qli_merge_attention(self, a, stream):
        return self._note("merge_attention", qli.MergeArgs.from_buffer_copy(a), stream)

    def qli_write_kv(self, *args):
        return self._note("write_kv", *args)

    def qli_read_kv(self, *args):
        return self._note("read_kv", *args)

    def qli_workspace_size(self, a, n):
        n._obj.value = 4096
        return 0

    def qli_run(self, a, workspace, n, stream):
        return self._note("run", workspace, n, stream)

    def qli_sparse_attention(self, a, stream):
        return self._note("sparse_attention", stream)

    def qli_quantize_q(self, *args):
        return self._note("quantize_q", *args)

    def qli_check_quant_rounding(self, counts, stream):
        return self._note("check_quant_rounding", counts, stream)

    def qli_status_string(self, status):
        return b"status %d" % status


@pytest.fixture
def fake(monkeypatch):
    """The patched world: `lib`, `stream` (current), `default`, `made` ((stream,
    tensor) of every allocation)."""
    w = types.SimpleNamespace(lib=FakeLib(), default=FakeStream("default", 0), made=[], device=DEVICE)
    here = threading.local()

    def current(device=None):
        return getattr(here, "stream", w.default)

    @contextlib.contextmanager
    def on(stream):
        before, here.stream = current(), stream
        yield
        here.stream = before

    def empty(*size, device=None, **kw):
        t = real_empty(*size, **kw)
        if device is not None and torch.device(device).type == "cuda":
            t = on_gpu(t)
            w.made.append((current(), t))
        return t

    w.on, w.current = on, current
    recorded.clear()
    w.recorded = recorded
    monkeypatch.setattr(torch.cuda, "current_stream", current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: w.default)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: w.device)
    monkeypatch.setattr(torch.cuda, "device", lambda index: contextlib.nullcontext())
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(qli, "_lib", w.lib)
    monkeypatch.setattr(qli, "_workspace_bytes", lambda some, device: 4096)
    return w


R, GEOMETRY = 64, dict(rows_per_page=64, page_stride=41216, kv_offset=0, kv_scale_offset=32768)


def attention_inputs(T=3, H=2, B=2, width=4, K=8):
    """Arguments of a listed kv_attention call."""
    return dict(q=on_gpu(torch.zeros(T, H, 512, dtype=torch.bfloat16)),
                cu_seqlens_q=on_gpu(torch.zeros(B + 1, dtype=torch.int32)),
                cache=on_gpu(torch.zeros(2, 41216, dtype=torch.uint8)),
                block_table=on_gpu(torch.zeros(B, width, dtype=torch.int32)),
                indices=on_gpu(torch.zeros(T, 1, K, dtype=torch.int32)), scale=1.0, **GEOMETRY)
