"""Memory that the 8-bit KV calls make for themselves belongs to the stream that
uses it: a block of the current stream's may still be in use by work pending
there, which a kernel on another stream does not wait for."""
import pytest
import torch

from fake_cuda import GEOMETRY, FakeStream, attention_inputs, fake, on_gpu  # noqa: F401
from sparse_attention_indexer_qli_gb300 import qli


def _attention(**kw):
    return qli.kv_attention(**attention_inputs(), **kw)


def _read(**kw):
    return (qli.read_kv(on_gpu(torch.zeros(2, 41216, dtype=torch.uint8)),
                        on_gpu(torch.zeros(5, dtype=torch.int64)), **GEOMETRY, **kw),)


def _merge(**kw):
    part = on_gpu(torch.zeros(3, 2, 512, dtype=torch.bfloat16))
    lse = on_gpu(torch.zeros(3, 2))
    return qli.merge_attention([part, part], [lse, lse], **kw)


CALLS = [(_attention, 2), (_read, 1), (_merge, 2)]
IDS = ["attention", "read", "merge"]


@pytest.mark.parametrize("call,outputs", CALLS, ids=IDS)
def test_another_stream_gets_its_own_memory(fake, call, outputs):  # noqa: F811
    here, there = FakeStream("here", 11), FakeStream("there", 12)
    with fake.on(here):
        results = call(stream=there)
    assert fake.lib.calls[-1][1][-1] == 12
    assert len(fake.made) >= outputs and all(s is there for s, _ in fake.made)
    # the results may be used, and dropped, on the stream that was current
    assert set(fake.recorded) == {(t.data_ptr(), here) for t in results}


@pytest.mark.parametrize("call,outputs", CALLS, ids=IDS)
@pytest.mark.parametrize("given", [False, True])
def test_the_current_stream_uses_its_own_memory(fake, call, outputs, given):  # noqa: F811
    here = FakeStream("here", 11)
    with fake.on(here):
        call(**(dict(stream=here) if given else {}))
    assert fake.lib.calls[-1][1][-1] == 11
    assert len(fake.made) >= outputs and all(s is here for s, _ in fake.made)
    assert not fake.recorded


def test_the_default_stream_from_another(fake):  # noqa: F811
    here = FakeStream("here", 11)
    kept = qli._default_stream_workspace(97)
    fake.made.clear()
    with fake.on(here):
        out, lse = _attention(stream=fake.default)
    name, (a, workspace, n, stream) = fake.lib.calls[-1]
    assert stream == 0 and workspace == kept.data_ptr()
    assert [s for s, _ in fake.made] == [fake.default, fake.default]
    assert set(fake.recorded) == {(out.data_ptr(), here), (lse.data_ptr(), here)}


def test_given_tensors_are_left_to_the_caller(fake):  # noqa: F811
    out, lse = on_gpu(torch.zeros(3, 2, 512, dtype=torch.bfloat16)), on_gpu(torch.zeros(3, 2))
    ws = on_gpu(torch.zeros(4096, dtype=torch.uint8))
    with fake.on(FakeStream("here", 11)):
        got = _attention(stream=FakeStream("there", 12), out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse and not fake.made and not fake.recorded
