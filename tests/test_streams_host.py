"""Memory that the indexer's, the quantiser's and the BF16 attention's calls make
for themselves belongs to the stream that uses it, and is read on it."""
import pytest
import torch

from fake_cuda import FakeStream, fake, on_gpu  # noqa: F401
from sparse_attention_indexer_qli_gb300 import qli


def _zeros(*shape, dtype=torch.int32):
    return on_gpu(torch.zeros(*shape, dtype=dtype))


def _index(**kw):
    mode = dict(cand_mode="source", cand_blocks=64)
    return qli.run(_zeros(2, 32, 128, dtype=torch.int8), _zeros(2), _zeros(1), None,
                   _zeros(1, 147712, dtype=torch.uint8), _zeros(1, 4), _zeros(2, 32, dtype=torch.float16),
                   _zeros(2, 32, dtype=torch.float16), ratio=1, rows_per_page=128, page_stride=147712,
                   k_offset=0, scale_offset=16384, topk=8, **mode, **kw)


def _quantise(**kw):
    return qli.quantize_q(_zeros(3, 2, 128, dtype=torch.bfloat16), **kw)


def _attend(**kw):
    return qli.sparse_attention(_zeros(2, 32, 512, dtype=torch.bfloat16), _zeros(2), _zeros(1, 147712, dtype=torch.uint8),
                                _zeros(1, 4), _zeros(2, 1, 8), rows_per_page=128, page_stride=147712, scale=1.0, **kw)


CALLS = [(_index, 3), (_quantise, 2), (_attend, 2)]
IDS = ["index", "quantise", "attend"]


@pytest.mark.parametrize("call,made", CALLS, ids=IDS)
def test_another_stream_gets_its_own_memory(fake, call, made):  # noqa: F811
    here, there = FakeStream("here", 11), FakeStream("there", 12)
    with fake.on(here):
        results = call(stream=there)
    assert fake.lib.calls[-1][1][-1] == 12
    assert len(fake.made) == made and all(s is there for s, _ in fake.made)
    assert set(fake.recorded) == {(t.data_ptr(), here) for t in results}


@pytest.mark.parametrize("call,made", CALLS, ids=IDS)
@pytest.mark.parametrize("given", [False, True])
def test_the_current_stream_uses_its_own_memory(fake, call, made, given):  # noqa: F811
    here = FakeStream("here", 11)
    with fake.on(here):
        call(**(dict(stream=here) if given else {}))
    assert fake.lib.calls[-1][1][-1] == 11
    assert len(fake.made) == made and all(s is here for s, _ in fake.made)
    assert not fake.recorded


def test_given_outputs_are_left_to_the_caller(fake):  # noqa: F811
    idx, cand = _zeros(2, 1, 8), _zeros(2, 1, 64)
    ws = _zeros(4096, dtype=torch.uint8)
    with fake.on(FakeStream("here", 11)):
        got = _index(stream=FakeStream("there", 12), indices_out=idx, cand_out=cand, workspace=ws)
    assert got[0] is idx and got[1] is cand and not fake.made and not fake.recorded


def test_the_rounding_check_is_read_on_its_stream(fake, monkeypatch):  # noqa: F811
    there, read_on = FakeStream("there", 12), []
    cpu = torch.Tensor.cpu
    monkeypatch.setattr(torch.Tensor, "cpu", lambda t: (read_on.append(fake.current()), cpu(t))[1])
    qli.check_quant_rounding(stream=there)
    assert fake.lib.calls[-1][1][-1] == 12 and set(read_on) == {there}
    assert [s for s, _ in fake.made] == [there]
