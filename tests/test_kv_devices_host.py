"""The 8-bit KV calls launch on the current device: tensors of another one, or of
two, are refused before anything is queued (a raw default stream names no device,
so the launch itself would not notice)."""
import contextlib

import pytest
import torch

from fake_cuda import DEVICE, GEOMETRY, attention_inputs, fake, on_gpu  # noqa: F401
from sparse_attention_indexer_qli_gb300 import qli


def _zeros(*shape, dtype=torch.int32):
    return on_gpu(torch.zeros(*shape, dtype=dtype))


def _attention(dense=False):
    kw = attention_inputs()
    if dense:
        kw.pop("indices")
        kw.update(k_lens=_zeros(2), residual=_zeros(2), ratio=2)
    kw.update(out=_zeros(3, 2, 512, dtype=torch.bfloat16), lse=_zeros(3, 2, dtype=torch.float32),
              workspace=_zeros(4096, dtype=torch.uint8), err_word=_zeros(1))
    return qli.kv_attention, kw


def _write():
    return qli.write_kv, dict(kv=_zeros(5, 512, dtype=torch.bfloat16), slot_mapping=_zeros(5, dtype=torch.int64),
                              cache=_zeros(2, 41216, dtype=torch.uint8), err_word=_zeros(1), **GEOMETRY)


def _read():
    return qli.read_kv, dict(cache=_zeros(2, 41216, dtype=torch.uint8), slots=_zeros(5, dtype=torch.int64),
                             out=_zeros(5, 512, dtype=torch.bfloat16), err_word=_zeros(1), **GEOMETRY)


def _merge():
    kw = {"out%d" % i: _zeros(3, 2, 512, dtype=torch.bfloat16) for i in range(2)}
    kw.update({"lse%d" % i: _zeros(3, 2, dtype=torch.float32) for i in range(2)})
    kw.update(out=_zeros(3, 2, 512, dtype=torch.bfloat16), lse=_zeros(3, 2, dtype=torch.float32))
    return (lambda out0, out1, lse0, lse1, **more: qli.merge_attention([out0, out1], [lse0, lse1], **more)), kw


CALLS = [(_attention, ()), (_attention, (True,)), (_write, ()), (_read, ()), (_merge, ())]
IDS = ["listed", "dense", "write", "read", "merge"]


@pytest.mark.parametrize("make,args", CALLS, ids=IDS)
def test_a_tensor_of_another_device_is_refused(fake, make, args):  # noqa: F811
    call, kw = make(*args)
    call(**kw)
    assert len(fake.lib.calls) == 1
    for name in [n for n, v in kw.items() if isinstance(v, torch.Tensor)]:
        with pytest.raises(ValueError, match="device"):
            call(**dict(kw, **{name: on_gpu(kw[name], elsewhere=True)}))
        with pytest.raises(TypeError):
            call(**dict(kw, **{name: torch.zeros(kw[name].shape, dtype=kw[name].dtype)}))
    assert len(fake.lib.calls) == 1


@pytest.mark.parametrize("make,args", CALLS, ids=IDS)
def test_a_device_that_is_not_current_is_refused(fake, make, args):  # noqa: F811
    call, kw = make(*args)
    there = {n: on_gpu(v, elsewhere=True) if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    with pytest.raises(ValueError, match="current device"):
        call(**there)
    assert not fake.lib.calls
    fake.device = DEVICE + 1
    call(**there)
    assert len(fake.lib.calls) == 1


def test_workspace_bytes_of_an_unnumbered_device(fake, monkeypatch):  # noqa: F811
    asked = []
    monkeypatch.setattr(qli, "_workspace_bytes", lambda some, device: asked.append(device) or 4096)
    monkeypatch.setattr(torch.cuda, "device", lambda index: contextlib.nullcontext())
    for device in (None, "cuda", torch.device("cuda"), "cuda:5", 6):
        qli.kv_attention_workspace_bytes(1, 64, device)
    assert asked == [DEVICE, DEVICE, DEVICE, 5, 6]
