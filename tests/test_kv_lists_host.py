"""Lists without entries: their tensor has no address, which the library reads as
no list at all, so the binding must not pass them on."""
import pytest
import torch

from fake_cuda import attention_inputs, fake, on_gpu  # noqa: F401
from sparse_attention_indexer_qli_gb300 import qli


def _lens(B):
    return dict(k_lens=on_gpu(torch.full((B,), 9, dtype=torch.int32)))


@pytest.mark.parametrize("more", [{}, _lens(2)], ids=["list", "list-and-lengths"])
def test_lists_without_entries_are_refused(fake, more):  # noqa: F811
    with pytest.raises(ValueError, match="indices"):
        qli.kv_attention(**dict(attention_inputs(K=0), **more))
    assert not fake.lib.calls


def test_no_tokens_need_no_entries(fake):  # noqa: F811
    out, lse = qli.kv_attention(**attention_inputs(T=0, K=0))
    assert out.shape == (0, 2, 512) and lse.shape == (0, 2)
    qli.kv_attention(**dict(attention_inputs(K=1), **_lens(2)))
    assert fake.lib.calls[-1][1][0].K == 1 and fake.lib.calls[-1][1][0].indices
