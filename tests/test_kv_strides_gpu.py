"""One token or one head whose stride along that dimension is any number: the same
bits as with contiguous tensors."""
import pytest

from kv8_cases import KVCase
from oracle import kv8
from test_kv_attn_gpu import SCALE, _lib  # noqa: F401
from sparse_attention_indexer_qli_gb300 import qli

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,strides", [(1, 64, (777, 512)), (1, 3, (1, 520)), (3, 1, (520, 5)), (1, 1, (1, 1))])
def test_dimensions_of_size_one(T, H, strides):
    import torch
    kw = KVCase(151 + T + H, [900], [T], 1, H, kv8.INT8).upload()
    want = qli.kv_attention(scale=SCALE, **kw)
    odd = lambda: torch.full((40000,), 7.0, dtype=torch.bfloat16, device="cuda").as_strided(  # noqa: E731
        (T, H, 512), (*strides, 1))
    q, part, out, merged = odd(), odd(), odd(), odd()
    q.copy_(kw["q"])
    got = qli.kv_attention(scale=SCALE, **dict(kw, q=q, out=out))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    part.copy_(want[0])
    got = qli.merge_attention([part], [want[1]], out=merged)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
