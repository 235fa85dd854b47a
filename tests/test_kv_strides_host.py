"""What the binding passes for the 8-bit KV calls' strides: the block table's width
apart from its row pitch, and nothing out of the stride of a dimension of size one,
which may be any number."""
import ctypes

import pytest
import torch

from fake_cuda import attention_inputs, fake, on_gpu  # noqa: F401
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli


def _table(fake, table, B):  # noqa: F811
    qli.kv_attention(**dict(attention_inputs(T=3, B=B), block_table=on_gpu(table)))
    a = fake.lib.calls[-1][1][0]
    assert a.block_table == table.data_ptr() and a.B == B
    return a.bt_stride, a.bt_width


def test_block_table_width_and_pitch(fake):  # noqa: F811
    wide = torch.zeros(3, 40, dtype=torch.int32)
    assert _table(fake, wide, 3) == (40, 40)
    assert _table(fake, wide[:, 3:10], 3) == (40, 7)
    assert _table(fake, wide[:, 3:4], 3) == (40, 1)
    # one row: its pitch names nothing
    assert _table(fake, wide[1:2, 3:10], 1) == (7, 7)
    one = torch.zeros(9, 1, dtype=torch.int32).t()
    assert one.stride() == (1, 1) and _table(fake, one, 1) == (9, 9)
    # one column: the stride along it names nothing
    column = torch.zeros(1, 3, dtype=torch.int32).t()
    assert column.stride() == (1, 3) and _table(fake, column, 3) == (1, 1)
    # rows that overlap
    assert _table(fake, torch.as_strided(wide, (3, 8), (2, 1)), 3) == (2, 8)
    with pytest.raises(ValueError):
        _table(fake, wide.t(), 3)


ODD = [((1, 2), (3, 600)), ((1, 2), (1, 520)), ((3, 1), (520, 7)), ((1, 1), (1, 1)), ((1, 1), (5, 0))]


@pytest.mark.parametrize("shape,strides", ODD)
def test_dimensions_of_size_one(fake, shape, strides):  # noqa: F811
    T, H = shape
    base = torch.zeros(4096, dtype=torch.bfloat16)
    odd = lambda: on_gpu(torch.as_strided(base, (T, H, 512), (*strides, 1)))  # noqa: E731
    lse = on_gpu(torch.zeros(T, H))
    qli.kv_attention(**dict(attention_inputs(T=T, H=H), q=odd(), out=odd()))
    a = fake.lib.calls[-1][1][0]
    for st, sh in ((a.q_stride_t, a.q_stride_h), (a.out_stride_t, a.out_stride_h)):
        for n, given, passed in ((T, strides[0], st), (H, strides[1], sh)):
            assert passed == given if n > 1 else passed >= 512 and passed % 8 == 0
    qli.merge_attention([odd(), odd()], [lse, lse], out=odd())
    a = fake.lib.calls[-1][1][0]
    assert a.out_stride_t == (strides[0] if T > 1 else 512) and a.out_stride_h == (strides[1] if H > 1 else 512)
    for i in range(2):
        assert a.part_stride_t[i] == (strides[0] if T > 1 else 0)
        assert a.part_stride_h[i] == (strides[1] if H > 1 else 0)


def test_the_library_refuses_a_negative_width():
    from test_kv_abi import INVALID, P, good_attn
    libbuild.build()
    L = qli.lib()
    for listed in (True, False):
        a = good_attn(listed, bt_width=-1)
        assert L.qli_kv_attention(ctypes.byref(a), P, 1 << 40, None) == INVALID
