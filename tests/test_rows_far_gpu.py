"""Offsets past 32 bits: rows, queries, page pools and drafted trees that lie more than
4 GB (and 2^32 elements) from the start of their tensors."""
import numpy as np
import pytest

from oracle import kv8
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    libbuild.build()
    qli.lib()
    yield
    torch.cuda.empty_cache()


def test_rows_and_queries():
    """The last tokens of a 9 GB tensor are treated as the same tokens alone."""
    import torch
    T, H, D, n = 70001, 128, 512, 5
    assert T * H * D > 2 ** 32
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    x[-n:] = torch.randn(n, H, D, device="cuda", generator=g).to(torch.bfloat16)
    x[:n] = torch.randn(n, H, D, device="cuda", generator=g).to(torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    r = qli.Rotary(64, layout="half")
    prep = qli.RowPrep(D, norm="rms", rotary=r, offset=448)
    ends = [(slice(0, n)), slice(T - n, T)]
    want = [(qli.rotate(x[e].contiguous(), pos[e].contiguous(), r, offset=448),
             qli.prepare_q(x[e].contiguous(), pos[e].contiguous(), prep)) for e in ends]
    out = qli.prepare_q(x, pos, prep)
    for e, (_, q) in zip(ends, want):
        assert torch.equal(out[e], q)
    del out
    out = qli.rotate(x, pos, r, offset=448)
    qli.rotate(x, pos, r, offset=448, out=x)
    for e, (y, _) in zip(ends, want):
        assert torch.equal(out[e], y) and torch.equal(x[e], y)
    assert not x[n:T - n].any()


@pytest.mark.parametrize("kv_mode", [0, kv8.FP8], ids=["bf16", "f8"])
def test_appended_rows(kv_mode):
    import torch
    R = 128
    L = synth.kv8_layout(R)
    k = R * 1024 if kv_mode == 0 else L["k_offset"]
    G = dict(rows_per_page=R, page_stride=k + R * 130, kv_offset=0, kv_scale_offset=R * 512, k_offset=k,
             scale_offset=k + R * 128, kv_mode=kv_mode, quant_mode=kv8.INT8)
    pages = 5 * 2 ** 30 // G["page_stride"]
    cache = torch.zeros(pages, G["page_stride"], dtype=torch.uint8, device="cuda")
    small = torch.zeros(2, G["page_stride"], dtype=torch.uint8, device="cuda")
    kv, ik = (torch.randn(R, d, device="cuda").to(torch.bfloat16) for d in (512, 128))
    pos, row = torch.arange(R, dtype=torch.int32, device="cuda"), torch.arange(R, device="cuda")
    preps = dict(kv_prep=qli.RowPrep(512, norm="rms", rotary=qli.Rotary(64), offset=448), index_prep=qli.RowPrep(128))
    qli.append_kv(kv, ik, pos, (pages - 1) * R + row, cache, **preps, **G)
    qli.append_kv(kv, ik, pos, R + row, small, **preps, **G)
    assert torch.equal(cache[-1], small[1]) and small[1].any()
    assert not cache[0].any() and not cache[-2].any()


def test_drafted_trees():
    import torch

    from test_kv_tree_gpu import SCALE, TreeCase
    case = TreeCase(81, [700, 300], [9, 5], 16, kv8.FP8, "tree")
    kw = case.upload()
    want = qli.kv_tree_attention(scale=SCALE, **kw)
    stride = kw["cache"].shape[1]
    far = 5 * 2 ** 30 // stride
    cache = torch.zeros(far + case.pages, stride, dtype=torch.uint8, device="cuda")
    cache[far:] = kw["cache"]
    bt = kw["block_table"]
    kw.update(cache=cache, block_table=torch.where(bt >= 0, bt + far, bt))
    assert all(torch.equal(a, b) for a, b in zip(qli.kv_tree_attention(scale=SCALE, **kw), want))
    assert np.isfinite(want[1].cpu().numpy()).all()
