"""The indexer, the quantiser, the BF16 attention and the rounding check on a
stream other than the current one: the same results."""
import pytest

from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli, synth

pytestmark = pytest.mark.gpu


def test_calls_on_another_stream():
    import torch
    libbuild.build()
    qli.lib()
    kw = synth.upload(synth.make_case(131, [9000, 3100], [1, 2], N=64, ratio=2, topk=512, cand_mode="source",
                                      cand_blocks=256, name="streams"), "cuda")
    x = torch.randn(300, 4, 128, device="cuda").to(torch.bfloat16)
    q = torch.randn(3, 32, 512, device="cuda").to(torch.bfloat16)
    pool = torch.randn(40, 128 * 512, device="cuda").to(torch.bfloat16).view(torch.uint8)
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    bt = torch.arange(40, dtype=torch.int32, device="cuda")[None]
    pos = torch.arange(3 * 200, dtype=torch.int32, device="cuda").view(3, 1, 200)

    def calls(**on):
        return [*qli.run(**kw, **on), *qli.quantize_q(x, **on),
                *qli.sparse_attention(q, cu, pool, bt, pos, rows_per_page=128, page_stride=128 * 1024,
                                      scale=0.04, **on)]

    want = calls()
    here, there = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    with torch.cuda.stream(here):
        for _ in range(10):
            got.append(calls())
            got.append(calls(stream=there))
        counts = qli.check_quant_rounding(stream=there)
    torch.cuda.synchronize()
    for g in got:
        assert len(g) == 6 and all(torch.equal(a, b) for a, b in zip(g, want))
    assert counts == qli.check_quant_rounding()
