"""The decode-step example merges stages over disjoint positions, as the merge is
defined: its output is the attention over the picked and the latest positions, each
counted once. Short requests, all of whose positions are in the window, among them."""
import pytest

from sparse_attention_indexer_qli_gb300 import qli
from test_kv8_example_gpu import example  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [qli.QUANT_INT8, qli.QUANT_FP8], ids=["i8", "f8"])
@pytest.mark.parametrize("window", [1, 100])
def test_no_position_counts_twice(example, mode, window):  # noqa: F811
    import torch
    pool = example.Pool([1, 60, 700, 5000], 2, mode, seed=6)
    for _ in range(2):
        step = example.decode_step(pool, topk=512, window=window)
        picked = 0
        for b in range(4):
            n = int(pool.lengths[b])
            listed = step["indices"][b, 0]
            listed = listed[listed >= 0].long()
            latest = torch.arange(max(0, n - window), n, device=listed.device)
            pos = torch.unique(torch.cat([listed, latest]))
            assert pos.numel() == listed.numel() + latest.numel()
            picked += listed.numel()
            kv = qli.read_kv(pool.cache, pool.slots(torch.full_like(pos, b), pos), **pool.kv_geometry()).float()
            z = step["scale"] * step["q"][b].float() @ kv.T
            # the bound of test_kv8_example_gpu.py
            assert (torch.softmax(z, 1) @ kv - step["out"][b].float()).abs().max().item() < 2.0 ** -4
            assert (torch.logsumexp(z, 1) - step["lse"][b]).abs().max().item() < 2.0 ** -4
        assert picked > 512
    assert int(pool.err.item()) == 0
