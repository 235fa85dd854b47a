"""How calls of drafted trees are split: the restated rules against the kernels that the
library queues, and against what the rules are for."""
import random

import pytest

import tree_launches as plan

SMS = 152


def _shapes(n=60, seed=41):
    rng = random.Random(seed)
    out = [(16, 512, 64, 1, 128, 32768), (16, 128, 64, 1, 128, 32768), (64, 8, 1, 1, 0, 2048), (64, 200, 16, 1, 0, 32768),
           (128, 126, 2, 1, 0, 65536), (16, 320, 40, 1, 64, 32768), (64, 19, 1, 1, 0, 2048), (64, 20, 1, 1, 0, 2048), (16, 96, 6, 1, 0, 4096), (16, 64, 4, 1, 0, 4096),
           (96, 40, 5, 1, 0, 8192), (16, 2000, 9, 4, 300, 4096)]
    while len(out) < n:
        B = rng.choice([1, 2, 5, 16, 64])
        out.append((rng.choice([1, 3, 8, 16, 20, 32, 40, 48, 64, 96, 100, 128]), B * rng.choice([1, 2, 4, 7, 8, 16, 30]), B,
                    rng.choice([1, 1, 2, 5]), rng.choice([0, 0, 1, 40, 64, 65, 128, 192, 700]),
                    rng.choice([128, 256, 384, 2048, 12800, 65536])))
    return out


def test_groups_are_formed_where_single_tokens_have_no_sm_a_unit():
    for H, T, B, words, window, positions in _shapes(2000):
        units = plan.most_units(T, words, window, positions, 1)
        k = plan.stack_of(H, T, B, words, window, positions, SMS)
        assert plan.tiles(H, k) <= k * plan.tiles(H, 1) and 1 <= k <= min(8, -(-T // B))
        if (1 if units <= 2 else units) * T * plan.tiles(H, 1) <= SMS:
            assert k == 1
        elif T >= 8 * B:
            assert (k == 1) == (H % 64 == 0)
    assert plan.split(16, 128, 64, 1, 128, 32768, SMS)[0][0] == "single"     # 64 trees of 2 tokens
    assert plan.split(16, 416, 64, 1, 128, 32768, SMS) == [("groups", 171)]   # of up to 8: whole row tiles
    assert plan.split(16, 512, 64, 1, 128, 32768, SMS) == [("groups", 152), ("join", False)]
    assert plan.split(64, 8, 1, 1, 0, 2048, SMS) == [("single", 152), ("join", True)]
    assert plan.split(64, 19, 1, 1, 0, 2048, SMS) == [("single", 152), ("join", True)]
    assert plan.split(64, 20, 1, 1, 0, 2048, SMS) == [("single", 152), ("join", False)]


@pytest.mark.gpu
@pytest.mark.parametrize("p", _shapes(), ids=lambda p: "-".join(map(str, p)))
def test_the_library_splits_calls_so(p):
    """Queued into a graph that does not run."""
    import torch

    from sparse_attention_indexer_qli_gb300 import build as libbuild
    from sparse_attention_indexer_qli_gb300 import qli
    libbuild.build()
    H, T, B, words, window, positions = p
    z = lambda *shape, dtype=torch.int32: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    q, cache, stride = z(T, H, 512, dtype=torch.bfloat16), z(1, 128 * 514, dtype=torch.uint8), 128 * 514
    kw = dict(k_lens=z(B), tree_mask=z(T, words, dtype=torch.int64), rows_per_page=128, page_stride=stride, kv_offset=0,
              kv_scale_offset=128 * 512, scale=1.0, window=window)
    cu, table = z(B + 1), z(B, positions // 128)
    got = plan.launches(lambda: qli.kv_tree_attention(q, cu, cache, table, **kw))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert got == plan.split(H, T, B, words, window, positions, sms)
