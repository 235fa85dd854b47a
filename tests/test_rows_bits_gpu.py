"""Codes and scales of rows that are left as they are (no norm, no rotation), bit by
bit against the quantisers' and the writers': E4M3's two zeros are told apart."""
import numpy as np
import pytest

from oracle import kv8
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    qli.lib()


def up(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def patterns(n, d, seed=21):
    """[n, d] finite BF16 patterns, a row's up to a size of its own; zeros of both signs."""
    rng = np.random.default_rng(seed)
    top = rng.integers(1, 255, size=(n, 1)) << 7                # one past the largest pattern's exponent
    x = (rng.random((n, d)) * top).astype(np.uint16)            # patterns, so sizes over all exponents below
    x[:, ::3] = np.maximum(top - rng.integers(1, 1 << 9, size=(n, len(range(0, d, 3)))), 0)
    x[rng.random((n, d)) < 0.1] = 0
    x[0] = 0
    return x | (rng.integers(0, 2, size=(n, d)) << 15).astype(np.uint16)


def bf16(x):
    import torch
    return up(x.view(np.int16)).view(torch.bfloat16)


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
def test_queries_left_as_they_are(quant):
    import torch
    x = bf16(patterns(1500, 128)).view(300, 5, 128)
    codes, scales = qli.prepare_q(x, None, qli.RowPrep(128), quant_mode=quant)
    want, want_s = qli.quantize_q(x, quant_mode=quant)
    assert torch.equal(codes.view(torch.uint8), want.view(torch.uint8)) and torch.equal(scales, want_s)


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
def test_cache_rows_left_as_they_are(quant):
    import torch
    n, L = 1200, synth.kv8_layout(64)
    kv, k = bf16(patterns(n, 512, 22)), bf16(patterns(n, 128, 23))
    slots = up(np.random.default_rng(24).permutation(20 * 64)[:n])
    one, two = (torch.zeros(20, L["page_stride"], dtype=torch.uint8, device="cuda") for _ in range(2))
    pages = dict(rows_per_page=64, page_stride=L["page_stride"], quant_mode=quant)
    at_kv, at_k = ({a: L[a] for a in names} for names in (("kv_offset", "kv_scale_offset"), ("k_offset", "scale_offset")))
    qli.append_kv(kv, k, None, slots, one, kv_prep=qli.RowPrep(512), index_prep=qli.RowPrep(128), kv_mode=quant,
                  **at_kv, **at_k, **pages)
    qli.write_kv(kv, slots, two, **at_kv, **pages)
    qli.write_index_k(k, slots, two, **at_k, **pages)
    assert torch.equal(one, two)
