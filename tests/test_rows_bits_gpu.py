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


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
@pytest.mark.parametrize("norm", [None, "rms", "layer"])
def test_cache_rows_that_are_not_finite_do_not_become_finite(norm, quant):
    """What reads such a row gets NaN in all of it, as after write_kv; its neighbours are
    those of a call without it."""
    import torch
    n, L = 40, synth.kv8_layout(64)
    x = np.random.default_rng(25).standard_normal((n, 512))
    pages = dict(rows_per_page=64, page_stride=L["page_stride"], quant_mode=quant, kv_offset=L["kv_offset"],
                 kv_scale_offset=L["kv_scale_offset"])
    slots = up(np.random.default_rng(26).permutation(64)[:n])
    prep = qli.RowPrep(512, norm=norm, rotary=qli.Rotary(64), offset=448)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")

    def rows(x):
        cache = torch.zeros(1, L["page_stride"], dtype=torch.uint8, device="cuda")
        kw = dict(pages, kv_mode=quant)
        qli.append_kv(x, None, pos, slots, cache, kv_prep=prep, **kw)
        return cache

    fine = bf16(kv8.f32_to_bf16(x))
    bad = fine.clone()
    bad[3, 7], bad[9, 500], bad[20, 0], bad[31] = float("nan"), float("nan"), float("-inf"), float("nan")
    hit = torch.zeros(n, dtype=torch.bool, device="cuda")
    hit[[3, 9, 20, 31]] = True
    got, want = (qli.read_kv(rows(t), slots, **pages) for t in (bad, fine))
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], want[~hit])
