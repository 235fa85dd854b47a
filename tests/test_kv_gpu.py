"""GPU parity of the 8-bit KV writer and reader (bit for bit) and of the merge
(to a derived tolerance) against oracle/kv8.py."""
import numpy as np
import pytest

from oracle import kv8
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli, synth

pytestmark = pytest.mark.gpu

QUANTS = [kv8.INT8, kv8.FP8]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    qli.lib()


def geometry(R, quant):
    L = synth.kv8_layout(R)
    return dict(rows_per_page=R, page_stride=L["page_stride"], kv_offset=L["kv_offset"],
                kv_scale_offset=L["kv_scale_offset"], quant_mode=quant)


def bf16(bits, dev="cuda"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(dev).view(torch.bfloat16)


def edge_rows(rng, n):
    """BF16 rows over the whole range: normal, tiny (scale rounds to zero or to
    a subnormal), huge (scale capped), zeros, one single value."""
    x = rng.standard_normal((n, 512)) * 10.0 ** rng.uniform(-9, 6, (n, 1))
    for i in range(0, n, 7):
        x[i] = 0
    for i in range(3, n, 11):
        x[i] = 0
        x[i, int(rng.integers(512))] = -3.0e38
    return kv8.f32_to_bf16(x)


def expected_pool(pool, x, slots, R, quant):
    L, out = synth.kv8_layout(R), pool.copy()
    c, s = kv8.quantise_rows(x, quant)
    for i, m in enumerate(slots):
        if 0 <= m < pool.shape[0] * R:
            page, row = out[m // R], m % R
            page[L["kv_offset"] + row * 512:][:512] = c[i]
            page[L["kv_scale_offset"] + 2 * row:][:2] = s[i:i + 1].view(np.uint8)
    return out


@pytest.mark.parametrize("quant", QUANTS)
@pytest.mark.parametrize("R", [64, 128])
@pytest.mark.parametrize("n,stride", [(1, 512), (2, 576), (63, 520), (700, 512), (5000, 640)])
def test_writer_is_bit_exact(quant, R, n, stride):
    import torch
    rng = np.random.default_rng(n + R + quant)
    x = edge_rows(rng, n)
    pages = -(-n // R) + 2
    slots = rng.permutation(pages * R)[:n].astype(np.int64)
    slots[rng.random(n) < 0.1] = -1
    pool = rng.integers(0, 256, (pages, synth.kv8_layout(R)["page_stride"]), dtype=np.uint8)
    cache = torch.from_numpy(pool.copy()).cuda()
    wide = torch.full((n, stride), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :512] = bf16(x)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qli.write_kv(wide[:, :512], torch.from_numpy(slots).cuda(), cache, err_word=err, **geometry(R, quant))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert np.array_equal(cache.cpu().numpy(), expected_pool(pool, x, slots, R, quant))


def test_writer_flags_slots_past_the_pool_and_writes_nothing_there():
    import torch
    rng = np.random.default_rng(5)
    R, pages = 64, 3
    x = edge_rows(rng, 4)
    slots = np.array([5, pages * R, -(1 << 40), 1 << 50], dtype=np.int64)
    pool = rng.integers(0, 256, (pages, 41216), dtype=np.uint8)
    # the pool sits inside a larger buffer whose rest must stay as it is
    big = torch.from_numpy(np.concatenate([pool, pool, pool])).cuda()
    before = big.cpu().numpy()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qli.write_kv(bf16(x), torch.from_numpy(slots).cuda(), big[pages:2 * pages], err_word=err,
                 **geometry(R, kv8.INT8))
    torch.cuda.synchronize()
    assert int(err.item()) == 8                                 # QLI_DEVERR_PAGE
    after = big.cpu().numpy()
    assert np.array_equal(after[pages:2 * pages], expected_pool(pool, x, slots, R, kv8.INT8))
    assert np.array_equal(after[:pages], before[:pages])
    assert np.array_equal(after[2 * pages:], before[2 * pages:])


@pytest.mark.parametrize("quant", QUANTS)
@pytest.mark.parametrize("R", [64, 128])
@pytest.mark.parametrize("n,stride", [(1, 512), (2, 1024), (65, 520), (3001, 512)])
def test_reader_is_bit_exact(quant, R, n, stride):
    import torch
    rng = np.random.default_rng(n + R + quant)
    pages = -(-n // R) + 2
    L = synth.kv8_layout(R)
    x = edge_rows(rng, pages * R)
    c, s = kv8.quantise_rows(x, quant)
    pool = rng.integers(0, 256, (pages, L["page_stride"]), dtype=np.uint8)
    pool[:, :R * 512] = c.reshape(pages, -1)
    pool[:, R * 512:R * 514] = s.view(np.uint8).reshape(pages, -1)
    slots = rng.integers(0, pages * R, n).astype(np.int64)      # a row may be read twice
    slots[rng.random(n) < 0.1] = -3
    if n > 1:
        slots[1] = pages * R + 12                               # past the pool: zeros, flagged
    out = torch.full((n, stride), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = qli.read_kv(torch.from_numpy(pool).cuda(), torch.from_numpy(slots).cuda(), out=out[:, :512],
                      err_word=err, **geometry(R, quant))
    torch.cuda.synchronize()
    ok = (slots >= 0) & (slots < pages * R)
    y = kv8.rows(c, s, quant)[np.where(ok, slots, 0)]
    want = np.where(ok[:, None], kv8.f32_to_bf16(y), 0).astype(np.uint16)
    assert np.array_equal(got.contiguous().view(torch.int16).cpu().numpy().view(np.uint16) & 0x7FFF, want & 0x7FFF)
    assert np.array_equal(got.float().cpu().numpy(), kv8.bf16_to_f64(want).astype(np.float32))
    assert int(err.item()) == (8 if n > 1 else 0)
    assert bool((out[:, 512:] == 7.0).all())


@pytest.mark.parametrize("quant", QUANTS)
def test_written_rows_read_back(quant):
    import torch
    rng = np.random.default_rng(9)
    n, R = 1000, 64
    x = kv8.f32_to_bf16(rng.standard_normal((n, 512)))
    cache = torch.zeros((20, 41216), dtype=torch.uint8, device="cuda")
    slots = torch.from_numpy(rng.permutation(20 * R)[:n].astype(np.int64)).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    qli.write_kv(bf16(x), slots, cache, stream=s, **geometry(R, quant))
    with torch.cuda.stream(s):
        got = qli.read_kv(cache, slots, **geometry(R, quant))
    torch.cuda.current_stream().wait_stream(s)
    want = kv8.f32_to_bf16(kv8.rows(*kv8.quantise_rows(x, quant), quant))
    assert np.array_equal(got.float().cpu().numpy(), kv8.bf16_to_f64(want).astype(np.float32))


def test_rows_beyond_four_gigabytes():
    import torch
    rng = np.random.default_rng(10)
    R, L = 128, synth.kv8_layout(128)
    pages = (1 << 32) // L["page_stride"] + 50
    cache = torch.zeros((pages, L["page_stride"]), dtype=torch.uint8, device="cuda")
    n = 300
    x = kv8.f32_to_bf16(rng.standard_normal((n, 512)))
    slots = torch.arange(pages * R - n, pages * R, device="cuda")
    qli.write_kv(bf16(x), slots, cache, **geometry(R, kv8.INT8))
    got = qli.read_kv(cache, slots, **geometry(R, kv8.INT8))
    want = kv8.f32_to_bf16(kv8.rows(*kv8.quantise_rows(x, kv8.INT8), kv8.INT8))
    assert np.array_equal(got.float().cpu().numpy(), kv8.bf16_to_f64(want).astype(np.float32))
    assert not bool(cache[:49].any())


# ---- merge --------------------------------------------------------------------

@pytest.mark.parametrize("parts", [1, 2, 3, 4])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (5, 33), (70, 64)])
def test_merge_matches_the_oracle(parts, wide, T, H):
    import torch
    rng = np.random.default_rng(parts + T)
    outs = rng.standard_normal((parts, T, H, 512)).astype(np.float32)
    bits = kv8.f32_to_bf16(outs)
    lses = (4 * rng.standard_normal((parts, T, H))).astype(np.float32)
    if parts > 1:
        lses[0][rng.random((T, H)) < 0.3] = -np.inf
        lses[1][0, 0] = -90.0
        lses[1][rng.random((T, H)) < 0.1] = 200.0
    lses[:, -1, -1] = -np.inf                                  # nothing anywhere
    if wide:
        parts_t, exact = [torch.from_numpy(o).cuda() for o in outs], outs.astype(np.float64)
    else:
        parts_t, exact = [bf16(b) for b in bits], kv8.bf16_to_f64(bits)
    for i in range(parts):                                      # what an empty part holds does not matter
        gone = torch.from_numpy(np.isneginf(lses[i])).cuda()
        parts_t[i][gone] = float("nan")
    out, lse = qli.merge_attention(parts_t, [torch.from_numpy(l).cuda() for l in lses])
    torch.cuda.synchronize()
    clean = np.where(np.isneginf(lses)[..., None], 0.0, exact)
    o_r, l_r = kv8.merge(list(clean), list(lses.astype(np.float64)))
    o_g, l_g = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isneginf(l_g), np.isneginf(l_r))
    # a weight: the FP32 difference of two lse (2^-24 of it, at most 300) and
    # the exponential; four FP32 additions; the quotient; BF16's half step
    dw = 300 * 2.0 ** -24 + 2.0 ** -21
    bound = 2.0 ** -8 * np.abs(o_r) + (2 * dw + 8 * 2.0 ** -24) * np.abs(clean).max(axis=0)
    assert np.all(np.abs(o_g - o_r) <= bound)
    fin = ~np.isneginf(l_r)
    assert np.all(np.abs(l_g[fin] - l_r[fin]) <= dw + 2.0 ** -22 * (1 + np.abs(l_r[fin])))


def test_merge_strides_and_broadcast_parts():
    import torch
    rng = np.random.default_rng(21)
    T, H = 6, 8
    a = torch.randn(H, T, 512, device="cuda").to(torch.bfloat16).transpose(0, 1)   # [T, H, 512]
    b = torch.randn(1, 1, 512, device="cuda").to(torch.bfloat16).expand(T, H, 512)
    la, lb = torch.randn(T, H, device="cuda"), torch.randn(T, H, device="cuda")
    out = torch.full((H, T, 520), 7.0, dtype=torch.bfloat16, device="cuda")
    got, lse = qli.merge_attention([a, b], [la, lb], out=out[:, :, :512].transpose(0, 1))
    want, want_lse = qli.merge_attention([a.contiguous(), b.contiguous()], [la, lb])
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    assert bool((out[:, :, 512:] == 7.0).all())
    del rng
