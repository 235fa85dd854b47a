"""GPU numerics of the rotation and preparation of rows (qli_rotate, qli_prepare_q,
qli_append_kv) against the float64 oracle (oracle/rows.py).

Bounds, from the arithmetic:
  - an angle's fraction of a turn is cut at 2^-32 and rounded to 24 bits (2^-24 of
    half a turn at most, 2^-22 rad), sine and cosine add 2 ulp (2^-22), and two
    products, a sum and the magnitude four roundings of 2^-24: a rotated value is off
    by at most 2^-20 (|a| + |b|) magnitude;
  - a norm: FP32 sums of up to 512 values in 21 steps at most (16 in a lane, 5 across
    lanes) are off by 2^-19 of the sum of magnitudes, a reciprocal square root by 2
    ulp, three products by 2^-24 each: 2^-18 of the value; the layer norm's mean is off
    by 2^-19 of the row's mean magnitude, which moves every value by that times
    weight / deviation;
  - BF16 is off by half a step, 2^-8 of the value;
  - a row's scale moves by the amax's error and one rounding to FP16 (2^-11, or half a
    step of 2^-24); codes by half a step of the code under that scale, and what lies
    past the largest code by the cut.
"""
import numpy as np
import pytest

from oracle import kv8
from oracle import rows as oracle
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


def bf16_up(bits):
    import torch
    return up(bits.view(np.int16)).view(torch.bfloat16)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def bits(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy()


FAR = [0, 1, -1, 2, 63, 4095, 131071, 1000003, -77777, 2 ** 31 - 1, -2 ** 31]


def positions(rng, n):
    p = rng.integers(0, 200000, size=n)
    k = min(n, len(FAR))
    p[:k] = FAR[:k]
    return p.astype(np.int32)


def turn_error(x, r, offset, half):
    """2^-20 (|a| + |b|) magnitude at the rotated values, else 0."""
    err, n = np.zeros(x.shape), r.dim // 2
    first = offset + (np.arange(n) if half else 2 * np.arange(n))
    second = first + (n if half else 1)
    e = 2.0 ** -20 * (np.abs(x[..., first]) + np.abs(x[..., second]))
    err[..., first] = err[..., second] = e
    return err


def near_bf16(got, want, err):
    bound = err + 2.0 ** -8 * (np.abs(want) + err) + 2.0 ** -133
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


ROTATE = [
    # T, H, D, dim, offset, half, padding between rows
    (1, 1, 16, 16, 0, False, 0), (1, 64, 512, 64, 448, False, 0), (7, 3, 192, 32, 0, True, 8),
    (64, 64, 512, 64, 448, True, 0), (5, 33, 128, 128, 0, True, 64), (300, 1, 128, 48, 8, False, 0),
    (257, 2, 72, 48, 24, True, 8), (3, 5, 200, 112, 88, False, 0), (1000, 9, 64, 64, 0, False, 24),
    (2, 700, 128, 80, 40, True, 0), (600, 1, 1024, 96, 504, False, 0), (1100, 1, 64, 16, 8, True, 0),
    (999, 2, 32, 16, 16, False, 8), (130, 1, 16, 16, 0, True, 0), (257, 1, 64, 32, 32, False, 0)]


@pytest.mark.parametrize("inplace", [False, True], ids=["out", "inplace"])
@pytest.mark.parametrize("inverse", [False, True], ids=["forth", "back"])
@pytest.mark.parametrize("p", ROTATE, ids=lambda p: "-".join(map(str, p)))
def test_rotate(p, inverse, inplace):
    import torch
    T, H, D, dim, offset, half, pad = p
    rng = np.random.default_rng(sum(p) + 2 * inverse)
    r = qli.Rotary(dim, layout="half" if half else "interleaved", factor=4.0, trained=8192, magnitude=1.25)
    x = kv8.f32_to_bf16(rng.standard_normal((T, H, D + pad)) * np.exp(rng.standard_normal((T, H, 1))))
    pos = positions(rng, T)
    wide = bf16_up(x)
    got = qli.rotate(wide[..., :D], up(pos), r, offset=offset, inverse=inverse, out=wide[..., :D] if inplace else None)
    torch.cuda.synchronize()
    v = kv8.bf16_to_f64(x[..., :D])
    want = oracle.rotate(v, pos, r.frequencies, offset, half, 1.25, inverse)
    near_bf16(f64(got), want, turn_error(v, r, offset, half) * (0.8 if inverse else 1.25))
    # the other values, and what lies between the rows, bit by bit
    same = np.ones(D + pad, dtype=bool)
    same[offset:offset + dim] = False
    assert np.array_equal(bits(got)[..., same[:D]], x.view(np.int16)[..., :D][..., same[:D]])
    assert np.array_equal(bits(wide)[..., same], x.view(np.int16)[..., same])


def test_rotate_leaves_the_rest_of_the_row_as_it_is():
    """NaN and infinities beside the rotated part, and in other rows."""
    import torch
    rng = np.random.default_rng(3)
    x = kv8.f32_to_bf16(rng.standard_normal((9, 4, 128)))
    x[:, :, :64] = rng.integers(0, 1 << 16, size=(9, 4, 64))              # any pattern
    x[4, 2] = 0x7FC0
    pos, r = positions(rng, 9), qli.Rotary(64)
    t = bf16_up(x)
    qli.rotate(t, up(pos), r, offset=64, out=t)
    torch.cuda.synchronize()
    assert np.array_equal(bits(t)[..., :64], x.view(np.int16)[..., :64])
    got, want = f64(t)[..., 64:], oracle.rotate(kv8.bf16_to_f64(x), pos, r.frequencies, 64, False)[..., 64:]
    assert np.isnan(got[4, 2]).all() and np.isfinite(np.delete(got.reshape(36, 64), 4 * 4 + 2, 0)).all()
    ok = np.ones((9, 4), dtype=bool)
    ok[4, 2] = False
    near_bf16(got[ok], want[ok], 2.0 ** -20 * 2 * np.abs(want[ok]).max() * np.ones(want[ok].shape))


def test_rotate_back_gives_the_row_again():
    rng = np.random.default_rng(4)
    x = kv8.f32_to_bf16(rng.standard_normal((40, 8, 128)))
    pos, r = up(positions(rng, 40)), qli.Rotary(128, layout="half", magnitude=1.5)
    y = f64(qli.rotate(qli.rotate(bf16_up(x), pos, r), pos, r, inverse=True))
    v = kv8.bf16_to_f64(x)
    pair = np.hypot(v[..., :64], v[..., 64:])
    # each way BF16 moves a value by 2^-8 of itself at most, so of its pair's length
    assert np.all(np.abs(y - v) <= np.tile(pair, 2) * (2 * 2.0 ** -8 * 1.5 + 2.0 ** -16))


def test_rotate_broadcast_and_transposed_inputs():
    import torch
    rng = np.random.default_rng(5)
    x, pos, r = kv8.f32_to_bf16(rng.standard_normal((6, 1, 128))), positions(rng, 6), qli.Rotary(64)
    t = bf16_up(x)
    want = bits(qli.rotate(t, up(pos), r))
    got = qli.rotate(t.expand(6, 5, 128), up(pos), r)                     # one row for all heads
    assert np.array_equal(bits(got), np.repeat(want, 5, 1))
    heads_first = torch.empty(5, 6, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    qli.rotate(t.expand(6, 5, 128), up(pos), r, out=heads_first)
    assert np.array_equal(bits(heads_first), np.repeat(want, 5, 1))
    assert qli.rotate(t[:0], up(pos[:0]), r).shape == (0, 1, 128)


# ---- queries -----------------------------------------------------------------------

def prep_of(rng, D, norm, dim, offset, half, bare=False):
    """(RowPrep, its weight, its bias) with random weights; dim 0: no rotation."""
    w = None if norm is None or bare else (1 + 0.3 * rng.standard_normal(D)).astype(np.float32)
    b = None if norm != "layer" or bare else (0.3 * rng.standard_normal(D)).astype(np.float32)
    r = qli.Rotary(dim, layout="half" if half else "interleaved", factor=16.0, trained=4096, magnitude=1.1) if dim else None
    return qli.RowPrep(D, norm=norm, weight=None if w is None else up(w), bias=None if b is None else up(b), eps=1e-5,
                       rotary=r, offset=offset), w, b, r


def prepared(v, pos, norm, w, b, r, offset, half):
    """(the oracle's row, its FP32 error)."""
    y = oracle.normalise(v, norm, w, b, 1e-5)
    err = np.zeros(v.shape)
    if norm is not None:
        err = 2.0 ** -18 * (np.abs(y) + (0 if b is None else np.abs(b)))
    if norm == "layer":
        dev = np.sqrt(v.var(axis=-1, keepdims=True) + 1e-5)
        err = err + 2.0 ** -18 * np.abs(v).mean(axis=-1, keepdims=True) / dev * (1 if w is None else np.abs(w))
    if r is not None:
        e = turn_error(y, r, offset, half) * 1.1
        n = r.dim // 2
        first = offset + (np.arange(n) if half else 2 * np.arange(n))
        second = first + (n if half else 1)
        both = 1.1 * (err[..., first] + err[..., second])
        err = err.copy()
        err[..., first] = err[..., second] = both
        err, y = err + e, oracle.rotate(y, pos, r.frequencies, offset, half, 1.1)
    return y, err


WIDTHS = [
    # T, H, D, dim, offset, half
    (1, 1, 64, 64, 0, False), (9, 5, 64, 32, 32, True), (1, 64, 128, 64, 0, True), (33, 7, 128, 128, 0, True),
    (300, 1, 128, 96, 32, False), (3, 33, 256, 64, 96, True), (1, 64, 512, 64, 448, False),
    (65, 3, 512, 128, 192, True), (17, 64, 512, 0, 0, False), (2, 1000, 128, 16, 56, True)]


@pytest.mark.parametrize("norm", [None, "rms", "layer"])
@pytest.mark.parametrize("p", WIDTHS, ids=lambda p: "-".join(map(str, p)))
def test_prepare_bf16(p, norm):
    T, H, D, dim, offset, half = p
    rng = np.random.default_rng(sum(p))
    x = kv8.f32_to_bf16(2 * rng.standard_normal((T, H, D + 8)) * np.exp(rng.standard_normal((T, H, 1))) + 0.5)
    prep, w, b, r = prep_of(rng, D, norm, dim, offset, half, bare=T == 17)
    pos = positions(rng, T)
    wide = bf16_up(x)
    got = qli.prepare_q(wide[..., :D], up(pos) if dim else None, prep)
    v = kv8.bf16_to_f64(x[..., :D])
    y, err = prepared(v, pos, norm, w, b, r, offset, half)
    near_bf16(f64(got), y, err)
    # in place, the same bits
    qli.prepare_q(wide[..., :D], up(pos), prep, out=wide[..., :D])
    assert np.array_equal(bits(wide[..., :D]), bits(got))
    assert np.array_equal(bits(wide)[..., D:], x.view(np.int16)[..., D:])


def near_codes(codes, scales, y, err, quant):
    """codes and scale bits against rows y [n, D] that are off by err."""
    top = {kv8.INT8: 127.0, kv8.FP8: 448.0}[quant]
    v, s = kv8.values(codes, quant), scales.view(np.float16).astype(np.float64)
    amax, worst = np.abs(y).max(axis=1), err.max(axis=1)
    ds = (2.0 ** -11 * (amax + worst) + worst) / top + 2.0 ** -25
    assert np.all(np.abs(s - np.minimum(amax / top, 65504.0)) <= ds)
    s, dead = s[:, None], (s == 0)[:, None]
    assert not v[dead[:, 0]].any()
    # the quotient is in reach of the code: half a step of INT8, or of E4M3 (2^-4 of the value,
    # 2^-10 near zero); a scale below amax / top cuts the largest values to top
    q = np.abs(y) / np.where(dead, 1.0, s)
    step = 0.5 if quant == kv8.INT8 else np.maximum(2.0 ** -4 * np.minimum(q, top), 2.0 ** -10)
    bound = (step + np.maximum(q - top, 0.0)) * s * (1 + 2.0 ** -22) + err
    bad = ~(np.abs(v * s - y) <= bound) & ~dead
    assert not bad.any(), (np.argwhere(bad)[:4], (v * s)[bad][:4], y[bad][:4])


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
@pytest.mark.parametrize("norm", [None, "rms", "layer"])
@pytest.mark.parametrize("p", [p for p in WIDTHS if p[2] == 128], ids=lambda p: "-".join(map(str, p)))
def test_prepare_codes(p, norm, quant):
    T, H, D, dim, offset, half = p
    rng = np.random.default_rng(sum(p) + quant)
    x = kv8.f32_to_bf16(rng.standard_normal((T, H, D)) * np.exp(rng.standard_normal((T, H, 1))))
    prep, w, b, r = prep_of(rng, D, norm, dim, offset, half)
    pos = positions(rng, T)
    codes, scales = qli.prepare_q(bf16_up(x), up(pos), prep, quant_mode=quant)
    y, err = prepared(kv8.bf16_to_f64(x), pos, norm, w, b, r, offset, half)
    near_codes(codes.cpu().numpy().view(np.uint8).reshape(-1, D), scales.cpu().numpy().view(np.uint16).reshape(-1),
               y.reshape(-1, D), err.reshape(-1, D), quant)


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
def test_rows_left_as_they_are_give_the_quantisers_bits(quant):
    """Without norm and rotation: codes and scales of quantize_q, and pages of write_kv
    and write_index_k, over every size of row, zeros and the largest values."""
    import torch
    rng = np.random.default_rng(9)
    size = 2.0 ** rng.integers(-133, 128, size=(300, 1)).astype(np.float64)
    x = kv8.f32_to_bf16(np.clip(rng.standard_normal((300, 512)) * size, -3.3e38, 3.3e38))
    x[7] = 0
    x[8, 3:] = 0
    k = bf16_up(x[:, :128])
    codes, scales = qli.prepare_q(k.reshape(60, 5, 128), None, qli.RowPrep(128), quant_mode=quant)
    want, want_s = qli.quantize_q(k.reshape(60, 5, 128).contiguous(), quant_mode=quant)
    same = lambda a, b: np.array_equal(kv8.values(a.cpu().numpy().view(np.uint8), quant),  # noqa: E731
                                       kv8.values(b.cpu().numpy().view(np.uint8), quant))
    assert same(codes, want) and torch.equal(scales, want_s)
    L = synth.kv8_layout(64)
    one, two = (torch.zeros(6, L["page_stride"], dtype=torch.uint8, device="cuda") for _ in range(2))
    slots, pages = up(rng.permutation(6 * 64)[:300]), dict(rows_per_page=64, page_stride=L["page_stride"], quant_mode=quant)
    kv = bf16_up(x)
    qli.append_kv(kv, k, None, slots, one, kv_prep=qli.RowPrep(512), index_prep=qli.RowPrep(128), kv_mode=quant,
                  kv_offset=L["kv_offset"], kv_scale_offset=L["kv_scale_offset"], k_offset=L["k_offset"],
                  scale_offset=L["scale_offset"], **pages)
    qli.write_kv(kv, slots, two, kv_offset=L["kv_offset"], kv_scale_offset=L["kv_scale_offset"], **pages)
    qli.write_index_k(k.contiguous(), slots, two, k_offset=L["k_offset"], scale_offset=L["scale_offset"], **pages)
    for at, n in ((L["kv_offset"], 64 * 512), (L["k_offset"], 64 * 128)):
        assert same(one[:, at:at + n], two[:, at:at + n])
    for at in (L["kv_scale_offset"], L["scale_offset"]):
        assert torch.equal(one[:, at:at + 128], two[:, at:at + 128])


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_rows_that_a_norm_can_trip_over(D, norm):
    """Zeros, one value, equal values, the smallest and large ones; a row with NaN or
    an infinity does not reach its neighbours."""
    rng = np.random.default_rng(11)
    v = rng.standard_normal((11, D))
    v[0], v[1], v[2] = 0, 0, 3.0
    v[1, D - 1] = 5.0
    v[3] = 2.0 ** -133 * rng.integers(-4, 5, size=D)
    v[4] = 2.0 ** 58 * np.where(rng.random(D) < 0.5, -1, 1)
    x = kv8.f32_to_bf16(v)
    x[6, 3], x[8, 5] = 0x7FC0, 0x7F80
    prep, w, b, r = prep_of(rng, D, norm, 16, 8, True)
    pos = positions(rng, 11)
    got = f64(qli.prepare_q(bf16_up(x)[:, None], up(pos), prep))[:, 0]
    fine = [0, 1, 2, 3, 4, 5, 7, 9, 10]
    y, err = prepared(kv8.bf16_to_f64(x[fine]), pos[fine], norm, w, b, r, 8, True)
    # an FP32 deviation far below eps leaves 1 / sqrt(eps) of the mean's error (row 2 and the like)
    near_bf16(got[fine], y, err)


def test_prepare_nothing():
    import torch
    x = torch.zeros(0, 3, 128, dtype=torch.bfloat16, device="cuda")
    codes, scales = qli.prepare_q(x, None, qli.RowPrep(128), quant_mode=qli.QUANT_INT8)
    assert codes.shape == (0, 3, 128) and scales.shape == (0, 3)


# ---- cache rows ---------------------------------------------------------------------

def page_layout(R, kv_mode):
    k = R * (1024 if kv_mode == 0 else 514)
    k += -k % 16
    return dict(rows_per_page=R, page_stride=k + R * 130 + 112, kv_offset=0, kv_scale_offset=R * 512, k_offset=k,
                scale_offset=k + R * 128)


APPEND = [
    # n, R, KV mode, index mode, rotation (KV), rotation (index), padding
    (1, 64, kv8.INT8, kv8.FP8, (64, 448, False), (64, 0, True), 0),      # the one row is padding
    (2, 64, kv8.FP8, kv8.INT8, (64, 448, False), (64, 0, True), 0),
    (64, 128, kv8.FP8, kv8.FP8, (64, 448, True), (32, 96, False), 8),
    (333, 64, 0, kv8.INT8, (128, 384, False), None, 64),
    (1000, 128, kv8.INT8, kv8.INT8, None, (128, 0, True), 0),
    (129, 128, 0, kv8.FP8, (16, 0, True), (16, 112, True), 24)]


@pytest.mark.parametrize("kinds", ["both", "kv", "index"])
@pytest.mark.parametrize("p", APPEND, ids=lambda p: "%d-%d-%d-%d" % p[:4])
def test_append(p, kinds):
    import torch
    n, R, kv_mode, quant, turn, iturn, pad = p
    rng = np.random.default_rng(n + R)
    G = page_layout(R, kv_mode)
    pages = -(-n // R) + 2
    slots = rng.permutation(pages * R)[:n].astype(np.int64)
    slots[rng.random(n) < 0.1] = -1                                      # padding
    if n > 5:
        slots[3], slots[5] = pages * R, 2 ** 40                           # past the pool
    bad = (slots >= pages * R).any()
    kv, ik = (kv8.f32_to_bf16(rng.standard_normal((n, d + pad)) * np.exp(rng.standard_normal((n, 1)))) for d in (512, 128))
    kp, kw, kb, kr = prep_of(rng, 512, "rms", *(turn or (0, 0, False)))
    ip, iw, ib, ir = prep_of(rng, 128, "layer", *(iturn or (0, 0, False)))
    pos = positions(rng, n)
    before = rng.integers(0, 256, size=(pages, G["page_stride"]), dtype=np.uint8)
    cache, err = up(before), torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = bf16_up(kv)[:, :512], bf16_up(ik)[:, :128]
    qli.append_kv(a if kinds != "index" else None, b if kinds != "kv" else None, up(pos), up(slots), cache, kv_prep=kp,
                  index_prep=ip, kv_mode=kv_mode, quant_mode=quant, err_word=err, **G)
    torch.cuda.synchronize()
    after = cache.cpu().numpy()
    assert int(err.item()) == (8 if bad else 0)
    touched = np.zeros(after.shape, dtype=bool)

    def part(at, width):
        rows = []
        for s in slots[live]:
            sl = np.s_[s // R, at + s % R * width:at + (s % R + 1) * width]
            touched[sl] = True
            rows.append(after[sl])
        return np.stack(rows) if rows else np.zeros((0, width), dtype=np.uint8)

    live = (slots >= 0) & (slots < pages * R)
    if kinds != "index":
        t = turn or (0, 0, False)
        y, e = prepared(kv8.bf16_to_f64(kv[live, :512]), pos[live], "rms", kw, kb, kr, t[1], t[2])
        if kv_mode == 0:
            near_bf16(kv8.bf16_to_f64(part(G["kv_offset"], 1024).view(np.uint16)), y, e)
        else:
            near_codes(part(G["kv_offset"], 512), part(G["kv_scale_offset"], 2).view(np.uint16)[:, 0], y, e, kv_mode)
    if kinds != "kv":
        t = iturn or (0, 0, False)
        y, e = prepared(kv8.bf16_to_f64(ik[live, :128]), pos[live], "layer", iw, ib, ir, t[1], t[2])
        near_codes(part(G["k_offset"], 128), part(G["scale_offset"], 2).view(np.uint16)[:, 0], y, e, quant)
    assert np.array_equal(after[~touched], before[~touched])


def test_append_nothing_and_no_pages():
    import torch
    G = page_layout(64, kv8.INT8)
    none = torch.zeros(0, G["page_stride"], dtype=torch.uint8, device="cuda")
    x, err = torch.zeros(3, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    one = torch.zeros(1, G["page_stride"], dtype=torch.uint8, device="cuda")
    qli.append_kv(x[:0], None, None, up(np.zeros(0, np.int64)), one, kv_prep=qli.RowPrep(512), **G)
    qli.append_kv(x, None, None, up(np.array([-1, 64, 700])), one, kv_prep=qli.RowPrep(512), err_word=err, **G)
    torch.cuda.synchronize()
    assert int(err.item()) == 8 and not one.any()
    with pytest.raises(qli.QLIError):                                      # a pool without memory
        qli.append_kv(x, None, None, up(np.array([0, 1, 2])), none, kv_prep=qli.RowPrep(512), **G)


# ---- streams and graphs ----------------------------------------------------------------

def _calls(T=37, seed=1):
    """name -> (call(stream) -> tensors, the inputs that a graph's user changes)."""
    import torch
    rng = np.random.default_rng(seed)
    r = qli.Rotary(64, layout="half")
    x = bf16_up(kv8.f32_to_bf16(rng.standard_normal((T, 6, 128))))
    pos = up(positions(rng, T))
    prep, _, _, _ = prep_of(np.random.default_rng(2), 128, "rms", 64, 0, True)
    kvp, _, _, _ = prep_of(np.random.default_rng(3), 512, "rms", 64, 448, False)
    G = page_layout(64, kv8.FP8)
    cache = torch.zeros(3, G["page_stride"], dtype=torch.uint8, device="cuda")
    kv, slots = bf16_up(kv8.f32_to_bf16(rng.standard_normal((T, 512)))), up(rng.permutation(192)[:T])

    def append(stream=None):
        qli.append_kv(kv, x[:, 0].contiguous() if stream is None else k, pos, slots, cache, kv_prep=kvp, index_prep=prep,
                      kv_mode=qli.QUANT_FP8, stream=stream, **G)
        return (cache,)
    k = x[:, 0].contiguous()
    return {"rotate": lambda stream=None: (qli.rotate(x, pos, r, offset=64, stream=stream),),
            "prepare": lambda stream=None: (qli.prepare_q(x, pos, prep, stream=stream),),
            "codes": lambda stream=None: qli.prepare_q(x, pos, prep, quant_mode=qli.QUANT_INT8, stream=stream),
            "append": append}, (x, pos, kv)


@pytest.mark.parametrize("name", ["rotate", "prepare", "codes", "append"])
def test_on_another_stream(name):
    import torch
    calls, _ = _calls()
    want = [t.clone() for t in calls[name]()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = calls[name](stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["rotate", "prepare", "codes", "append"])
def test_captured_and_replayed(name):
    import torch
    calls, inputs = _calls()
    other, changed = _calls(seed=7)
    calls[name]()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = calls[name]()
    for a, b in zip(inputs, changed):
        a.copy_(b)
    g.replay()
    replayed = [t.clone() for t in got]
    want = calls[name]()
    assert all(torch.equal(a, b) for a, b in zip(replayed, want))
