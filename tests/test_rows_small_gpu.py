"""Norms of rows of every size under an eps that does not cover their squares (0 among
them), against the float64 oracle. Bounds as in test_rows_gpu.py: 2^-18 of the value from
the norm, 2^-18 of the row's mean magnitude over its deviation from the layer norm's mean,
which is moreover a multiple of 2^-149 (half of that over the deviation)."""
import numpy as np
import pytest

from oracle import kv8
from oracle import rows as oracle
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli
from test_rows_gpu import bf16_up, f64, near_bf16, near_codes, positions, turn_error, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    qli.lib()


def rows_of_all_sizes(D, seed):
    """BF16 rows of sizes 2^-131 to 2^56; a few where one value is far above the rest."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((210, D)) * 2.0 ** np.linspace(-131, 56, 210)[:, None]
    v[200:] = rng.integers(-4, 5, size=(10, D)) * 2.0 ** -133
    v[200:, 0] = 2.0 ** -131
    v[::17, D // 2] = 2.0 ** np.linspace(-131, 56, 13)
    return kv8.f32_to_bf16(rng.permutation(v))


def normed(x, norm, w, b, eps):
    v = kv8.bf16_to_f64(x)
    y = oracle.normalise(v, norm, w, b, eps)
    err = 2.0 ** -18 * (np.abs(y) + (0 if b is None else np.abs(b)))
    if norm == "layer":
        dev = np.sqrt(v.var(axis=-1, keepdims=True) + eps)
        err = err + (2.0 ** -18 * np.abs(v).mean(axis=-1, keepdims=True) + 2.0 ** -150) / dev * np.abs(w)
    return y, err


EPS = [0.0, 1.5e-45, 1e-38, 2.0 ** -101, 2.0 ** -99]


@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_rows_of_all_sizes(D, norm, eps):
    rng = np.random.default_rng(D)
    x = rows_of_all_sizes(D, D + 1)
    w = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32)
    b = (0.3 * rng.standard_normal(D)).astype(np.float32) if norm == "layer" else None
    prep = qli.RowPrep(D, norm=norm, weight=up(w), bias=None if b is None else up(b), eps=eps)
    y, err = normed(x, norm, w, b, float(np.float32(eps)))
    near_bf16(f64(qli.prepare_q(bf16_up(x)[:, None], None, prep))[:, 0], y, err)
    if D == 128:
        for quant in (kv8.INT8, kv8.FP8):
            codes, scales = qli.prepare_q(bf16_up(x)[:, None], None, prep, quant_mode=quant)
            near_codes(codes.cpu().numpy().view(np.uint8)[:, 0], scales.cpu().numpy().view(np.uint16)[:, 0], y, err, quant)


@pytest.mark.parametrize("quant", [0, kv8.INT8, kv8.FP8], ids=["bf16", "i8", "f8"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("dim,offset,half", [(64, 32, False), (64, 64, True), (32, 48, True), (128, 0, True), (128, 0, False)])
def test_rows_of_all_sizes_rotated(dim, offset, half, norm, quant):
    x, pos = rows_of_all_sizes(128, dim + offset), positions(np.random.default_rng(7), 210)
    r = qli.Rotary(dim, layout="half" if half else "interleaved")
    prep = qli.RowPrep(128, norm=norm, eps=0.0, rotary=r, offset=offset)
    y, err = normed(x, norm, np.ones(128), None, 0.0)
    first = offset + (np.arange(dim // 2) if half else 2 * np.arange(dim // 2))
    second = first + (dim // 2 if half else 1)
    both = err[:, first] + err[:, second]
    err[:, first] = err[:, second] = both
    err, y = err + turn_error(y, r, offset, half), oracle.rotate(y, pos, r.frequencies, offset, half)
    if quant == 0:
        near_bf16(f64(qli.prepare_q(bf16_up(x)[:, None], up(pos), prep))[:, 0], y, err)
    else:
        codes, scales = qli.prepare_q(bf16_up(x)[:, None], up(pos), prep, quant_mode=quant)
        near_codes(codes.cpu().numpy().view(np.uint8)[:, 0], scales.cpu().numpy().view(np.uint16)[:, 0], y, err, quant)


def of_usual_size(D, seed):
    return kv8.f32_to_bf16(np.random.default_rng(seed).standard_normal((210, D)))


@pytest.mark.parametrize("kinds", ["both", "kv-small", "index-small", "index-plain"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_cache_rows_of_all_sizes(norm, kinds):
    """Also with the other kind under a usual eps, or without a norm."""
    import torch
    eps = {"both": (0.0, 0.0), "kv-small": (0.0, 1e-5), "index-small": (1e-5, 0.0), "index-plain": (0.0, None)}[kinds]
    x, k = (rows_of_all_sizes(d, 31) if e == 0.0 else of_usual_size(d, 32) for d, e in zip((512, 128), eps))
    n, stride = 210, 128 * (1024 + 130)
    w, wk = (np.random.default_rng(33).uniform(0.5, 2, d).astype(np.float32) for d in (512, 128))
    index = qli.RowPrep(128) if eps[1] is None else qli.RowPrep(128, norm=norm, weight=up(wk), eps=eps[1])
    cache = torch.zeros(2, stride, dtype=torch.uint8, device="cuda")
    qli.append_kv(bf16_up(x), bf16_up(k), None, torch.arange(n, device="cuda"), cache, rows_per_page=128, page_stride=stride,
                  kv_mode=qli.KV_BF16, quant_mode=qli.QUANT_FP8, k_offset=128 * 1024, scale_offset=128 * 1152,
                  kv_prep=qli.RowPrep(512, norm=norm, weight=up(w), eps=eps[0]), index_prep=index)
    page = cache.cpu().numpy()
    part = lambda at, width, kind: page[:, at:at + 128 * width].copy().view(kind).reshape(256, -1)[:n]  # noqa: E731
    near_bf16(kv8.bf16_to_f64(part(0, 1024, np.uint16)), *normed(x, norm, w, None, float(np.float32(eps[0]))))
    y, err = ((kv8.bf16_to_f64(k), np.zeros(k.shape)) if eps[1] is None else
              normed(k, norm, wk, None, float(np.float32(eps[1]))))
    near_codes(part(128 * 1024, 128, np.uint8), part(128 * 1152, 2, np.uint16)[:, 0], y, err, kv8.FP8)


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_a_row_without_a_size_stays_alone(norm):
    """Under eps 0 a row of zeros (or of equal values, about their mean) is 0 / 0."""
    v = np.random.default_rng(34).standard_normal((9, 128)) * 2.0 ** -120
    v[4] = 0 if norm == "rms" else 2.0 ** -121
    x = kv8.f32_to_bf16(v)
    got = f64(qli.prepare_q(bf16_up(x)[:, None], None, qli.RowPrep(128, norm=norm, eps=0.0)))[:, 0]
    assert np.isnan(got[4]).all()
    fine = np.arange(9) != 4
    near_bf16(got[fine], *normed(x[fine], norm, np.ones(128), None, 0.0))
