"""CPU oracle of the 8-bit KV cache: row quantisation, read-back, attention over
the rows and the merge of attention stages — TEST INFRASTRUCTURE.

Only the tests and the example's check may import this module. It shares no
code with the CUDA library and reads nothing the CUDA path produced. Sums are
float64 (numpy); the FP32 and FP16 roundings that the definition names are
taken where it names them:

  row        s = FP16(FP32(amax / Q)) capped at 65504, c = code(FP32(x / s)),
             Q = 127 (INT8, ties to even, clamped) or 448 (E4M3 "fn": bias 7,
             ties to even, saturated); s = 0 gives codes 0 and scale +0
  read       BF16(c * s)
  attention  kv_j = c_j s_j, z_j = scale q . kv_j, softmax over the token's
             positions; none give out 0 and lse -inf
  merge      weights exp(lse_i - logsumexp(lse))
"""
from __future__ import annotations

import numpy as np

INT8, FP8 = 2, 1


def bf16_to_f64(bits: np.ndarray) -> np.ndarray:
    b = np.ascontiguousarray(bits, dtype=np.uint16)
    return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f32_to_bf16(x: np.ndarray) -> np.ndarray:
    """Finite FP32 values to BF16 bits, ties to even."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def e4m3_values() -> np.ndarray:
    """Value of every E4M3 code (NaN for 0x7F and 0xFF)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[(c & 0x7F) == 0x7F] = np.nan
    return np.where(c & 0x80, -v, v)


def e4m3_codes(x: np.ndarray) -> np.ndarray:
    """Nearest E4M3 code, ties to the even code, saturated to +-448."""
    grid = e4m3_values()[:127]
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def quantise_rows(x_bits: np.ndarray, quant: int):
    """BF16 rows [n, D] -> (codes uint8 [n, D], scales FP16 bits uint16 [n])."""
    x = bf16_to_f64(x_bits).astype(np.float32)
    top = np.float32(127.0 if quant == INT8 else 448.0)
    amax = np.abs(x).max(axis=1)
    with np.errstate(over="ignore"):
        s = (amax / top).astype(np.float16)
    s = np.where(np.isinf(s), np.float16(65504.0), s)
    d = s.astype(np.float32)
    y = np.divide(x, d[:, None], out=np.zeros_like(x), where=d[:, None] != 0)
    if quant == INT8:
        c = np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    else:
        c = e4m3_codes(y.astype(np.float64))
        c[d == 0] = 0
    return c, s.view(np.uint16)


def values(codes: np.ndarray, quant: int) -> np.ndarray:
    return codes.view(np.int8).astype(np.float64) if quant == INT8 else e4m3_values()[codes]


def rows(codes: np.ndarray, scales: np.ndarray, quant: int) -> np.ndarray:
    """float64 values of rows [n, D] with FP16 scale bits [n]."""
    return values(codes, quant) * scales.view(np.float16).astype(np.float64)[:, None]


def visible(q_len: int, i: int, k_len: int, residual: int, ratio: int) -> int:
    """Compressed positions the i-th of a request's q_len queries sees: the
    queries are the last raw tokens, position j ends at raw token
    j * ratio + ratio - 1."""
    seen = k_len * ratio + residual - q_len + i + 1
    return max(0, min(k_len, seen // ratio))


def attend(q: np.ndarray, kv: np.ndarray, scale: float):
    """q [H, D], kv [n, D] float64 -> (o [H, D], lse [H])."""
    if kv.shape[0] == 0:
        return np.zeros(q.shape), np.full(q.shape[0], -np.inf)
    z = scale * (kv @ q.T)
    m = z.max(axis=0)
    p = np.exp(z - m)
    l = p.sum(axis=0)
    return (p.T @ kv) / l[:, None], m + np.log(l)


def merge(outs, lses):
    """Parts [P][T, H, D], [P][T, H] float64 -> (out, lse)."""
    lse = np.stack(lses)
    m = lse.max(axis=0)
    w = np.exp(lse - np.where(np.isneginf(m), 0.0, m))
    total = w.sum(axis=0)
    out = np.zeros(outs[0].shape)
    for o, wi in zip(outs, w):
        out += np.where(wi[..., None] > 0, wi[..., None] * o, 0.0)
    with np.errstate(divide="ignore"):
        return out / np.where(total == 0, 1.0, total)[..., None], m + np.log(total)
