"""Inputs and tolerances shared by the tests of the 8-bit KV cache."""
import numpy as np

from oracle import kv8
from sparse_attention_indexer_qli_gb300 import synth

D = 512


class KVCase:
    """A batch over paged 8-bit KV rows, in host memory. Every byte of the pool
    that no row of a request uses is random, so unused rows hold NaN codes,
    NaN, infinite and negative scales."""

    def __init__(self, seed, raw, q_lens, ratio, H, quant, K=None, rows_per_page=None,
                 row_size=1.0, spare=3, q_size=1.0):
        self.rng = rng = np.random.default_rng(seed)
        self.ratio, self.H, self.quant = ratio, H, quant
        self.R = R = rows_per_page or {1: 128, 2: 64}[ratio]
        self.layout = synth.kv8_layout(R)
        raw = np.asarray(raw, dtype=np.int64)
        q_lens = np.asarray(q_lens, dtype=np.int64)
        self.B, self.q_lens = len(raw), q_lens
        self.k_lens = (raw // ratio).astype(np.int32)
        self.residual = (raw % ratio).astype(np.int32) if ratio > 1 else None
        self.cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.T = int(self.cu[-1])
        per = -(-self.k_lens.astype(np.int64) // R)
        self.pages = int(per.sum()) + spare
        perm = rng.permutation(self.pages).astype(np.int32)
        self.bt = np.full((self.B, max(1, int(per.max()))), -5, dtype=np.int32)
        at = 0
        for b in range(self.B):
            self.bt[b, :per[b]] = perm[at:at + per[b]]
            at += per[b]
        self.codes, self.scales = [], []
        for b in range(self.B):
            n = int(self.k_lens[b])
            x = rng.standard_normal((n, D)) * np.exp(row_size * 0.5 * rng.standard_normal((n, 1)))
            c, s = kv8.quantise_rows(kv8.f32_to_bf16(x), quant)
            self.codes.append(c)
            self.scales.append(s)
        self.q = kv8.f32_to_bf16(q_size * rng.standard_normal((self.T, H, D)))
        self.indices = None
        if K is not None:
            self.indices = np.full((self.T, 1, K), -1, dtype=np.int32)
            for t in range(self.T):
                n = int(self.k_lens[self.request(t)])
                m = min(n, K if rng.random() < 0.7 else int(rng.integers(0, K + 1)))
                self.indices[t, 0, :m] = np.sort(rng.choice(n, m, replace=False)) if m else []

    def request(self, t):
        return int(np.searchsorted(self.cu[1:], t, side="right"))

    def positions(self, t, window=0):
        """Positions token t attends to (listed or visible)."""
        b = self.request(t)
        if self.indices is not None:
            js = self.indices[t, 0]
            return js[js >= 0]
        res = 0 if self.residual is None else int(self.residual[b])
        V = kv8.visible(int(self.q_lens[b]), t - int(self.cu[b]), int(self.k_lens[b]), res, self.ratio)
        return np.arange(max(0, V - window) if window else 0, V)

    def kv(self, b, js):
        return kv8.rows(self.codes[b][js], self.scales[b][js], self.quant)

    def pool(self):
        p = self.rng.integers(0, 256, size=(self.pages, self.layout["page_stride"]), dtype=np.uint8)
        L, R = self.layout, self.R
        for b in range(self.B):
            for i in range(-(-int(self.k_lens[b]) // R)):
                c, s = self.codes[b][i * R:(i + 1) * R], self.scales[b][i * R:(i + 1) * R]
                page = p[self.bt[b, i]]
                page[L["kv_offset"]:L["kv_offset"] + c.size] = c.reshape(-1)
                page[L["kv_scale_offset"]:L["kv_scale_offset"] + 2 * len(s)] = s.view(np.uint8)
        return p

    def geometry(self):
        return {"rows_per_page": self.R, "page_stride": self.layout["page_stride"],
                "kv_offset": self.layout["kv_offset"],
                "kv_scale_offset": self.layout["kv_scale_offset"], "quant_mode": self.quant}

    def upload(self, dev="cuda"):
        import torch
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        kw = dict(self.geometry(), q=t(self.q.view(np.int16)).view(torch.bfloat16),
                  cu_seqlens_q=t(self.cu), cache=t(self.pool()), block_table=t(self.bt))
        if self.indices is not None:
            kw["indices"] = t(self.indices)
        else:
            kw.update(k_lens=t(self.k_lens), ratio=self.ratio,
                      residual=None if self.residual is None else t(self.residual))
        return kw


def attention_bounds(q, kv, o, lse, scale):
    """Elementwise bounds of |out - o| [H, D] and |lse_gpu - lse| [H] for q [H, D]
    and kv [n, D], from the arithmetic:
      - codes and queries multiply exactly; a sum of 512 FP32 terms is off by
        at most 512 * 2^-24 of the sum of magnitudes, twice that if the adder
        truncates, so z by dz = 2^-14 * scale * max_j sum_d |q kv_j|, plus the
        FP32 products that turn it into an exponent (6 * 2^-24 of |z|) and the
        exponential's own 2^-21;
      - a weight moves by that twice over (itself and its share of the
        normaliser) and by the FP16 rounding of weight times scale (2^-11);
        weights below 2^-31 of the head's largest may vanish;
      - FP32 sums of n terms: n * 2^-23;
      - out is rounded to BF16 (2^-8 of the value).
    """
    if kv.shape[0] == 0:
        return np.zeros(q.shape), np.zeros(q.shape[0])
    n = kv.shape[0]
    mag = np.abs(kv) @ np.abs(q).T * abs(scale)                       # [n, H]
    dz = mag.max(axis=0) * (2.0 ** -14 + 6 * 2.0 ** -24) + 2.0 ** -21
    top = np.abs(kv).max()
    dw = 2.0 ** -11 + 2 * dz + n * 2.0 ** -23 + n * 2.0 ** -31
    do = dw * (1 + dw) * top
    return do[:, None] * np.ones(q.shape[1]) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(o), \
        dz + (n * 2.0 ** -23) + 2.0 ** -21 * (1 + np.abs(lse))
