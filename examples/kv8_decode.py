"""One decode step of an attention layer over an 8-bit page pool.

The pages hold, per position, an 8-bit latent KV row of 512 values with its FP16
scale and the index-K row of the indexer with its own (synth.kv8_layout). The
step, as a serving loop makes it for a batch of requests with one new token each:

  1. the new tokens' KV rows and index-K rows are quantised into their slots;
  2. the indexer scores every visible position and picks the best;
  3. each token attends over a window of the latest positions, and over the
     picked ones before the window, so that none counts twice;
  4. the two stages are merged by their log-sum-exps;
  5. the rows of one request's window are read back, for example to hand the
     request over to another cache.

Run: python examples/kv8_decode.py [--quant int8|fp8] [--requests N] [--check]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

HEADS, INDEX_HEADS, D = 64, 64, 512


class Pool:
    """A page pool of 8-bit KV rows and index-K rows, and the requests on it."""

    def __init__(self, lengths, room, quant_mode, seed=0, device="cuda"):
        import torch

        from sparse_attention_indexer_qli_gb300 import qli, synth
        self.R, self.quant_mode = 128, quant_mode
        self.layout = synth.kv8_layout(self.R)
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.g = g
        per = [-(-(n + room) // self.R) for n in lengths]
        perm = torch.randperm(sum(per) + 2, generator=g, device=device).to(torch.int32)
        self.block_table = torch.zeros(len(lengths), max(per), dtype=torch.int32, device=device)
        at = 0
        for b, n in enumerate(per):
            self.block_table[b, :n] = perm[at:at + n]
            at += n
        self.cache = torch.zeros(sum(per) + 2, self.layout["page_stride"], dtype=torch.uint8, device=device)
        self.lengths = torch.zeros(len(lengths), dtype=torch.int32, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        for b, n in enumerate(lengths):                 # the prompts, as a prefill leaves them
            self.append(torch.full((n,), b, device=device), torch.arange(n, device=device),
                        self.random(n, D), self.random(n, 128))
        self.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
        self.qli = qli

    def random(self, *shape):
        import torch
        return torch.randn(*shape, device=self.cache.device, generator=self.g).to(torch.bfloat16)

    def slots(self, request, position):
        """Page slots of positions [n] of requests [n]."""
        page = self.block_table[request, position // self.R].long()
        return page * self.R + position % self.R

    def append(self, request, position, kv, index_k):
        from sparse_attention_indexer_qli_gb300 import qli
        L, slots = self.layout, self.slots(request, position)
        pages = dict(rows_per_page=self.R, page_stride=L["page_stride"], err_word=self.err,
                     quant_mode=self.quant_mode)
        qli.write_kv(kv, slots, self.cache, kv_offset=L["kv_offset"],
                     kv_scale_offset=L["kv_scale_offset"], **pages)
        qli.write_index_k(index_k, slots, self.cache, k_offset=L["k_offset"],
                          scale_offset=L["scale_offset"], **pages)

    def kv_geometry(self):
        L = self.layout
        return dict(rows_per_page=self.R, page_stride=L["page_stride"], kv_offset=L["kv_offset"],
                    kv_scale_offset=L["kv_scale_offset"], quant_mode=self.quant_mode)


def decode_step(pool: Pool, topk: int, window: int):
    """Appends one token to every request and attends for it. Returns the step's
    tensors by name."""
    import torch

    from sparse_attention_indexer_qli_gb300 import qli
    B, dev = pool.lengths.numel(), pool.cache.device
    request = torch.arange(B, device=dev)
    pool.append(request, pool.lengths.long(), pool.random(B, D), pool.random(B, 128))
    pool.lengths += 1
    cu = torch.arange(B + 1, dtype=torch.int32, device=dev)
    # the indexer over the index-K rows
    codes, scales = qli.quantize_q(pool.random(B, INDEX_HEADS, 128), quant_mode=pool.quant_mode)
    weights = (0.1 * torch.randn(B, INDEX_HEADS, device=dev, generator=pool.g)).to(torch.float16)
    L = pool.layout
    indices, _ = qli.run(codes, cu, pool.lengths, None, pool.cache, pool.block_table, weights,
                         scales.view(torch.float16), ratio=1, rows_per_page=pool.R,
                         page_stride=L["page_stride"], k_offset=L["k_offset"],
                         scale_offset=L["scale_offset"], topk=topk, quant_mode=pool.quant_mode)
    # the window's positions are the other stage's
    indices.masked_fill_(indices >= (pool.lengths - window)[:, None, None], -1)
    # the two stages over the KV rows, and their merge
    q, scale = pool.random(B, HEADS, D), 1.0 / math.sqrt(D)
    picked = qli.kv_attention(q, cu, pool.cache, pool.block_table, indices=indices, scale=scale,
                              err_word=pool.err, **pool.kv_geometry())
    latest = qli.kv_attention(q, cu, pool.cache, pool.block_table, k_lens=pool.lengths, window=window,
                              scale=scale, err_word=pool.err, **pool.kv_geometry())
    out, lse = qli.merge_attention([picked[0], latest[0]], [picked[1], latest[1]])
    n = int(min(window, pool.lengths[0]))
    last = torch.arange(int(pool.lengths[0]) - n, int(pool.lengths[0]), device=dev)
    rows = qli.read_kv(pool.cache, pool.slots(torch.zeros_like(last), last), err_word=pool.err,
                       **pool.kv_geometry())
    return dict(q=q, scale=scale, indices=indices, window=window, out=out, lse=lse, rows=rows)


def check(pool: Pool, step: dict) -> float:
    """Largest difference of the step's output from attention computed on the rows
    read back, in FP32."""
    import torch
    worst = 0.0
    for b in range(pool.lengths.numel()):
        n = int(pool.lengths[b])
        every = torch.arange(n, device=pool.cache.device)
        kv = pool.qli.read_kv(pool.cache, pool.slots(torch.full_like(every, b), every),
                              **pool.kv_geometry()).float()
        picked = step["indices"][b, 0]
        pos = torch.cat([picked[picked >= 0].long(), every[max(0, n - step["window"]):]])
        z = step["scale"] * step["q"][b].float() @ kv[pos].T
        worst = max(worst, float((torch.softmax(z, 1) @ kv[pos] - step["out"][b].float()).abs().max()),
                    float((torch.logsumexp(z, 1) - step["lse"][b]).abs().max()))
    return worst


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--quant", default="fp8", choices=["int8", "fp8"])
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--context", type=int, default=8192)
    ap.add_argument("--topk", type=int, default=2048)
    ap.add_argument("--window", type=int, default=128)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--check", action="store_true", help="compare with attention over the rows read back")
    args = ap.parse_args(argv)
    import torch

    from sparse_attention_indexer_qli_gb300 import qli
    mode = qli.QUANT_INT8 if args.quant == "int8" else qli.QUANT_FP8
    lengths = [max(1, args.context * (b + 1) // args.requests) for b in range(args.requests)]
    pool = Pool(lengths, args.steps, mode)
    for i in range(args.steps):
        step = decode_step(pool, args.topk, args.window)
        torch.cuda.synchronize()
        line = "step %d: %d requests, up to %d positions" % (i, args.requests, int(pool.lengths.max()))
        if args.check:
            line += ", largest difference %.2e" % check(pool, step)
        print(line)
    if int(pool.err.item()):
        raise SystemExit("device error word %d" % int(pool.err.item()))


if __name__ == "__main__":
    main()
