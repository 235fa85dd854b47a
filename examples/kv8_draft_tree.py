"""One verification step of a drafted token tree over an 8-bit page pool.

Every request has a prefix in the pages and a tree of drafted tokens behind it. The
step, for one attention layer, from the layer's projections:

  1. the drafted tokens' KV rows and index-K rows are normed, rotated to their
     positions (prefix + depth) and quantised into the next page slots, in one kernel;
  2. their queries are normed and rotated, the indexer's rotated and quantised;
  3. the indexer picks positions of the prefix for each token;
  4. each token attends over the last positions of its own path through the tree (a
     window), and over the picked ones before it;
  5. the stages are merged and the output's tail is rotated back, in place;
  6. of each request one path is accepted, and its rows are appended again behind
     the prefix, where the next step expects them.

Run: python examples/kv8_draft_tree.py [--quant int8|fp8] [--requests N] [--check]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

INDEX_HEADS, D, DI, ROT, WINDOW = 64, 512, 128, 64, 128


class Layer:
    """The plans of a layer: the rotation and what is done to each kind of row."""

    def __init__(self, g, device="cuda"):
        import torch

        from sparse_attention_indexer_qli_gb300 import qli

        def weights(n):
            return 1 + 0.1 * torch.randn(n, device=device, generator=g)
        self.rotary = qli.Rotary(ROT, layout="interleaved", factor=16.0, trained=8192)
        self.queries = qli.RowPrep(D, norm="rms", weight=weights(D), rotary=self.rotary, offset=D - ROT)
        self.kv = qli.RowPrep(D, norm="rms", weight=weights(D), rotary=self.rotary, offset=D - ROT)
        self.index_k = qli.RowPrep(DI, norm="layer", weight=weights(DI), bias=0.1 * weights(DI), rotary=self.rotary)
        self.index_q = qli.RowPrep(DI, rotary=self.rotary)


class Requests:
    """A page pool with the prefixes of some requests in it."""

    def __init__(self, lengths, room, quant_mode, seed=0, device="cuda"):
        import torch

        from sparse_attention_indexer_qli_gb300 import synth
        self.R, self.quant_mode, self.device = 128, quant_mode, device
        self.layout = synth.kv8_layout(self.R)
        self.g = torch.Generator(device=device)
        self.g.manual_seed(seed)
        self.layer = Layer(self.g, device)
        per = [-(-(n + room) // self.R) for n in lengths]
        perm = torch.randperm(sum(per) + 2, generator=self.g, device=device).to(torch.int32)
        self.block_table = torch.zeros(len(lengths), max(per), dtype=torch.int32, device=device)
        at = 0
        for b, n in enumerate(per):
            self.block_table[b, :n] = perm[at:at + n]
            at += n
        self.cache = torch.zeros(sum(per) + 2, self.layout["page_stride"], dtype=torch.uint8, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device=device)
        for b, n in enumerate(lengths):                # the prefixes, as a prefill leaves them
            pos = torch.arange(n, device=device)
            self.append(torch.full_like(pos, b), pos, pos, self.random(n, D), self.random(n, DI))

    def random(self, *shape):
        import torch
        return torch.randn(*shape, device=self.device, generator=self.g).to(torch.bfloat16)

    def append(self, request, place, position, kv, index_k):
        """Rows of `request` [n] into its places [n] of the cache, rotated to positions [n]."""
        import torch

        from sparse_attention_indexer_qli_gb300 import qli
        slots = self.block_table[request, place // self.R].long() * self.R + place % self.R
        qli.append_kv(kv, index_k, position.to(torch.int32), slots, self.cache, kv_prep=self.layer.kv,
                      index_prep=self.layer.index_k, rows_per_page=self.R, err_word=self.err,
                      kv_mode=self.quant_mode, quant_mode=self.quant_mode, **self.layout)

    def kv_geometry(self):
        L = self.layout
        return dict(rows_per_page=self.R, page_stride=L["page_stride"], kv_offset=L["kv_offset"],
                    kv_scale_offset=L["kv_scale_offset"], quant_mode=self.quant_mode)


def draft(parents, device="cuda"):
    """(masks int64 [n], depths [n]) of a tree: parents[i] < i, or -1 for the prefix."""
    import torch
    masks, depths = [], []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
        depths.append(depths[p] + 1 if p >= 0 else 0)
    signed = [m - (1 << 64) if m >> 63 else m for m in masks]
    return torch.tensor(signed, dtype=torch.int64, device=device), torch.tensor(depths, device=device)


def verify_step(r: Requests, parents, heads=64, topk=512):
    """Attends for the same tree behind every request. Returns the step's tensors by name."""
    import torch

    from sparse_attention_indexer_qli_gb300 import qli
    dev, n, B = r.device, len(parents), r.lengths.numel()
    masks, depths = draft(parents, dev)
    request = torch.arange(B, device=dev).repeat_interleave(n)
    node, T = torch.arange(n, device=dev).repeat(B), B * n
    prefix = r.lengths[request]
    position = (prefix + depths[node]).to(torch.int32)
    kv, index_k = r.random(T, D), r.random(T, DI)
    r.append(request, prefix.long() + node, position, kv, index_k)
    # queries
    x = r.random(T, heads, D)
    q = qli.prepare_q(x, position, r.layer.queries)
    codes, scales = qli.prepare_q(r.random(T, INDEX_HEADS, DI), position, r.layer.index_q, quant_mode=r.quant_mode)
    # the indexer over the prefix: every token on its own, with the pages of its request
    weights = (0.1 * torch.randn(T, INDEX_HEADS, device=dev, generator=r.g)).to(torch.float16)
    each, table, L = torch.arange(T + 1, dtype=torch.int32, device=dev), r.block_table[request], r.layout
    indices, _ = qli.run(codes, each, prefix, None, r.cache, table, weights, scales.view(torch.float16), ratio=1,
                         rows_per_page=r.R, page_stride=L["page_stride"], k_offset=L["k_offset"],
                         scale_offset=L["scale_offset"], topk=topk, quant_mode=r.quant_mode)
    # a token's window has its path of depth + 1 nodes and the prefix's end
    first = (prefix - (WINDOW - depths[node] - 1)).clamp(min=0)
    indices.masked_fill_(indices >= first[:, None, None], -1)
    scale, cu = 1.0 / math.sqrt(D), n * torch.arange(B + 1, dtype=torch.int32, device=dev)
    tree = masks.repeat(B)
    picked = qli.kv_attention(q, each, r.cache, table, indices=indices, scale=scale, err_word=r.err, **r.kv_geometry())
    latest = qli.kv_tree_attention(q, cu, r.cache, r.block_table, k_lens=r.lengths + n, tree_mask=tree, window=WINDOW,
                                   scale=scale, err_word=r.err, **r.kv_geometry())
    out, lse = qli.merge_attention([picked[0], latest[0]], [picked[1], latest[1]])
    merged = out.clone()
    qli.rotate(out, position, r.layer.rotary, offset=D - ROT, inverse=True, out=out)
    return dict(x=x, kv=kv, index_k=index_k, q=q, scale=scale, indices=indices, first=first, request=request, node=node,
                prefix=prefix, position=position, masks=masks, depths=depths, merged=merged, out=out, lse=lse)


def accept(r: Requests, step: dict, path):
    """Keeps the nodes of `path` (from the root on) behind every prefix."""
    import torch
    n, B = step["masks"].numel(), r.lengths.numel()
    rows = (n * torch.arange(B, device=r.device)[:, None] + torch.tensor(path, device=r.device)).reshape(-1)
    place = (step["prefix"][rows] + torch.arange(len(path), device=r.device).repeat(B)).long()
    r.append(step["request"][rows], place, step["position"][rows], step["kv"][rows], step["index_k"][rows])
    r.lengths += len(path)


def check(r: Requests, step: dict) -> float:
    """Largest difference of the step's merged output and log-sum-exps from attention
    over the rows read back, in FP32. Called before the tree's rows are overwritten."""
    import torch

    from sparse_attention_indexer_qli_gb300 import qli
    worst, n = 0.0, step["masks"].numel()
    for t in range(step["request"].numel()):
        b, p = int(step["request"][t]), int(step["prefix"][t])
        nodes = [p + i for i in range(n) if int(step["masks"][step["node"][t]]) >> i & 1]
        picked = step["indices"][t, 0]
        pos = torch.cat([picked[picked >= 0].long(), torch.arange(int(step["first"][t]), p, device=r.device),
                         torch.tensor(nodes, device=r.device)])
        slots = r.block_table[b, pos // r.R].long() * r.R + pos % r.R
        rows = qli.read_kv(r.cache, slots, **r.kv_geometry()).float()
        z = step["scale"] * step["q"][t].float() @ rows.T
        worst = max(worst, float((torch.softmax(z, 1) @ rows - step["merged"][t].float()).abs().max()),
                    float((torch.logsumexp(z, 1) - step["lse"][t]).abs().max()))
    return worst


TREE = [-1, 0, 0, 1, 1, 2, 3, -1, 7, 8]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--quant", default="fp8", choices=["int8", "fp8"])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--context", type=int, default=8192)
    ap.add_argument("--heads", type=int, default=64)
    ap.add_argument("--topk", type=int, default=512)
    ap.add_argument("--steps", type=int, default=3)
    ap.add_argument("--check", action="store_true", help="compare with attention over the rows read back")
    args = ap.parse_args(argv)
    import torch

    from sparse_attention_indexer_qli_gb300 import qli
    mode = qli.QUANT_INT8 if args.quant == "int8" else qli.QUANT_FP8
    lengths = [max(1, args.context * (b + 1) // args.requests) for b in range(args.requests)]
    r = Requests(lengths, args.steps * 4 + len(TREE), mode)
    for i in range(args.steps):
        step = verify_step(r, TREE, args.heads, args.topk)
        torch.cuda.synchronize()
        line = "step %d: %d requests, up to %d positions" % (i, args.requests, int(r.lengths.max()))
        if args.check:
            line += ", largest difference %.2e" % check(r, step)
        print(line)
        accept(r, step, [0, 1, 3] if i % 2 else [7, 8])
    if int(r.err.item()):
        raise SystemExit("device error word %d" % int(r.err.item()))


if __name__ == "__main__":
    main()
