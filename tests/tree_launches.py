"""How the attention of drafted trees splits a call: what a call launches, read out of a
captured graph, and the library's rules restated (test_kv_tree_plan_gpu.py holds one
against the other)."""
import os
import re
import tempfile
import warnings

HT, WORST, POS, CHUNK, MAX_STACK = 64, 2 ** 31 - 1, 64, 512, 8
KINDS = {0: "causal", 1: "single", 2: "groups"}


def tiles(H, tokens):
    return -(-tokens * H // HT)


def most_units(T, words, window, positions, stack):
    """Most units of a row tile; `positions`: those a row of the block table holds."""
    n = min(positions, WORST)
    if window:
        n = min(n, window + (min(T, 64 * words) if stack > 1 else 0))
    return max(1, -(-n // POS))


def stack_of(H, T, B, words, window, positions, sms):
    """Tokens that share row tiles."""
    units = most_units(T, words, window, positions, 1)
    if (1 if units <= 2 else units) * T * tiles(H, 1) <= sms:
        return 1
    best = 1
    for k in range(2, min(MAX_STACK, (T - 1) // B + 1) + 1):
        if tiles(H, k) * best < tiles(H, best) * k:
            best = k
    return best


def split(H, T, B, words, window, positions, sms):
    """The call's launches: (kind, CTAs), and after those that cut row tiles
    ("join", few row tiles or not)."""
    stack = stack_of(H, T, B, words, window, positions, sms)
    most = most_units(T, words, window, positions, stack)
    groups = lambda tokens: min(tokens, tokens // stack + B + 3)  # noqa: E731
    whole_units = 4 if stack > 1 else 2
    ht = HT
    while ht > 16 and (1 if most <= whole_units else most) * groups(T) * -(-stack * H // (ht // 2)) <= sms:
        ht //= 2
    hg = -(-stack * H // ht)
    out = []
    for t0 in range(0, T, CHUNK):
        tc = min(CHUNK, T - t0)
        n = groups(tc) * hg
        likely = (n + -(-tc // stack) * hg) // 2 if stack > 1 else n
        whole = most <= whole_units and likely <= sms
        ctas = n if whole else min(n * most, sms)
        out.append((KINDS[2 if stack > 1 else 1], ctas))
        if ctas > 1 and not whole:
            out.append(("join", 8 * likely <= ctas <= 256))
    return out


def launches(call):
    """The same of a call, from the names and grids of the kernels in its graph."""
    import torch
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    with tempfile.TemporaryDirectory() as d, warnings.catch_warnings():
        warnings.simplefilter("ignore")
        path = os.path.join(d, "graph.dot")
        g.debug_dump(path)
        text = open(path).read()
    names = re.findall(r"\| (_Z\S*?)\\<\\<\\<(\\\{[^}]*\}|\d+),", text)
    # the graph prints its kernels in the order they were queued
    out = []
    for name, grid in names:
        main, join = re.search(r"kv_attn_kernelILb[01]ELi(\d)E", name), re.search(r"merge_pieces_kernelILb([01])ELb([01])E", name)
        assert main or join, name
        out.append((KINDS[int(main.group(1))], int(grid)) if main else ("join", join.group(2) == "1"))
    assert out, text
    return out


def split_of(kw, window, sms):
    """split() of the arguments of a call."""
    T, H, _ = kw["q"].shape
    mask, table = kw["tree_mask"], kw["block_table"]
    return split(H, T, table.shape[0], mask.shape[1] if mask.dim() == 2 else 1, window,
                 table.shape[1] * kw["rows_per_page"], sms)


def wide(kw, pages):
    """The call with a block table of that many pages a request (those added are outside the pool)."""
    import torch
    table = kw["block_table"]
    more = torch.full((table.shape[0], pages - table.shape[1]), -5, dtype=table.dtype, device=table.device)
    return dict(kw, block_table=torch.cat([table, more], 1).contiguous())
