"""Cases of the operators around the paged cache: the rotation of positions
(`qli.rotate`), the norm and rotation of queries (`qli.prepare_q`), the same for
new cache rows on their way into the pages (`qli.append_kv`) and the attention
of drafted token trees over 8-bit rows (`qli.kv_tree_attention`), each beside its
plain form in elementary torch operations.

A page holds R = 128 rows: the KV rows (512 values each: BF16, or 8-bit codes
with the rows' FP16 scales behind them), then the index K rows (128 codes each)
and their FP16 scales.
"""
import functools
import math

import numpy as np
import torch

own = False

D, DI, ROWS = 512, 128, 128     # values of a KV row and of an index K row, rows per page
INT8, FP8, BF16 = 2, 1, 0       # the framework's quantisation modes; BF16 rows
SCALE = 1.0 / math.sqrt(D)
EPS = 1e-6
DEV = "cuda"


# ---- cases -------------------------------------------------------------------
# rot: values of a row that rotate; offset: the first of them; half: pairs half of
# `rot` apart, else neighbours; factor: context extension (1: none); far: positions
# below it; pad: values between rows of a wider tensor.

def listed():
    return [
        # a decode batch's attention output: the tail of every head rotated back, in place
        {"name": "rotate-decode", "op": "rotate", "T": 64, "H": 64, "D": 512, "rot": 64, "offset": 448, "half": False,
         "inverse": True, "inplace": True, "factor": 1.0, "far": 32768, "pad": 0},
        # the queries of an odd prefill chunk, cut out of a wider projection, far into an extended context
        {"name": "rotate-chunk-half", "op": "rotate", "T": 4093, "H": 33, "D": 512, "rot": 64, "offset": 448,
         "half": True, "inverse": False, "inplace": False, "factor": 16.0, "far": 1000000, "pad": 64},
        # the index queries of one decoding request, quantised
        {"name": "queries-one-i8", "op": "queries", "T": 1, "H": 32, "D": 128, "rot": 64, "offset": 0, "half": True,
         "factor": 1.0, "far": 8192, "norm": "none", "quant": INT8},
        # the index queries of a prefill chunk, quantised
        {"name": "queries-chunk-f8", "op": "queries", "T": 4096, "H": 64, "D": 128, "rot": 64, "offset": 0, "half": True,
         "factor": 16.0, "far": 131072, "norm": "none", "quant": FP8},
        # the attention queries of a prefill chunk: RMS norm of each head, the tail rotated
        {"name": "queries-chunk-bf16", "op": "queries", "T": 2047, "H": 64, "D": 512, "rot": 64, "offset": 448,
         "half": False, "factor": 16.0, "far": 131072, "norm": "rms", "quant": BF16},
        # one new position for each of 64 decoding requests
        {"name": "append-decode-i8", "op": "append", "n": 64, "kv": INT8, "index": INT8, "rot": 64, "half": False,
         "factor": 1.0, "far": 32768, "pad": 0},
        # the rows of a prefill chunk over BF16 pages
        {"name": "append-chunk-bf16", "op": "append", "n": 4093, "kv": BF16, "index": FP8, "rot": 64, "half": True,
         "factor": 1.0, "far": 131072, "pad": 64},
        # the rows of two 32K-token prompts
        {"name": "append-prompt-f8", "op": "append", "n": 65536, "kv": FP8, "index": FP8, "rot": 64, "half": False,
         "factor": 16.0, "far": 131072, "pad": 64},
        # one request's 8 drafted tokens over a short context
        {"name": "tree-one-f8", "op": "tree", "quant": FP8, "B": 1, "L": 8, "uneven": False, "H": 64, "lo": 2048,
         "hi": 2048, "window": 0},
        # 16 requests with trees of up to 16 tokens over 8K to 32K positions
        {"name": "tree-batch-f8", "op": "tree", "quant": FP8, "B": 16, "L": 16, "uneven": True, "H": 64, "lo": 8192,
         "hi": 32768, "window": 0},
        # the sliding-window stage of a drafting batch with few heads
        {"name": "tree-window-i8", "op": "tree", "quant": INT8, "B": 64, "L": 8, "uneven": True, "H": 16, "lo": 8192,
         "hi": 32768, "window": 128},
        # wide trees over two long contexts
        {"name": "tree-long-i8", "op": "tree", "quant": INT8, "B": 2, "L": 63, "uneven": False, "H": 128, "lo": 40001,
         "hi": 65536, "window": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "queries", "append", "tree", "tree"])
    place = {"half": rng.random() < 0.5, "factor": rng.choice([1.0, 4.0, 16.0]), "far": _log(rng, 64, 1000000)}
    if op == "append":
        return {"op": op, "n": _log(rng, 1, 65536), "kv": rng.choice([INT8, FP8, BF16]), "index": rng.choice([INT8, FP8]),
                "rot": rng.choice([32, 64, 128]), "pad": rng.choice([0, 8, 64]), **place}
    if op == "tree":
        window = rng.choice([0, 0, 0, _log(rng, 1, 1024)])
        hi = _log(rng, 100, 65536)
        case = {"op": op, "quant": rng.choice([INT8, FP8]), "B": _log(rng, 1, 64), "L": _log(rng, 1, min(100, hi // 2)),
                "uneven": rng.random() < 0.5, "H": rng.choice([8, 16, 32, 64, 64, 96, 128]),
                "lo": max(hi // 2, hi // rng.randint(1, 5)), "hi": hi, "window": window}
        return _no_larger(_no_larger(case, "L"), "B")
    if op == "rotate":
        d = rng.choice([64, 128, 192, 512])
        case = {"op": op, "T": _log(rng, 1, 4096), "H": rng.choice([1, 8, 33, 64]), "D": d,
                "inverse": rng.random() < 0.5, "inplace": rng.random() < 0.5, "pad": rng.choice([0, 8, 64])}
    else:
        d = rng.choice([64, 128, 128, 256, 512])
        case = {"op": op, "T": _log(rng, 1, 4096), "H": rng.choice([1, 8, 33, 64]), "D": d,
                "norm": rng.choice(["none", "rms", "layer"]), "quant": rng.choice([INT8, FP8, BF16]) if d == DI else BF16}
    rot = rng.choice([r for r in (16, 32, 64, 128) if r <= d])
    return _no_larger({**case, "rot": rot, "offset": rng.choice([0, d - rot]), **place}, "T")


def _no_larger(case, size):
    """The case, `size` halved until it is within the largest listed ones."""
    most = {"tree": (1.05e9, 4e12)}.get(case["op"], (2.8e8, 1e12))
    while case[size] > 1 and (work(case)["bytes"] > most[0] or work(case)["flops"] > most[1] or
                              case.get("B", 0) * case.get("hi", 0) * (D + 132) > 1e9):
        case[size] //= 2
    return case


# ---- sizes that follow from a case -------------------------------------------

def _layout(kv):
    """(kv scale offset, index offset, index scale offset, page stride) in bytes; the KV rows start the page."""
    k = ROWS * (2 * D if kv == BF16 else D + 2)
    return ROWS * D, k, k + ROWS * DI, k + ROWS * (DI + 2)


def _lengths(case):
    """Per request its positions (drafted ones included) and drafted tokens."""
    B = case["B"]
    at = (np.arange(B, dtype=np.int64) * 7919) % max(1, B)
    k = case["lo"] + (case["hi"] - case["lo"]) * at // max(1, B - 1)
    n = np.full(B, case["L"], dtype=np.int64)
    if case["uneven"]:
        n = np.maximum(1, case["L"] - (np.arange(B) * 3) % max(1, (case["L"] + 1) // 2))
    return k, np.minimum(n, k)


def work(case):
    op = case["op"]
    if op == "rotate":
        rows = case["T"] * case["H"]
        return {"bytes": rows * 4 * (case["rot"] if case["inplace"] else case["D"]) + 4 * case["T"],
                "flops": 3 * case["rot"] * rows}
    if op == "queries":
        rows, d = case["T"] * case["H"], case["D"]
        each = {"none": 0, "rms": 4, "layer": 6}[case["norm"]]
        return {"bytes": rows * (4 * d if case["quant"] == BF16 else 3 * d + 2) + 4 * case["T"],
                "flops": rows * (each * d + 3 * case["rot"] + (0 if case["quant"] == BF16 else 3 * d))}
    if op == "append":
        kv = 2 * D if case["kv"] == BF16 else D + 2
        return {"bytes": case["n"] * (2 * D + 2 * DI + kv + DI + 2 + 12), "flops": case["n"] * 8 * (D + DI)}
    k, n = _lengths(case)
    T, H, w = int(n.sum()), case["H"], case["window"]
    # of its tree's nodes a token sees its path: a handful
    path = np.minimum((n + 1) / 2.0, 6.0)
    seen = k - n + path
    rows = k.astype(float)
    if w:
        seen, rows = np.minimum(seen, w), np.minimum(rows, w + n)
    return {"bytes": float(rows.sum()) * (D + 2) + T * H * (4 * D + 4) + 8 * T * _words(case),
            "flops": 4.0 * D * H * float((seen * n).sum())}


def _words(case):
    return -(-int(_lengths(case)[1].max()) // 64)


# ---- inputs ------------------------------------------------------------------

TRAINED = 8192                   # positions that the frequencies of an extended context were made for
RAMP = (1.0, 32.0)               # turns over them between which a pair is blended


def _frequencies(case):
    """Radians per position of each pair, in FP64: base^(-2i/rot); of an extended context, pairs that turn less
    than RAMP[0] times over the trained one slow down by the factor, those above RAMP[1] keep, a blend between."""
    f = 10000.0 ** (-2.0 * np.arange(case["rot"] // 2, dtype=np.float64) / case["rot"])
    keep = np.clip((TRAINED * f / (2 * math.pi) - RAMP[0]) / (RAMP[1] - RAMP[0]), 0.0, 1.0)
    return f * (keep + (1.0 - keep) / case["factor"])


def _magnitude(case):
    return 1.0 if case["factor"] == 1.0 or case["op"] == "rotate" else 1.0 + 0.1 * math.log(case["factor"])


def _randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _rows(g, n, d):
    """BF16 rows: normal values whose size varies from row to row."""
    return (_randn(g, n, d) * torch.exp(0.5 * _randn(g, n, 1))).to(torch.bfloat16)


def _wide(rows, pad):
    """The same rows cut out of wider ones."""
    wide = torch.zeros(*rows.shape[:-1], rows.shape[-1] + pad, dtype=rows.dtype, device=DEV)
    wide[..., :rows.shape[-1]] = rows
    return wide[..., :rows.shape[-1]]


def _quantise(x, quant):
    """Rows of FP32 values -> (codes as bytes, FP16 scales)."""
    top = 127.0 if quant == INT8 else 448.0
    s = (x.abs().amax(-1) / top).clamp(max=65504.0).to(torch.float16)
    d = s.float()[..., None]
    y = x / torch.where(d == 0, 1.0, d)
    y = torch.where(d == 0, 0.0, y).clamp(-top, top)
    c = y.round().to(torch.int8) if quant == INT8 else y.to(torch.float8_e4m3fn)
    return c.view(torch.uint8), s


def _part(cache, at, width, kind):
    """[pages, ROWS, width] values of `kind` (of a byte count `width` a row) that start at byte `at` of each page."""
    size = torch.empty((), dtype=kind).element_size()
    flat = cache.view(kind)
    return torch.as_strided(flat, (cache.shape[0], ROWS, width // size), (cache.shape[1] // size, width // size, 1),
                            at // size)


def _parts(st):
    """The pool's KV rows, their scales (None for BF16), index K rows and scales."""
    s_kv, k, s_k, _ = _layout(st["kv"])
    if st["kv"] == BF16:
        kv, scales = _part(st["cache"], 0, 2 * D, torch.bfloat16), None
    else:
        kv, scales = _part(st["cache"], 0, D, torch.uint8), _part(st["cache"], s_kv, 2, torch.float16)[..., 0]
    return kv, scales, _part(st["cache"], k, DI, torch.uint8), _part(st["cache"], s_k, 2, torch.float16)[..., 0]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 17)
    op, st = case["op"], {"case": case}
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    if op != "tree":
        rng, n = np.random.default_rng(int(seed) + 7), case["n"] if op == "append" else case["T"]
        # runs of neighbouring positions, as the requests of a batch have them
        run = 1 if n <= 64 else 512
        start = rng.integers(0, case["far"], size=-(-n // run))
        pos = np.minimum(np.repeat(start, run)[:n] + np.arange(n) % run, case["far"] - 1)
        st["positions"] = up(pos.astype(np.int32))
        st["f"] = up(_frequencies(case))
        st["magnitude"] = _magnitude(case)
    if op in ("rotate", "queries"):
        T, H, d = case["T"], case["H"], case["D"]
        st["x"] = _wide(_rows(g, T * H, d).view(T, H, d), case.get("pad", 0))
    if op == "rotate":
        st["out"] = st["x"] if case["inplace"] else torch.empty(T, H, d, dtype=torch.bfloat16, device=DEV)
        return st
    if op == "queries":
        norm = case["norm"]
        st["weight"] = 1 + 0.2 * _randn(g, d) if norm != "none" else None
        st["bias"] = 0.2 * _randn(g, d) if norm == "layer" else None
        code = {BF16: torch.bfloat16, INT8: torch.int8, FP8: torch.int8}[case["quant"]]
        st["out"] = torch.empty(T, H, d, dtype=code, device=DEV)
        st["scales"] = torch.empty(T, H, dtype=torch.int16, device=DEV)
        return st
    if op == "append":
        n, st["kv"] = case["n"], case["kv"]
        pages = -(-n // ROWS) + 3
        st["cache"] = torch.zeros(pages, _layout(case["kv"])[3], dtype=torch.uint8, device=DEV)
        slots = torch.randperm(pages * ROWS, device=DEV, generator=g)[:n]
        st["slots"] = torch.where(torch.rand(n, device=DEV, generator=g) < 0.01, -1, slots)       # padding
        st["rows"], st["index"] = _wide(_rows(g, n, D), case["pad"]), _wide(_rows(g, n, DI), case["pad"])
        st["kv_weight"] = 1 + 0.2 * _randn(g, D)
        st["weight"], st["bias"] = 1 + 0.2 * _randn(g, DI), 0.2 * _randn(g, DI)
        return st
    k, n = _lengths(case)
    B, T, H = case["B"], int(n.sum()), case["H"]
    st["quant"] = st["kv"] = case["quant"]
    per = -(-k // ROWS)
    pages = int(per.sum()) + 3
    st["cache"] = torch.zeros(pages, _layout(case["quant"])[3], dtype=torch.uint8, device=DEV)
    codes, scales, _, _ = _parts(st)
    for p in range(0, pages, 2048):
        c, s = _quantise(_rows(g, min(2048, pages - p) * ROWS, D).float(), case["quant"])
        codes[p:p + 2048], scales[p:p + 2048] = c.view(-1, ROWS, D), s.view(-1, ROWS)
    rng = np.random.default_rng(int(seed))
    perm, bt = rng.permutation(pages).astype(np.int32), np.zeros((B, int(per.max())), dtype=np.int32)
    mask = np.zeros((T, _words(case)), dtype=np.uint64)
    t = 0
    for b in range(B):
        first = int(per[:b].sum())
        bt[b, :per[b]] = perm[first:first + per[b]]
        for i in range(int(n[b])):
            # drafts branch near the root: a node hangs on one of the few before it, or on the prefix
            parent = int(rng.integers(max(-1, i - 6), i)) if i else -1
            if parent >= 0:
                mask[t + i] = mask[t + parent]
            mask[t + i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
        t += int(n[b])
    st["bt"], st["mask"] = up(bt), up(mask.view(np.int64))
    st["cu"], st["k_lens"] = up(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)), up(k.astype(np.int32))
    sharp = torch.exp(0.5 * _randn(g, 1, H, 1))                          # some heads look closely
    st["q"] = (_randn(g, T, H, D) * sharp).to(torch.bfloat16)
    st["most"] = (int(n.max()), int(k.max()))
    st["out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.empty(T, H, device=DEV)
    return st


# ---- one pass ----------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return _run_own(op, state) if own else _run_plain(op, state)


def _as_values(codes, scales, quant):
    """8-bit codes as numbers (INT8 ones as BF16), and their scales."""
    c = codes.view(torch.int8).to(torch.bfloat16) if quant == INT8 else codes.view(torch.float8_e4m3fn)
    return {"codes": c, "scales": scales.view(torch.float16)}


def _pages_as_values(st):
    kv, scales, index, index_scales = _parts(st)
    return {"kv": {"rows": kv} if scales is None else _as_values(kv, scales, st["kv"]),
            "index": _as_values(index, index_scales, st["case"]["index"])}


@functools.lru_cache(maxsize=64)
def _rotary(rot, half, factor, magnitude):
    from sparse_attention_indexer_qli_gb300 import qli
    return qli.Rotary(rot, layout="half" if half else "interleaved", factor=factor, trained=TRAINED, ramp=RAMP,
                      magnitude=magnitude)


def _run_own(op, st):
    from sparse_attention_indexer_qli_gb300 import qli
    case = st["case"]
    if op == "tree":
        out, lse = qli.kv_tree_attention(
            st["q"], st["cu"], st["cache"], st["bt"], k_lens=st["k_lens"], tree_mask=st["mask"], window=case["window"],
            scale=SCALE, rows_per_page=ROWS, page_stride=_layout(st["kv"])[3], kv_offset=0,
            kv_scale_offset=_layout(st["kv"])[0], quant_mode=st["quant"], out=st["out"], lse=st["lse"])
        return {"out": out, "lse": lse}
    rotary = _rotary(case["rot"], case["half"], case["factor"], st["magnitude"])
    if op == "rotate":
        return {"out": qli.rotate(st["x"], st["positions"], rotary, offset=case["offset"], inverse=case["inverse"],
                                  out=st["out"])}
    plan = st.get("plan")
    if op == "queries":
        if plan is None:                                 # as a program makes it with the weights
            plan = st["plan"] = qli.RowPrep(case["D"], norm=None if case["norm"] == "none" else case["norm"], eps=EPS,
                                            weight=st["weight"], bias=st["bias"], rotary=rotary, offset=case["offset"])
        if case["quant"] == BF16:
            return {"out": qli.prepare_q(st["x"], st["positions"], plan, out=st["out"])}
        codes, scales = qli.prepare_q(st["x"], st["positions"], plan, out=st["out"], scale_out=st["scales"],
                                      quant_mode=case["quant"])
        return _as_values(codes, scales, case["quant"])
    if plan is None:
        plan = st["plan"] = (qli.RowPrep(D, norm="rms", weight=st["kv_weight"], eps=EPS, rotary=rotary,
                                         offset=D - case["rot"]),
                             qli.RowPrep(DI, norm="layer", weight=st["weight"], bias=st["bias"], eps=EPS, rotary=rotary))
    s_kv, k, s_k, stride = _layout(case["kv"])
    qli.append_kv(st["rows"], st["index"], st["positions"], st["slots"], st["cache"], kv_prep=plan[0], index_prep=plan[1],
                  rows_per_page=ROWS, page_stride=stride, kv_offset=0, kv_scale_offset=s_kv, k_offset=k, scale_offset=s_k,
                  kv_mode=case["kv"], quant_mode=case["index"])
    return _pages_as_values(st)


def _angles(st):
    """Cosines and sines [T, rot / 2]; the angles of far positions in FP64."""
    a = st["positions"].double()[:, None] * st["f"]
    return (a.cos() * st["magnitude"]).float(), (a.sin() * st["magnitude"]).float()


def _turned(x, cos, sin, half):
    """FP32 [..., rot] rotated by pairs."""
    if half:
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _normed(x, norm, weight, bias):
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    if norm != "none":
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    return x + bias if norm == "layer" else x


def _run_plain(op, st):
    case = st["case"]
    if op == "tree":
        return _attend(st)
    cos, sin = _angles(st)
    if op == "append":
        R, o = case["rot"], D - case["rot"]
        kv = _normed(st["rows"].float(), "rms", st["kv_weight"], None)
        kv = torch.cat([kv[:, :o], _turned(kv[:, o:], cos, sin, case["half"])], -1)
        index = _normed(st["index"].float(), "layer", st["weight"], st["bias"])
        index = torch.cat([_turned(index[:, :R], cos, sin, case["half"]), index[:, R:]], -1)
        keep = st["slots"] >= 0
        # rows without a slot are written over the row of the first that has one, with that row's own values
        src = torch.where(keep, torch.arange(keep.numel(), device=DEV), keep.to(torch.int8).argmax())
        live, slot = keep.any(), st["slots"][src].clamp(min=0)
        at = (slot // ROWS, slot % ROWS)
        rows, scales, codes, index_scales = _parts(st)
        c, s = _quantise(index, case["index"])
        new = [(codes, c), (index_scales, s)]
        if scales is None:
            new.append((rows, kv.to(torch.bfloat16)))
        else:
            new += zip((rows, scales), _quantise(kv, case["kv"]))
        for into, values in new:
            values = values[src]
            into[at] = torch.where(live, values, into[at])
        return _pages_as_values(st)
    cos, sin = cos[:, None], sin[:, None]
    o, R = case["offset"], case["rot"]
    if op == "rotate":
        if case["inverse"]:
            sin = -sin
        if not case["inplace"]:
            st["out"].copy_(st["x"])
        st["out"][..., o:o + R] = _turned(st["x"][..., o:o + R].float(), cos, sin, case["half"]).to(torch.bfloat16)
        return {"out": st["out"]}
    x = _normed(st["x"].float(), case["norm"], st["weight"], st["bias"])
    x = torch.cat([x[..., :o], _turned(x[..., o:o + R], cos, sin, case["half"]), x[..., o + R:]], -1)
    if case["quant"] == BF16:
        return {"out": x.to(torch.bfloat16)}
    return _as_values(*_quantise(x, case["quant"]), case["quant"])


def _attend(st):
    case, q, (L, N) = st["case"], st["q"].float(), st["most"]
    (T, H), cu, k = q.shape[:2], st["cu"].long(), st["k_lens"].long()
    req = torch.searchsorted(cu[1:], torch.arange(T, device=DEV), right=True)
    step = torch.arange(T, device=DEV) - cu[req]
    prefix = (k - (cu[1:] - cu[:-1]))[req]
    # with a window, only the positions that one can hold
    window = case["window"]
    N = min(N, window + L) if window else N
    low = (cu[:-1] - cu[1:] + k - window).clamp(min=0) if window else torch.zeros_like(k)
    every = torch.minimum(low[:, None] + torch.arange(N, device=DEV), k[:, None])           # [B, N]; k: none
    pos = every[req]
    node = pos - prefix[:, None]                                            # [T, N]
    at = node.clamp(0, 64 * st["mask"].shape[1] - 1)
    bit = (st["mask"].gather(1, at // 64) >> (at % 64)) & 1
    ok = (node < 0) | ((bit == 1) & (pos < k[req][:, None]))
    if window:
        later = ok.sum(1, keepdim=True) - ok.cumsum(1)                      # seen positions behind this one
        ok = ok & (later < window)
    codes, scales, _, _ = _parts(st)
    codes = codes.view(torch.int8 if st["quant"] == INT8 else torch.float8_e4m3fn)
    every = torch.minimum(every, k[:, None] - 1)
    page = st["bt"].long().gather(1, every // ROWS)
    rows = codes[page, every % ROWS].float() * scales[page, every % ROWS].float()[..., None]    # [B, N, D]
    tok = (cu[:-1, None] + torch.arange(L, device=DEV)).clamp(max=T - 1)    # [B, L]
    s = torch.matmul(q[tok].flatten(1, 2), rows.transpose(1, 2)) * SCALE    # [B, L * H, N]
    s = s.view(-1, L, H, N).masked_fill_(~ok[tok][:, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(1, 2), rows).view(-1, L, H, D) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total))[..., 0]
    return {"out": out[req, step].to(torch.bfloat16), "lse": lse[req, step]}


# ---- the definition in 64 bits ------------------------------------------------

def _exact_turn(x, case, st, offset, sign):
    """x [n, .., d] FP64: pair i of token t turns by position * frequency, as complex numbers."""
    R, f = case["rot"], 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEV) / case["rot"])
    if case["factor"] != 1.0:
        turns = TRAINED * f / (2 * math.pi)
        blend = ((turns - RAMP[0]) / (RAMP[1] - RAMP[0])).clamp(0, 1)
        f = blend * f + (1 - blend) * f / case["factor"]
    angle = sign * torch.outer(st["positions"].double(), f)
    unit = st["magnitude"] * torch.polar(torch.ones_like(angle), angle)
    while unit.dim() < x.dim():
        unit = unit[:, None]
    first = offset + (torch.arange(R // 2, device=DEV) if case["half"] else torch.arange(0, R, 2, device=DEV))
    second = first + (R // 2 if case["half"] else 1)
    z = torch.complex(x[..., first], x[..., second]) * unit
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_norm(x, norm, weight, bias):
    if norm == "none":
        return x
    if norm == "rms":
        return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
    var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
    return (x - mean) / (var + EPS).sqrt() * weight.double() + bias.double()


def _exact_codes(y, quant):
    top = 127.0 if quant == INT8 else 448.0
    scale = (y.abs().amax(-1) / top).clamp(max=65504.0).to(torch.float16).double()
    c = torch.where(scale[..., None] > 0, y / scale.clamp(min=2.0 ** -24)[..., None], 0.0).clamp(-top, top)
    return (c.round() if quant == INT8 else c.to(torch.float8_e4m3fn).double()), scale


def exact(case, seed):
    if work(case)["flops"] > 3e12:
        return None
    st, op = prepare(case, seed), case["op"]
    if op == "rotate":
        return {"out": _exact_turn(st["x"].double(), case, st, case["offset"], -1.0 if case["inverse"] else 1.0)}
    if op == "queries":
        y = _exact_turn(_exact_norm(st["x"].double(), case["norm"], st["weight"], st["bias"]), case, st, case["offset"], 1.0)
        if case["quant"] == BF16:
            return {"out": y}
        codes, scales = _exact_codes(y, case["quant"])
        return {"codes": codes, "scales": scales}
    if op == "append":
        keep = st["slots"] >= 0
        slots, count = st["slots"][keep], st["cache"].shape[0] * ROWS

        def pool(v):
            full = torch.zeros(count, *v.shape[1:], dtype=torch.float64, device=DEV)
            full[slots] = v[keep]
            return full.view(-1, ROWS, *v.shape[1:])

        kv = _exact_turn(_exact_norm(st["rows"].double(), "rms", st["kv_weight"], None), case, st, D - case["rot"], 1.0)
        index = _exact_turn(_exact_norm(st["index"].double(), "layer", st["weight"], st["bias"]), case, st, 0, 1.0)
        each = [{"rows": pool(kv)}] if case["kv"] == BF16 else []
        for y, quant in ([] if case["kv"] == BF16 else [(kv, case["kv"])]) + [(index, case["index"])]:
            codes, scales = _exact_codes(y, quant)
            each.append({"codes": pool(codes), "scales": pool(scales)})
        return {"kv": each[0], "index": each[1]}
    k, n = _lengths(case)
    codes, scales, _, _ = _parts(st)
    kind = torch.int8 if case["quant"] == INT8 else torch.float8_e4m3fn
    mask, bt, outs, lses, t = st["mask"].cpu().numpy().view(np.uint64), st["bt"].long(), [], [], 0
    for b in range(case["B"]):
        every, prefix = torch.arange(int(k[b]), device=DEV), int(k[b] - n[b])
        page, row = bt[b, every // ROWS], every % ROWS
        rows = codes[page, row].view(kind).double() * scales[page, row].double()[:, None]
        for i in range(int(n[b])):
            nodes = [prefix + j for j in range(int(n[b])) if int(mask[t, j // 64]) >> (j % 64) & 1]
            seen = torch.zeros(int(k[b]), dtype=torch.bool, device=DEV)
            seen[:prefix] = True
            seen[nodes] = True
            if case["window"]:
                at = seen.nonzero()[:, 0]
                seen[at[:max(0, len(at) - case["window"])]] = False
            kv = rows[seen]
            z = st["q"][t].double() @ kv.T * SCALE
            lse = torch.logsumexp(z, -1)
            outs.append(torch.exp(z - lse[:, None]) @ kv)
            lses.append(lse)
            t += 1
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
