"""GPU parity of the attention of drafted trees (qli_kv_tree_attention) against the
float64 oracle, to the bounds of kv8_cases.attention_bounds."""
import numpy as np
import pytest

from kv8_cases import KVCase
from oracle import kv8
from oracle import rows as oracle
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(512.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    qli.lib()


class TreeCase(KVCase):
    """Requests of `raw` positions whose last `nodes` are drafted. masks: "tree" (self
    and ancestors of a random tree), "chain", "any" (any bits, also past the nodes and
    empty rows)."""

    def __init__(self, seed, raw, nodes, H, quant, masks="tree", words=None, **kw):
        super().__init__(seed, raw, nodes, 1, H, quant, **kw)
        most = int(max(nodes)) if len(nodes) else 0
        self.words = words or max(1, -(-most // 64))
        self.masks = []
        for b in range(self.B):
            n = int(self.q_lens[b])
            m = []
            for i in range(n):
                if masks == "any":
                    bits = int.from_bytes(self.rng.bytes(8 * self.words), "little")
                    m.append(0 if self.rng.random() < 0.2 else bits)
                else:
                    parent = i - 1 if masks == "chain" else int(self.rng.integers(max(-1, i - 7), i)) if i else -1
                    m.append((m[parent] if parent >= 0 else 0) | 1 << i)
            self.masks += m

    def positions(self, t, window=0):
        b = self.request(t)
        mask = self.masks[t] & ((1 << 64 * self.words) - 1)
        return oracle.tree_positions(int(self.k_lens[b]), int(self.q_lens[b]), mask, window)

    def upload(self, dev="cuda"):
        import torch
        kw = super().upload(dev)
        kw.pop("ratio"), kw.pop("residual")
        words = np.array([[m >> 64 * w & (1 << 64) - 1 for w in range(self.words)] for m in self.masks], dtype=np.uint64)
        kw["tree_mask"] = torch.from_numpy(words.reshape(-1, self.words).view(np.int64)).to(dev)
        return kw


def run(case, window=0, err_want=0, **more):
    import torch
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = qli.kv_tree_attention(scale=SCALE, err_word=err, window=window, **dict(case.upload(), **more))
    torch.cuda.synchronize()
    assert int(err.item()) == err_want
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def check(case, window=0, **kw):
    from test_kv_attn_gpu import compare
    compare(case, run(case, window, **kw), window=window)


CASES = [
    # name, positions, nodes, H, masks, window
    ("one-token", [300], [1], 64, "tree", 0),
    ("one-position", [1], [1], 64, "tree", 0),
    ("whole-prompt-drafted", [7, 64], [7, 64], 33, "tree", 0),
    ("small-trees", [2000, 129, 64], [8, 5, 3], 64, "tree", 0),
    ("few-heads", [1500, 700], [13, 16], 8, "tree", 0),
    ("many-heads", [900, 1111], [6, 3], 128, "tree", 0),
    ("h96", [777], [20], 96, "tree", 0),
    ("two-words", [400, 200], [65, 130], 16, "tree", 0),
    ("any-masks", [70, 333], [70, 50], 32, "any", 0),
    ("any-masks-empty-prefix", [40, 5], [40, 5], 64, "any", 0),
    ("long", [20001], [4], 64, "tree", 0),
    ("window-1", [300, 9], [9, 9], 64, "tree", 1),
    ("window-cuts-nodes", [300, 40], [40, 40], 20, "chain", 7),
    ("window-128", [3000, 128, 140], [8, 8, 8], 16, "tree", 128),
    ("window-any", [500, 90], [90, 90], 48, "any", 33),
    ("window-wide", [5000, 64], [5, 2], 64, "tree", 3000),
    ("two-words-any", [400, 130], [65, 130], 16, "any", 0),
    ("two-words-window", [400, 200], [65, 130], 16, "any", 50),
    ("five-words", [300, 1000], [300, 280], 24, "any", 0),
    ("five-words-window", [310], [300], 64, "tree", 9),
    ("one-head", [500, 90], [20, 90], 1, "any", 0),
    ("two-heads", [500, 30], [9, 30], 2, "tree", 0),
    ("three-heads-window", [700, 50], [30, 17], 3, "any", 25),
]


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
@pytest.mark.parametrize("p", CASES, ids=[p[0] for p in CASES])
def test_tree_parity(p, quant):
    name, raw, nodes, H, masks, window = p
    check(TreeCase(len(name) + 100 * quant, raw, nodes, H, quant, masks), window)


def _fuzz(n=20, seed=20261208):
    rng = np.random.default_rng(seed)
    out = []
    for i in range(n):
        B = int(rng.integers(1, 6))
        raw = rng.integers(1, 3000, size=B)
        nodes = np.minimum(rng.integers(0, 40, size=B), raw)
        nodes[0] = max(1, nodes[0])
        out.append((int(rng.integers(1 << 30)), raw.tolist(), nodes.tolist(), int(rng.integers(1, 129)),
                    int(rng.choice([kv8.INT8, kv8.FP8])), str(rng.choice(["tree", "any"])),
                    int(rng.integers(1, 300)) if rng.random() < 0.4 else 0, int(rng.choice([64, 128]))))
    return out


@pytest.mark.parametrize("p", _fuzz(), ids=lambda p: "h%d-%s-w%d" % (p[3], p[5], p[6]))
def test_tree_seeded_sweep(p):
    seed, raw, nodes, H, quant, masks, window, R = p
    check(TreeCase(seed, raw, nodes, H, quant, masks, rows_per_page=R), window)


def test_more_tokens_than_one_plan_holds():
    check(TreeCase(51, [200] * 40, [16] * 40, 16, kv8.INT8, "tree"))        # 640 tokens


def test_nodes_past_the_mask_are_not_seen():
    case = TreeCase(52, [300], [80], 32, kv8.FP8, "tree", words=1)
    assert all(m >> 64 for m in case.masks[64:])
    check(case)


def test_more_words_than_nodes():
    check(TreeCase(53, [300, 20], [5, 3], 32, kv8.FP8, "any", words=3))


@pytest.mark.parametrize("H", [64, 128])
def test_a_chain_is_the_causal_attention(H):
    """Bit for bit where tokens do not share row tiles: the units hold the same positions."""
    import torch
    case = TreeCase(54, [900, 64, 131], [7, 64, 3], H, kv8.INT8, "chain")
    kw = case.upload()
    tree = qli.kv_tree_attention(scale=SCALE, **kw)
    kw.pop("tree_mask")
    causal = qli.kv_attention(scale=SCALE, ratio=1, **kw)
    assert all(torch.equal(a, b) for a, b in zip(tree, causal))


def test_requests_shorter_than_their_tree_are_flagged():
    case = TreeCase(55, [300, 50], [4, 6], 64, kv8.FP8, "tree")
    case.k_lens = case.k_lens.copy()
    case.k_lens[1] = 5
    out, lse = run(case, err_want=2)
    assert not out[4:].any() and np.isneginf(lse[4:]).all()
    good = TreeCase(55, [300, 50], [4, 6], 64, kv8.FP8, "tree")
    want, _ = run(good)
    assert np.array_equal(out[:4], want[:4])


def test_pages_outside_the_pool_are_skipped_and_flagged():
    case = TreeCase(56, [400, 300], [5, 4], 32, kv8.INT8, "tree")
    bt = case.bt.copy()
    kept = case.upload()
    import torch
    bt[0, 1] = case.pages
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept["block_table"] = torch.from_numpy(bt).cuda()
    got = qli.kv_tree_attention(scale=SCALE, err_word=err, **kept)
    assert int(err.item()) == 8
    from test_kv_attn_gpu import compare
    got = tuple(t.float().cpu().numpy().astype(np.float64) for t in got)
    compare(case, got, tokens=range(5), skip=range(case.R, 2 * case.R))
    compare(case, got, tokens=range(5, 9))


def test_the_same_call_gives_the_same_bits():
    import torch
    case = TreeCase(57, [5000, 3000], [16, 9], 64, kv8.FP8, "tree")
    kw = case.upload()
    one = [t.clone() for t in qli.kv_tree_attention(scale=SCALE, **kw)]
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(one, qli.kv_tree_attention(scale=SCALE, **kw)))


@pytest.mark.parametrize("H,window", [(64, 0), (16, 0), (64, 100), (16, 100)])
def test_several_launches_give_the_same_bits(H, window):
    """More tokens than three launches hold, over short and uneven contexts; some of the
    last launch's row tiles are whole."""
    import torch
    raw = [30 + 61 * (i % 7) for i in range(55)]
    case = TreeCase(84, raw, [30] * 55, H, kv8.FP8, "tree", row_size=0.5)
    kw = case.upload()
    one = [t.clone() for t in qli.kv_tree_attention(scale=SCALE, window=window, **kw)]
    for _ in range(12):
        got = qli.kv_tree_attention(scale=SCALE, window=window, **kw)
        assert all(torch.equal(a, b) for a, b in zip(one, got))
    from test_kv_attn_gpu import compare
    got = tuple(t.float().cpu().numpy().astype(np.float64) for t in one)
    compare(case, got, window=window, tokens=[0, 511, 512, 513, 700, 1023, 1024, 1100, 1535, 1536, case.T - 1])


def test_on_another_stream_and_in_a_graph():
    import torch
    case = TreeCase(58, [2500, 400], [12, 3], 64, kv8.FP8, "tree")
    kw = case.upload()
    want = [t.clone() for t in qli.kv_tree_attention(scale=SCALE, **kw)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = qli.kv_tree_attention(scale=SCALE, stream=s, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.empty(qli.kv_attention_workspace_bytes(case.T, case.H), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = qli.kv_tree_attention(scale=SCALE, workspace=ws, **kw)
    # another tree of the same size, in the tensors that were captured
    other = TreeCase(58, [2500, 400], [12, 3], 64, kv8.FP8, "any")
    kw["tree_mask"].copy_(other.upload()["tree_mask"])
    g.replay()
    replayed = [t.clone() for t in out]
    assert all(torch.equal(a, b) for a, b in zip(replayed, qli.kv_tree_attention(scale=SCALE, **kw)))
    assert not torch.equal(replayed[0], want[0])


def test_queries_of_other_strides():
    import torch
    case = TreeCase(59, [600], [9], 24, kv8.INT8, "tree")
    kw = case.upload()
    want = qli.kv_tree_attention(scale=SCALE, **kw)
    kw["q"] = kw["q"].transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.zeros(24, 9, 512, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    got = qli.kv_tree_attention(scale=SCALE, out=out, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- tokens that share row tiles ----------------------------------------------------

def stack_of(H, T, B):
    """Tokens that share row tiles, as the library chooses them."""
    best = 1
    for k in range(2, min(8, (T - 1) // B + 1) + 1):
        if -(-k * H // 64) * best < -(-best * H // 64) * k:
            best = k
    return best


SHARED = [(1, 3), (5, 8), (8, 8), (16, 4), (16, 7), (20, 6), (32, 2), (32, 9), (40, 8), (48, 5), (96, 4), (100, 8)]


@pytest.mark.parametrize("window", [0, 5, 40])
@pytest.mark.parametrize("H,n", SHARED, ids=lambda v: str(v))
def test_tokens_that_share_tiles(H, n, window):
    assert stack_of(H, 3 * n, 3) > 1 or H == 100 or n < 3
    check(TreeCase(71 + H + n, [700, 66, n], [n, n, n], H, kv8.FP8, "any" if H % 3 else "tree"), window)


@pytest.mark.parametrize("H", [8, 16, 48])
def test_trees_of_uneven_sizes_share_tiles(H):
    check(TreeCase(72, [900, 70, 64, 130, 3], [9, 1, 0, 17, 3], H, kv8.INT8, "tree"))


def test_groups_across_launches():
    """384 tokens are planned at a time; the trees do not end there."""
    check(TreeCase(73, [150] * 17, [50] * 17, 16, kv8.FP8, "tree"))


def _shared_case():
    """Two branches of one tree in one row tile: nodes 0, 1 and nodes 2, 3."""
    case = TreeCase(74, [100], [4], 16, kv8.FP8, "tree")
    case.masks = [0b0001, 0b0011, 0b0100, 0b1100]
    return case


def test_nan_in_rows_that_all_see():
    """A prefix row that is not finite reaches every token, whichever half of the unit it
    is in (node positions are in the other one)."""
    for j in (3, 40, 70, 96):                                    # units of 64: nodes are 96 .. 99
        case = _shared_case()
        kw = case.upload()
        want = qli.kv_tree_attention(scale=SCALE, **kw)
        page, row = int(case.bt[0, j // case.R]), j % case.R
        kw["cache"][page, case.layout["kv_offset"] + 512 * row + 9] = 0x7F
        out, lse = qli.kv_tree_attention(scale=SCALE, **kw)
        import torch
        for t in range(4):
            if j < 96 or t < 2:                                  # node 0 is in the path of tokens 0 and 1
                assert not torch.isfinite(out[t]).any(), (j, t)
            else:
                assert torch.equal(out[t], want[0][t]), (j, t)


@pytest.mark.parametrize("what", ["codes", "scale", "infinite-scale"])
def test_nan_in_rows_of_another_branch(what):
    """A drafted token whose row is not finite (the last one of a branch) makes the
    tokens that see it NaN, not their neighbours in the row tile."""
    import torch
    case = _shared_case()
    kw = case.upload()
    want = [t.clone() for t in qli.kv_tree_attention(scale=SCALE, **kw)]
    j = 97                                                       # node 1
    page, row = int(case.bt[0, j // case.R]), j % case.R
    if what == "codes":
        at = case.layout["kv_offset"] + 512 * row
        kw["cache"][page, at + 3] = 0x7F
        kw["cache"][page, at + 500] = 0xFF
    else:
        at = case.layout["kv_scale_offset"] + 2 * row
        bits = 0x7E00 if what == "scale" else 0x7C00
        kw["cache"][page, at:at + 2] = torch.tensor([bits & 255, bits >> 8], dtype=torch.uint8)
    out, lse = qli.kv_tree_attention(scale=SCALE, **kw)
    for t in (0, 2, 3):
        assert torch.equal(out[t], want[0][t]) and torch.equal(lse[t], want[1][t]), t
    assert not torch.isfinite(out[1]).any()


def test_a_query_that_is_not_finite_stays_alone():
    import torch
    for masks in ([0b0001, 0b0011, 0b0100, 0b1100], [1, 0, 4, 8]):
        case = _shared_case()
        case.masks = masks
        kw = case.upload()
        if masks[1] == 0:                                        # and without a position
            kw["k_lens"] = torch.tensor([4], dtype=torch.int32, device="cuda")
        want = [t.clone() for t in qli.kv_tree_attention(scale=SCALE, **kw)]
        kw["q"][1, 3, 7] = float("nan")
        kw["q"][1, 4] = float("inf")
        out, lse = qli.kv_tree_attention(scale=SCALE, **kw)
        for t in (0, 2, 3):
            assert torch.equal(out[t], want[0][t]) and torch.equal(lse[t], want[1][t]), t
        if masks[1] == 0:
            assert not out[1].any() and torch.isneginf(lse[1]).all()
        else:
            assert torch.isnan(out[1, 3]).all() and torch.isnan(out[1, 4]).all()
            assert torch.equal(out[1, 5:], want[0][1, 5:]) and torch.equal(out[1, :3], want[0][1, :3])


def test_rows_that_see_their_first_position_late():
    """Rows of one tile with far smaller scores than the others, whose first positions
    come after units of which they see nothing: each row has its own reference."""
    n = 150
    case = TreeCase(75, [n], [n], 16, kv8.INT8, "tree")
    case.masks = [(1 << t + 1) - 1 if t % 2 == 0 else 1 << t for t in range(n)]
    for t in range(1, n, 2):
        case.masks[t] = (1 << t) | (1 << n - 1) | (1 << n - 3)   # its own and the last nodes
    q = kv8.bf16_to_f64(case.q)
    q[1::2] *= 40.0                                              # references far from 0, on both sides
    case.q = kv8.f32_to_bf16(q)
    check(case)


@pytest.mark.parametrize("window", [0, 64])
def test_boundaries_that_fall_are_flagged(window):
    """No access leaves its buffer and every token gets an answer, in shared and in whole
    row tiles."""
    import torch
    case = TreeCase(76, [300] * 12, [8] * 12, 16, kv8.FP8, "tree")
    kw = case.upload()
    cu = [8 * b for b in range(13)]
    cu[3], cu[7] = 40, 16
    kw["cu_seqlens_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((96, 16, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((96, 16), float("nan"), device="cuda")
    qli.kv_tree_attention(scale=SCALE, err_word=err, window=window, out=out, lse=lse, **kw)
    assert int(err.item()) & 1
    assert torch.isfinite(out.float()).all() and not torch.isnan(lse).any()


@pytest.mark.parametrize("window", [0, 64])
@pytest.mark.parametrize("H", [16, 64])
def test_tokens_that_no_request_covers(H, window):
    """A padded batch: tokens before the first and behind the last request are flagged
    and see nothing; the others are as without them."""
    import torch
    case = TreeCase(77, [400, 90], [9, 6], H, kv8.FP8, "tree")
    kw = case.upload()
    want = qli.kv_tree_attention(scale=SCALE, window=window, **kw)
    for before, behind in ((0, 600), (3, 0), (11, 50)):
        T = 15 + before + behind
        q = torch.full((T, H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
        mask = torch.full((T, 1), -1, dtype=torch.int64, device="cuda")
        q[before:before + 15], mask[before:before + 15] = kw["q"], kw["tree_mask"]
        cu = torch.tensor([before, before + 9, before + 15], dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((T, H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, H), float("nan"), device="cuda")
        qli.kv_tree_attention(scale=SCALE, window=window, err_word=err, out=out, lse=lse,
                              **dict(kw, q=q, tree_mask=mask, cu_seqlens_q=cu))
        assert int(err.item()) == 1
        a, b = out[before:before + 15].float(), want[0].float()
        # other shares of the work round differently: BF16 steps of the output (2^-8 of it
        # each way), and FP16 weights (2^-11 of the largest value)
        assert torch.all((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -9 * b.abs().amax())
        assert torch.all((lse[before:before + 15] - want[1]).abs() <= 2.0 ** -10)
        rest = torch.cat([torch.arange(before), torch.arange(before + 15, T)])
        assert not out[rest].any() and torch.isneginf(lse[rest]).all()
