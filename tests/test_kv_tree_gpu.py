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


def test_a_chain_is_the_causal_attention():
    """Bit for bit: the units hold the same positions."""
    import torch
    case = TreeCase(54, [900, 64, 131], [7, 64, 3], 40, kv8.INT8, "chain")
    kw = case.upload()
    tree = qli.kv_tree_attention(scale=SCALE, **kw)
    kw.pop("tree_mask")
    causal = qli.kv_attention(scale=SCALE, ratio=1, **kw)
    assert all(torch.equal(a, b) for a, b in zip(tree, causal))


def test_requests_shorter_than_their_tree_are_flagged():
    import torch
    case = TreeCase(55, [300, 50], [4, 6], 64, kv8.FP8, "tree")
    case.k_lens = case.k_lens.copy()
    case.k_lens[1] = 5
    out, lse = run(case, err_want=2)
    assert not out[4:].any() and np.isneginf(lse[4:]).all()
    case.positions_of_second = None
    good = TreeCase(55, [300, 50], [4, 6], 64, kv8.FP8, "tree")
    want, _ = run(good)
    assert np.array_equal(out[:4], want[:4])
    del torch


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
