"""Drafted tokens that share row tiles: every case here is one in which the library forms
groups (each test reads that from the kernels it queues)."""
import pytest

import tree_launches as plan
from oracle import kv8
from oracle import rows as oracle
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli
from test_kv_tree_gpu import SCALE, TreeCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    qli.lib()


def sms():
    import torch
    return torch.cuda.get_device_properties(0).multi_processor_count


def attend(kw, window=0, err_want=0, out=None, lse=None):
    """(out, lse) of a call that has been seen to form groups."""
    import torch
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: qli.kv_tree_attention(scale=SCALE, window=window, err_word=err, out=out, lse=lse, **kw)  # noqa: E731
    kinds = {kind for kind, _ in plan.launches(call)}
    assert kinds - {"join"} == {"groups"}
    got = [t.clone() for t in call()]
    assert int(err.item()) == err_want
    return got


# ---- what is not finite stays with the tokens that see it --------------------------------

H, NODES = 16, 4
BRANCHES = [0b0001, 0b0011, 0b0100, 0b1100]              # nodes 0, 1 and nodes 2, 3


def few_trees(raw, quant, masks=BRANCHES):
    """One tree over a long context, whose row tile is cut: units of 64 positions, the nodes
    in the last one."""
    case = TreeCase(74, [raw], [NODES], H, quant)
    case.masks = list(masks)
    kw = case.upload()
    return case, plan.wide(kw, max(case.bt.shape[1], 64 * (sms() + 1) // case.R + 1))


def many_trees(quant, masks=BRANCHES):
    """As many trees under a window as have no SM a token: whole row tiles."""
    B = sms() // NODES + 2
    case = TreeCase(75, [300 + 13 * (b % 5) for b in range(B)], [NODES] * B, H, quant)
    case.masks = list(masks) * B
    return case, case.upload()


def row_bytes(case, kw, b, j):
    """(codes, scale) of position j of request b: views of the pool."""
    page, row = kw["cache"][int(case.bt[b, j // case.R])], j % case.R
    at, s = case.layout["kv_offset"] + 512 * row, case.layout["kv_scale_offset"] + 2 * row
    return page[at:at + 512], page[s:s + 2]


def poison(case, kw, b, j, what):
    import torch
    codes, scale = row_bytes(case, kw, b, j)
    if what == "codes":
        codes[3], codes[500] = 0x7F, 0xFF
    else:
        scale.copy_(torch.tensor([0x00, {"scale": 0x7E, "infinite-scale": 0x7C}[what]], dtype=torch.uint8))


WHAT = [(kv8.FP8, "codes"), (kv8.FP8, "scale"), (kv8.FP8, "infinite-scale"), (kv8.INT8, "scale"), (kv8.INT8, "infinite-scale")]


def check_poisoned(case, make, b, j, what, window=0):
    """Position j of request b made not finite: NaN (or Inf times 0) for the tokens that see
    it, the same bits for all others."""
    import torch
    want = attend(make, window)
    cache = make["cache"].clone()
    kw = dict(make, cache=cache)
    poison(case, kw, b, j, what)
    out, lse = attend(kw, window)
    for t in range(case.T):
        if case.request(t) == b and j in case.positions(t, window):
            assert not torch.isfinite(out[t]).any(), (j, t)
        else:
            assert torch.equal(out[t], want[0][t]) and torch.equal(lse[t], want[1][t]), (j, t)


# the last unit has 8, 34 or 48 positions: nodes in its first half, across both, in the second
@pytest.mark.parametrize("raw", [5000, 5026, 5040])
@pytest.mark.parametrize("quant,what", WHAT, ids=lambda v: str(v))
def test_rows_that_are_not_finite_in_cut_tiles(quant, what, raw):
    case, kw = few_trees(raw, quant)
    nodes = raw - NODES
    # a node of each branch; prefix rows in the last unit's halves, in other units
    for j in (nodes, nodes + 1, nodes + 2, nodes + 3, nodes - 1, raw // 64 * 64, raw // 64 * 64 + 2, 2500, 63, 0):
        check_poisoned(case, kw, 0, j, what)


@pytest.mark.parametrize("quant,what", WHAT, ids=lambda v: str(v))
@pytest.mark.parametrize("window", [64, 3])
def test_rows_that_are_not_finite_in_whole_tiles(window, quant, what):
    case, kw = many_trees(quant)
    assert len(plan.split_of(kw, window, sms())) == 1                  # nothing is joined
    for b in (0, 7, case.B - 1):
        nodes = int(case.k_lens[b]) - NODES
        for j in (nodes, nodes + 1, nodes + 3, nodes - 1, nodes - 2, nodes - window + 1, nodes - window + 2, nodes - window - 1):
            check_poisoned(case, kw, b, j, what, window)


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
@pytest.mark.parametrize("masks", [BRANCHES, [1, 0, 4, 8]], ids=["branches", "one-sees-none"])
@pytest.mark.parametrize("cut", [True, False], ids=["cut", "whole"])
def test_a_query_that_is_not_finite_stays_alone(cut, masks, quant):
    """In a row tile with other tokens' rows; also that of a token without a position."""
    import torch
    case, kw = few_trees(5026, quant, masks) if cut else many_trees(quant, masks)
    window = 0 if cut else 64
    if masks[1] == 0:                                                  # and no prefix
        kw["k_lens"] = torch.full_like(kw["k_lens"], NODES)
    want = attend(kw, window)
    for t in (1, case.T - 3):                                          # token 1 of the first and of the last tree
        q = kw["q"].clone()
        q[t, 3, 7], q[t, 4] = float("nan"), float("inf")
        out, lse = attend(dict(kw, q=q), window)
        others = torch.arange(case.T, device="cuda") != t
        assert torch.equal(out[others], want[0][others]) and torch.equal(lse[others], want[1][others])
        if masks[1] == 0:
            assert not out[t].any() and torch.isneginf(lse[t]).all()
        else:
            assert torch.isnan(out[t, 3:5]).all()
            heads = [h for h in range(H) if h not in (3, 4)]
            assert torch.equal(out[t, heads], want[0][t, heads]) and torch.equal(lse[t, heads], want[1][t, heads])


# ---- every way of sharing, with and without a window -------------------------------------

def compared(case, window=0, kw=None, err_want=0):
    from test_kv_attn_gpu import compare
    got = attend(case.upload() if kw is None else kw, window, err_want)
    compare(case, tuple(t.double().cpu().numpy() for t in got), window=window)


SHARED = [(1, 3), (2, 8), (5, 8), (8, 8), (16, 4), (16, 7), (20, 6), (32, 2), (32, 9), (40, 8), (48, 5), (96, 4), (100, 8),
          (16, 70), (96, 70), (24, 130)]


@pytest.mark.parametrize("window", [0, 1, 5, 40, 100, 200])
@pytest.mark.parametrize("H,n", SHARED, ids=lambda v: str(v))
def test_tokens_that_share_tiles(H, n, window):
    """As many requests as it takes; any masks (empty ones too) or trees."""
    words, B = -(-n // 64), 3
    while plan.stack_of(H, B * n, B, words, window, 768, sms()) == 1:
        B += 1
    raw = [[700, 66 + n, n, 300, 129 + n][b % 5] for b in range(B)]
    compared(TreeCase(76 + H + n, raw, [n] * B, H, [kv8.FP8, kv8.INT8][(H + n + window) % 2], "any" if H % 3 else "tree"),
             window)


# ---- boundaries that fall, tokens that no request covers ----------------------------------

class Disturbed(TreeCase):
    """Other boundaries than the tokens were made for; each token belongs to the last
    request that a search over the clamped boundaries finds to start at or before it."""

    def disturb(self, cu):
        self.given = cu
        return self

    def range_of(self, t):
        cu, lo, hi = [min(max(c, 0), self.T) for c in self.given], 0, self.B - 1
        while lo < hi:
            mid = (lo + hi + 1) // 2
            lo, hi = (mid, hi) if cu[mid] <= t else (lo, mid - 1)
        return lo, cu[lo], max(cu[lo], cu[lo + 1])

    def request(self, t):
        return self.range_of(t)[0]

    def positions(self, t, window=0):
        b, q0, q1 = self.range_of(t)
        if not q0 <= t < q1:
            return super().positions(t, window)[:0]
        n = q1 - q0
        return oracle.tree_positions(int(self.k_lens[b]), n, self.masks[t] & (1 << min(n, 64 * self.words)) - 1, window)

    def upload(self, dev="cuda"):
        import torch
        return dict(super().upload(dev), cu_seqlens_q=torch.tensor(self.given, dtype=torch.int32, device=dev))


def disturbed(H, swaps, seed=78):
    """Trees of 8 tokens, as many as it takes for groups under a window; boundary i of
    `swaps` by another value."""
    B = sms() // 8 + 1
    case = Disturbed(seed, [300 + 7 * (b % 9) for b in range(B)], [8] * B, H, kv8.FP8)
    cu = case.cu.tolist()
    for i, v in swaps.items():
        cu[i % (B + 1)] = v if v >= 0 else cu[-1] + v
    return case.disturb(cu)


@pytest.mark.parametrize("window", [64, 128])
@pytest.mark.parametrize("H", [16, 32])
@pytest.mark.parametrize("swaps", [{3: 40, 7: 16}, {1: 100}, {-2: 5, 4: 0}], ids=["two", "one", "last"])
def test_boundaries_that_fall_in_whole_tiles(swaps, H, window):
    """Each token stays alone then, which makes more row tiles than the launch has CTAs:
    they take several each, and every token gets the answer of its request."""
    import torch
    case = disturbed(H, swaps)
    kw = case.upload()
    (kind, ctas), = plan.split_of(kw, window, sms())                   # nothing is joined
    assert kind == "groups" and ctas < case.T
    out = torch.full((case.T, H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case.T, H), float("nan"), device="cuda")
    got = attend(kw, window, err_want=1, out=out, lse=lse)
    from test_kv_attn_gpu import compare
    compare(case, tuple(t.double().cpu().numpy() for t in got), window=window)


@pytest.mark.parametrize("window", [0, 64])
@pytest.mark.parametrize("H", [16, 32])
def test_tokens_that_no_request_covers_in_groups(H, window):
    """Before the first boundary and behind the last; a request without tokens among them."""
    case = disturbed(H, {0: 5, 2: 8, -1: -3})
    compared(case, window, err_want=1)
