"""GPU parity of the attention over 8-bit KV rows (qli_kv_attention) against the
float64 oracle (oracle/kv8.py), to bounds derived from the arithmetic
(kv8_cases.attention_bounds)."""
import numpy as np
import pytest

from kv8_cases import KVCase, attention_bounds
from oracle import kv8
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli, synth

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(512.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    qli.lib()


def run(case, scale=SCALE, window=0, err_want=0, **more):
    import torch
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = case.upload()
    kw.update(more)
    if window:
        kw["window"] = window
    out, lse = qli.kv_attention(scale=scale, err_word=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == err_want
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def compare(case, got, scale=SCALE, window=0, tokens=None, skip=()):
    o_g, l_g = got
    for t in range(case.T) if tokens is None else tokens:
        b = case.request(t)
        js = case.positions(t, window)
        js = js[~np.isin(js, list(skip))]
        q = kv8.bf16_to_f64(case.q[t])
        kv = case.kv(b, js)
        o, lse = kv8.attend(q, kv, scale)
        if js.size == 0:
            assert not o_g[t].any() and np.all(np.isneginf(l_g[t])), t
            continue
        do, dl = attention_bounds(q, kv, o, lse, scale)
        bad = ~(np.abs(o_g[t] - o) <= do)
        assert not bad.any(), (t, np.argwhere(bad)[:4], o_g[t][bad][:4], o[bad][:4])
        assert np.all(np.abs(l_g[t] - lse) <= dl), (t, l_g[t] - lse, dl)


CASES = [
    # name, raw lengths, query lengths, ratio, H, K (None: visible positions), window
    ("listed-h64-k512", [2048], [1], 2, 64, 512, 0),
    ("listed-h64-k2048", [9000, 5000], [1, 1], 1, 64, 2048, 0),
    ("listed-h1-k1", [500, 40], [1, 1], 1, 1, 1, 0),
    ("listed-h33-k129", [3000], [3], 2, 33, 129, 0),
    ("listed-h128-k300", [2600, 1111, 4000], [1, 2, 1], 1, 128, 300, 0),
    ("listed-h16-k127", [1000, 1000], [1, 1], 2, 16, 127, 0),
    ("listed-h32-k128", [1000, 130], [2, 1], 2, 32, 128, 0),
    ("dense-h64", [3001, 700, 1], [2, 1, 1], 2, 64, None, 0),
    ("dense-h32-pages", [128, 129, 127, 255], [1, 1, 1, 1], 1, 32, None, 0),
    ("dense-h100-chunk", [300, 77], [40, 77], 1, 100, None, 0),
    ("dense-h5-whole-prompt", [67, 5], [67, 5], 2, 5, None, 0),
    ("dense-long", [30011], [1], 1, 64, None, 0),
    ("window-1", [900, 30], [1, 2], 1, 64, None, 1),
    ("window-128", [4000, 100, 129], [3, 2, 1], 2, 48, None, 128),
    ("window-200-h96", [777], [5], 1, 96, None, 200),
]


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
@pytest.mark.parametrize("p", CASES, ids=[p[0] for p in CASES])
def test_attention_parity(p, quant):
    name, raw, ql, ratio, H, K, window = p
    case = KVCase(len(name) + 100 * quant, raw, ql, ratio, H, quant, K=K)
    compare(case, run(case, window=window), window=window)


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
@pytest.mark.parametrize("R,ratio", [(64, 1), (128, 2)])
def test_either_page_size_with_either_ratio(R, ratio, quant):
    case = KVCase(31, [1500, 333], [2, 1], ratio, 64, quant, rows_per_page=R)
    compare(case, run(case))


def _fuzz(n=24, seed=20261206):
    rng = np.random.default_rng(seed)
    out = []
    for i in range(n):
        B = int(rng.integers(1, 6))
        ratio = int(rng.integers(1, 3))
        H = int(rng.integers(1, 129))
        raw = rng.integers(1, 5000, size=B)
        ql = np.minimum(rng.integers(1, 7, size=B), raw)
        K = int(rng.choice([1, 3, 64, 128, 129, 500, 1024])) if rng.random() < 0.5 else None
        window = int(rng.integers(1, 600)) if K is None and rng.random() < 0.4 else 0
        out.append((int(rng.integers(1 << 30)), raw.tolist(), ql.tolist(), ratio, H,
                    int(rng.choice([kv8.INT8, kv8.FP8])), K, window,
                    float(SCALE * rng.choice([0.0, 1.0, 1.0, 4.0, -1.0])),
                    float(rng.choice([0.0, 1.0, 4.0]))))
    return out


@pytest.mark.parametrize("p", _fuzz(), ids=lambda p: "h%d-k%s-w%d" % (p[4], p[6], p[7]))
def test_attention_seeded_sweep(p):
    seed, raw, ql, ratio, H, quant, K, window, scale, spread = p
    case = KVCase(seed, raw, ql, ratio, H, quant, K=K, row_size=spread)
    compare(case, run(case, scale, window), scale, window)


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
def test_holes_duplicates_and_empty_lists(quant):
    case = KVCase(41, [2000, 700, 300], [2, 1, 1], 2, 64, quant, K=384)
    rng = np.random.default_rng(3)
    row = case.indices[0, 0]
    row[:] = np.sort(rng.choice(1000, 384, replace=False))
    row[rng.choice(384, 100, replace=False)] = -1
    case.indices[1, 0, :20] = 17                                 # one position twenty times
    case.indices[2] = -1
    case.indices[3] = -1
    case.indices[3, 0, 383] = 5                                  # the last entry alone
    compare(case, run(case))


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
def test_requests_without_positions(quant):
    # raw length 1 at ratio 2 has no compressed position; the first queries of
    # a whole prompt see none either
    case = KVCase(42, [1, 600, 3, 0], [1, 1, 3, 0], 2, 64, quant)
    assert [case.positions(t).size for t in range(case.T)] == [0, 300, 0, 1, 1]
    compare(case, run(case))


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
def test_dominant_and_rising_scores(quant):
    """Weights concentrated on few rows, and scores that rise along the context
    so that the running maximum moves in every piece."""
    case = KVCase(43, [3000, 2000], [1, 1], 1, 64, quant, q_size=6.0)
    compare(case, run(case, scale=0.4), scale=0.4)
    q0 = kv8.bf16_to_f64(case.q[0, 0])
    for b in range(2):
        n = int(case.k_lens[b])
        grow = np.linspace(-2, 2, n)[:, None] * np.sign(q0)[None] + 0.01 * case.rng.standard_normal((n, 512))
        case.codes[b], case.scales[b] = kv8.quantise_rows(kv8.f32_to_bf16(grow), quant)
    case.q[:] = case.q[0, 0]
    compare(case, run(case))


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
def test_zero_rows_and_extreme_scales(quant):
    case = KVCase(44, [700], [1], 1, 64, quant)
    rng = np.random.default_rng(6)
    x = rng.standard_normal((700, 512))
    x[::5] = 0                                                   # zero rows: weight e^0, value 0
    x[1::5] *= 2.0 ** -20                                        # subnormal scales
    x[2::5] *= 2.0 ** 4
    case.codes[0], case.scales[0] = kv8.quantise_rows(kv8.f32_to_bf16(x), quant)
    compare(case, run(case))
    x[:] = 0                                                     # nothing but zero rows
    case.codes[0], case.scales[0] = kv8.quantise_rows(kv8.f32_to_bf16(x), quant)
    o, lse = run(case)
    assert not o.any() and np.allclose(lse, np.log(700), atol=1e-5)
    # codes under a zero scale stand for zeros
    case.codes[0][::2] = 5
    o, lse = run(case)
    assert not o.any() and np.allclose(lse, np.log(700), atol=1e-5)


def test_queries_far_from_one():
    """Query magnitudes whose products only fit FP32 with the power of two taken
    out, zero queries, and heads of very different size side by side."""
    case = KVCase(45, [900], [1], 1, 64, kv8.INT8)
    x = kv8.bf16_to_f64(case.q)
    size = 2.0 ** np.linspace(-100, 100, 64)
    x = x * size[None, :, None]
    x[0, 5] = 0
    x[0, 6, 1:] = 0
    case.q = kv8.f32_to_bf16(x)
    # one softmax scale for all: heads beyond 2^7 put everything on one row
    got = run(case, scale=SCALE)
    fine = [h for h in range(64) if abs(np.log2(size[h])) < 8 or h in (5, 6)] + list(range(0, 30))
    q = kv8.bf16_to_f64(case.q[0])[fine]
    kv = case.kv(0, case.positions(0))
    o, lse = kv8.attend(q, kv, SCALE)
    do, dl = attention_bounds(q, kv, o, lse, SCALE)
    assert np.all(np.abs(got[0][0][fine] - o) <= do) and np.all(np.abs(got[1][0][fine] - lse) <= dl)
    # the others: one row each
    for h in range(44, 64):
        z = kv @ kv8.bf16_to_f64(case.q[0, h])
        best = kv[int(z.argmax())]
        if np.sort(z)[-1] - np.sort(z)[-2] > 1e3 / SCALE:
            assert np.all(np.abs(got[0][0, h] - best) <= (2.0 ** -8 + 2.0 ** -11) * np.abs(best) + 1e-30)


def test_a_non_finite_query_stays_in_its_row():
    import torch
    case = KVCase(46, [500, 500], [1, 1], 1, 64, kv8.FP8)
    want = run(case)
    case.q[0, 3, 7] = 0x7F80                                     # +inf
    case.q[1, 60, 1] = 0x7FC0                                    # NaN
    got = run(case)
    keep = np.ones((2, 64), dtype=bool)
    keep[0, 3] = keep[1, 60] = False
    assert np.array_equal(got[0][keep], want[0][keep]) and np.array_equal(got[1][keep], want[1][keep])
    del torch


def test_strides_of_queries_and_outputs():
    import torch
    case = KVCase(47, [800, 90], [2, 1], 2, 24, kv8.INT8)
    want = run(case)
    kw = case.upload()
    wide = torch.full((24, 3, 584), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :, :512] = kw["q"].transpose(0, 1)
    out = torch.full((24, 3, 520), 7.0, dtype=torch.bfloat16, device="cuda")
    kw["q"] = wide[:, :, :512].transpose(0, 1)
    got, lse = qli.kv_attention(scale=SCALE, out=out[:, :, :512].transpose(0, 1), **kw)
    torch.cuda.synchronize()
    assert np.array_equal(got.float().cpu().numpy(), want[0].astype(np.float32))
    assert bool((out[:, :, 512:] == 7.0).all())


def test_block_table_wider_than_its_requests_and_strided():
    import torch
    case = KVCase(48, [800, 90], [1, 1], 1, 64, kv8.FP8)
    want = run(case)
    bt = torch.full((2, 40), 1 << 30, dtype=torch.int32, device="cuda")
    bt[:, 3:3 + case.bt.shape[1]] = torch.from_numpy(case.bt).cuda()
    got = run(case, block_table=bt[:, 3:3 + case.bt.shape[1]])
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_bad_positions_and_pages_are_skipped_and_flagged():
    case = KVCase(49, [1000], [1], 2, 64, kv8.INT8, K=64)
    case.indices[0, 0] = np.arange(64)
    cap = case.bt.shape[1] * case.R
    case.indices[0, 0, 5] = cap + 3                              # past the table
    case.indices[0, 0, 6] = 2 ** 31 - 1
    got = run(case, err_want=8)
    case.indices[0, 0, 5:7] = -1
    compare(case, got)
    # pages outside the pool: dense, the second and third of eight
    case = KVCase(50, [1000], [1], 2, 64, kv8.INT8)
    pages = case.bt.copy()
    bad = pages.copy()
    bad[0, 1], bad[0, 2] = -1, case.pages
    import torch
    got = run(case, err_want=8, block_table=torch.from_numpy(bad).cuda())
    compare(case, got, skip=range(64, 192))


def test_bad_metadata_is_clamped_and_flagged():
    import torch
    case = KVCase(51, [400, 300], [1, 1], 2, 64, kv8.FP8)
    cap = case.bt.shape[1] * case.R
    # request 1's pages past its own are -5: those positions are skipped
    k = torch.tensor([200, cap + 1], dtype=torch.int32, device="cuda")
    o, lse = run(case, err_want=2 | (8 if case.bt[1, -1] < 0 else 0), k_lens=k)
    compare(case, (o, lse), tokens=[0])
    k = torch.tensor([200, -4], dtype=torch.int32, device="cuda")
    o, lse = run(case, err_want=2, k_lens=k)
    compare(case, (o, lse), tokens=[0])
    assert not o[1].any() and np.all(np.isneginf(lse[1]))
    r = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    run(case, err_want=4, residual=r)
    cu = torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")   # nobody owns token 1
    o, lse = run(case, err_want=1, cu_seqlens_q=cu)
    compare(case, (o, lse), tokens=[0])
    assert not o[1].any() and np.all(np.isneginf(lse[1]))


def test_no_tokens():
    import torch
    case = KVCase(52, [400], [1], 2, 64, kv8.INT8)
    kw = case.upload()
    kw["q"] = kw["q"][:0]
    out, lse = qli.kv_attention(scale=SCALE, **kw)
    assert out.shape == (0, 64, 512) and lse.shape == (0, 64)
    del torch


def test_many_tokens():
    """More query tokens than are planned at once, most of them short."""
    raw = [40] * 50 + [3] * 30 + [5000]
    ql = [40] * 50 + [3] * 30 + [6]
    case = KVCase(53, raw, ql, 1, 3, kv8.FP8)
    assert case.T > 2048
    got = run(case)
    compare(case, got, tokens=list(range(0, case.T, 37)) + list(range(case.T - 8, case.T)))
    assert np.isfinite(got[1]).all()


def test_same_call_gives_the_same_bits_and_leaves_the_workspace_to_others():
    import torch
    case = KVCase(54, [20000, 300], [1, 2], 1, 64, kv8.FP8)
    other = KVCase(55, [700, 900], [1, 1], 1, 64, kv8.INT8, K=300)
    a, b = case.upload(), other.upload()
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda").random_(0, 255)
    first = [t.clone() for t in qli.kv_attention(scale=SCALE, workspace=ws, **a)]
    for _ in range(5):
        qli.kv_attention(scale=SCALE, workspace=ws, **b)
        again = qli.kv_attention(scale=SCALE, workspace=ws, **a)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_on_another_stream_and_in_a_graph():
    import torch
    case = KVCase(56, [5000, 300], [1, 2], 2, 64, kv8.INT8)
    kw = case.upload()
    want = [t.clone() for t in qli.kv_attention(scale=SCALE, **kw)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = qli.kv_attention(scale=SCALE, stream=s, **kw)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qli.kv_attention(scale=SCALE, out=out, lse=lse, workspace=ws, **kw)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_pages_beyond_four_gigabytes():
    import torch
    case = KVCase(57, [900, 100], [1, 1], 1, 64, kv8.FP8)
    want = run(case)
    L = synth.kv8_layout(128)
    shift = (1 << 32) // L["page_stride"] + 5
    small = torch.from_numpy(case.pool()).cuda()
    cache = torch.empty((shift + case.pages, L["page_stride"]), dtype=torch.uint8, device="cuda")
    cache[:shift].fill_(0x7F)
    cache[shift:] = small
    got = run(case, cache=cache, block_table=torch.from_numpy(case.bt + shift).cuda())
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_workspace_too_small_is_refused():
    import torch
    case = KVCase(58, [900], [1], 1, 64, kv8.FP8)
    kw = case.upload()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    n = qli.kv_attention_workspace_bytes(1, 64)
    if n <= 256:
        pytest.skip("this call needs no workspace")
    with pytest.raises(qli.QLIError) as e:
        qli.kv_attention(scale=SCALE, workspace=ws, **kw)
    assert e.value.status == 5


def test_two_stages_merged_are_one_attention():
    """The window and the positions before it, merged, against both at once."""
    import torch
    case = KVCase(59, [3000, 2500], [1, 1], 2, 64, kv8.INT8)
    kw = case.upload()
    both = run(case)
    w = qli.kv_attention(scale=SCALE, window=100, **kw)
    V = [case.positions(t).size for t in range(2)]
    idx = torch.full((2, 1, 1500), -1, dtype=torch.int32, device="cuda")
    for t in range(2):
        idx[t, 0, :V[t] - 100] = torch.arange(V[t] - 100, dtype=torch.int32)
    for name in ("k_lens", "residual", "ratio"):
        kw.pop(name)
    rest = qli.kv_attention(scale=SCALE, indices=idx, **kw)
    out, lse = qli.merge_attention([w[0], rest[0]], [w[1], rest[1]])
    o, l = out.float().cpu().numpy(), lse.cpu().numpy()
    for t in range(2):
        q, kv = kv8.bf16_to_f64(case.q[t]), case.kv(t, case.positions(t))
        want, want_lse = kv8.attend(q, kv, SCALE)
        do, dl = attention_bounds(q, kv, want, want_lse, SCALE)
        # two stages rounded to BF16 before the merge rounds again
        top = np.abs(kv).max()
        assert np.all(np.abs(o[t] - want) <= 2 * do + 2.0 ** -8 * top)
        assert np.all(np.abs(l[t] - want_lse) <= 2 * dl + 2.0 ** -20)
    assert both[0].shape == o.shape
