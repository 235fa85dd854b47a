"""The index arithmetic of the attention of drafted trees and of the row kernels,
restated in Python and checked against plain definitions (the GPU tests check the
kernels themselves): which tokens share row tiles, the positions of a group, the rows
that see them, the bounds the launches rest on, and the whole-number angles."""
import math
import random

import numpy as np
import pytest

from oracle import rows as oracle

HT, MAX_STACK = 64, 8


def stack_of(H, T, B):
    best = 1
    for k in range(2, min(MAX_STACK, (T - 1) // max(1, B) + 1) + 1):
        if -(-k * H // HT) * best < -(-best * H // HT) * k:
            best = k
    return best


def test_stacks_leave_no_more_rows_empty_than_single_tokens():
    for H in range(1, 129):
        for T, B in ((1, 1), (7, 1), (64, 8), (64, 64), (300, 2)):
            k = stack_of(H, T, B)
            assert 1 <= k <= MAX_STACK and -(-k * H // HT) <= k * -(-H // HT)
    assert [stack_of(H, 64, 4) for H in (8, 16, 32, 40, 48, 64, 96, 128)] == [8, 4, 2, 8, 4, 1, 2, 1]


def groups_of(cu, T, t0, tc, stack):
    """(first token, tokens) of the groups of a launch, as the plan makes them."""
    out = []
    for t in range(t0, t0 + tc):
        b = max([i for i in range(len(cu) - 1) if min(max(cu[i], 0), T) <= t], default=0)
        q0 = min(max(cu[b], 0), T)
        q1 = min(max(cu[b + 1], q0), T)
        begin, end = (0, q0) if t < q0 else (q0, q1) if t < q1 else (q1, T)
        if (t - max(begin, t0)) % stack == 0:
            out.append((t, min(stack, min(end, t0 + tc) - t)))
    return out


def test_groups_cover_every_token_once_and_stay_in_their_request():
    rng = random.Random(1)
    for trial in range(400):
        B, stack, chunk = rng.randint(1, 9), rng.randint(1, 8), rng.choice([16, 64, 512])
        cu = [rng.choice([0, 0, 5])]
        for _ in range(B):
            cu.append(cu[-1] + rng.choice([0, 1, 3, 8, 40]))
        T = max(1, cu[-1] + rng.choice([0, 0, 1, 30]))
        seen = []
        for t0 in range(0, T, chunk):
            tc = min(chunk, T - t0)
            groups = groups_of(cu, T, t0, tc, stack)
            assert len(groups) <= min(tc, tc // stack + B + 3)       # what a launch makes room for
            for t, n in groups:
                assert n >= 1 and t + n <= t0 + tc
                owner = [max([i for i in range(B) if cu[i] <= x < cu[i + 1]], default=-1) for x in range(t, t + n)]
                assert len(set(owner)) == 1
                seen += range(t, t + n)
        assert sorted(seen) == list(range(T))


def group_positions(P, nodes, masks, window):
    """(positions, rows that see each) of a group of tokens with these masks."""
    own = [bin(m & (1 << nodes) - 1).count("1") for m in masks]
    union = 0
    for m in masks:
        union |= m & (1 << nodes) - 1
    any_ = bin(union).count("1")
    V = any_ + (min(P, max(0, window - min(own))) if window else P)
    if len(masks) == 1 and window:
        V = min(V, window)
    bits = [i for i in range(nodes) if union >> i & 1]
    out = []
    for e in range(V):
        rank = any_ - V + e
        j = P + (rank if rank < 0 else bits[rank])
        see = []
        for k, m in enumerate(masks):
            if rank < 0:
                see.append(not window or -rank <= window - own[k])
            else:
                later = bin((m & (1 << nodes) - 1) >> bits[rank]).count("1")
                see.append(bool(m >> bits[rank] & 1) and (not window or own[k] <= window or later <= window))
        out.append((j, see if len(masks) > 1 else [True]))
    return out


def test_a_groups_positions_and_rows():
    rng = random.Random(2)
    for trial in range(600):
        P, nodes, count = rng.choice([0, 1, 30, 200]), rng.randint(1, 64), rng.randint(1, 8)
        masks = [rng.choice([0, rng.getrandbits(64), rng.getrandbits(64) & rng.getrandbits(64), 1 << rng.randrange(64)])
                 for _ in range(count)]
        window = rng.choice([0, 0, 1, 5, 64, 100])
        got = group_positions(P, nodes, masks, window)
        assert [j for j, _ in got] == sorted({j for j, _ in got})
        if window:                                               # the bound on a group's units
            assert len(got) <= window + (nodes if count > 1 else 0)
        for k, m in enumerate(masks):
            want = oracle.tree_positions(P + nodes, nodes, m & (1 << nodes) - 1, window)
            assert [j for j, see in got if see[k]] == want.tolist()


def bit_of(m, rank):
    at = 0
    for s in (32, 16, 8, 4, 2, 1):
        low = bin(m & (1 << s) - 1).count("1")
        if rank >= low:
            rank, m, at = rank - low, m >> s, at + s
    return at


def test_the_set_bit_of_a_rank():
    rng = random.Random(3)
    for trial in range(300):
        m = rng.getrandbits(64) & rng.choice([rng.getrandbits(64), (1 << 64) - 1]) | 1 << rng.randrange(64)
        assert [bit_of(m, r) for r in range(bin(m).count("1"))] == [i for i in range(64) if m >> i & 1]


def test_rows_of_a_tile_that_belong_to_a_token():
    for H in range(1, 129):
        per_head = (2 ** 32 - 1) // H + 1
        stack = stack_of(H, 64, 4)
        for v in range(stack * H):
            assert H == 1 or (v * per_head >> 32) == v // H
        for ht in (16, 32, 64):
            for g in range(-(-stack * H // ht)):
                rows = {}
                for k in range(stack):
                    lo, hi = max(0, k * H - g * ht), min(ht, (k + 1) * H - g * ht)
                    for r in range(lo, hi):
                        assert r not in rows
                        rows[r] = k
                assert rows == {r: (g * ht + r) // H for r in range(ht) if g * ht + r < stack * H}


def share_begin(total, ctas, c):
    each = total // ctas
    return each * c + min(c, total - each * ctas)


def test_the_share_that_has_a_unit():
    rng = random.Random(4)
    for trial in range(3000):
        ctas, total = rng.randint(1, 152), rng.choice([rng.randint(1, 400), rng.randint(1, 1 << 30)])
        u = rng.randrange(total)
        each = total // ctas
        more = total - each * ctas
        of_more = more * (each + 1)
        c = u // (each + 1) if u < of_more else more + (u - of_more) // each
        assert share_begin(total, ctas, c) <= u < share_begin(total, ctas, c + 1)


# ---- the row kernels --------------------------------------------------------------

def test_quotients_by_the_heads():
    rng = random.Random(5)
    for d in list(range(1, 300)) + [rng.randint(1, 1 << 30) for _ in range(200)]:
        s = 0
        while 1 << s < d:
            s += 1
        m = ((1 << 31 + s) + d - 1) // d
        assert m < 1 << 32 or d == 1
        for r in [0, 1, d - 1, d, 2 ** 30 - 1] + [rng.randrange(1 << 31) for _ in range(50)]:
            assert d == 1 or (r * m >> 32) >> s - 1 == r // d


def tokens_of(count, rows, H):
    n = min(rows, count)
    return min((n - 2 + H) // H + 1, n)


def test_tables_hold_the_tokens_of_their_blocks():
    rng = random.Random(6)
    for trial in range(2000):
        H, T, block = rng.choice([1, 2, 3, 7, 33, 64, 1000]), rng.randint(1, 60), rng.choice([4, 8, 32, 64, 85, 128])
        rows = T * H
        for r0 in range(0, rows, block):
            end = min(rows, r0 + block)
            assert (end - 1) // H - r0 // H + 1 <= tokens_of(block, rows, H)


@pytest.mark.parametrize("pairs", range(8, 72, 8))
def test_table_entries_by_token_and_pair(pairs):
    per_pair = (2 ** 32 - 1) // pairs + 1
    assert all((i * per_pair >> 32) == i // pairs for i in range(1 << 14))


def table_place(half, pair):
    log2, columns = (3, 8) if half else (2, 16)
    return 2 * (((pair & (1 << log2) - 1) >> 1) * columns + (pair >> log2)) + (pair & 1)


@pytest.mark.parametrize("half", [False, True])
def test_pairs_of_a_token_in_the_table(half):
    places = [table_place(half, p) for p in range(64)]
    assert sorted(places) == list(range(64))
    for u in range(8 if half else 16):                           # what a lane reads for unit u
        of_unit = [8 * u + i for i in range(8)] if half else [4 * u + i for i in range(4)]
        read = [2 * (k * (8 if half else 16) + u) + i for k in range(4 if half else 2) for i in range(2)]
        assert [places[p] for p in of_unit] == read


@pytest.mark.parametrize("pairs", range(8, 72, 8))
def test_tables_of_rotated_rows_fit(pairs):
    for H in (1, 2, 3, 64):
        for rows in (1, 5, 100, 10 ** 6):
            block = 128 // (pairs // 8)
            while 512 * tokens_of(block, rows, H) > 16 * 1024:
                block //= 2
            assert block >= 1
    for D in (64, 128, 256, 512):                                # one set of prepared rows
        assert 512 * tokens_of(128 // (D // 16), 10 ** 6, 1) <= 16 * 1024


def turn_of(frac, scale=1.0, inverse=False):
    """The kernel's cosine and sine of 2^-32 frac turns in FP32 (fused products by way of
    FP64, which holds them but for the double rounding)."""
    f = np.float32
    fma = lambda a, b, c: f(np.float64(a) * np.float64(b) + np.float64(c))  # noqa: E731
    hi_c = f(2 * math.pi / 2 ** 32)
    lo_c = f(2 * math.pi / 2 ** 32 - float(hi_c))
    s_hi = f(scale)
    s_lo = f(scale - float(s_hi))
    quarter = (frac + 0x20000000 & 0xFFFFFFFF) >> 30
    rest = (frac - (quarter << 30) + 2 ** 31) % 2 ** 32 - 2 ** 31
    hi = f(rest)
    lo = f(rest - int(hi))
    t = f(hi * hi_c)
    e = f(fma(hi, hi_c, -t) + fma(hi, lo_c, f(lo * hi_c)))
    t2 = f(t * t)
    t2e = fma(t, t, -t2)
    p = fma(t2, f(1 / 362880), f(-1 / 5040))
    p = fma(p, t2, f(1 / 120))
    p = fma(p, t2, f(-1 / 6))
    q = fma(t2, f(-1 / 3628800), f(1 / 40320))
    q = fma(q, t2, f(-1 / 720))
    q = fma(q, t2, f(1 / 24))
    sin_r = fma(f(t * t2), p, fma(f(f(-0.5) * t2), e, e))
    one = f(f(1) - f(f(0.5) * t2))
    cos_r = fma(f(t2 * t2), q, f(f(f(f(1) - one) - f(f(0.5) * t2)) - fma(t, e, f(f(0.5) * t2e))))
    sin_t = fma(s_hi, t, fma(s_hi, sin_r, f(s_lo * t)))
    cos_t = fma(s_hi, one, fma(s_hi, cos_r, f(s_lo * one)))
    a, b = (sin_t, cos_t) if quarter & 1 else (cos_t, sin_t)
    return (-a if quarter + 1 & 2 else a), (-b if (quarter >> 1 & 1) != inverse else b)


@pytest.mark.parametrize("scale", [1.0, 1.2772588722239782, 0.3])
@pytest.mark.parametrize("inverse", [False, True])
def test_cosine_and_sine_of_a_turn(scale, inverse):
    """Within the last rounding (half a step of what lies below the next power of two of
    the magnitude: 2^-25 of that), the sine series' rest of t^11 / 11! < 2^-29, and what
    the sums before the last one are off: numbers below 2^-3 in four roundings, 4 * 2^-28 / 2
    at most, and the part of the products that FP64 rounds."""
    rng = random.Random(7)
    bound = 2.0 ** (math.ceil(math.log2(scale)) - 25) + scale * (2.0 ** -29 + 2.0 ** -27)
    for frac in [0, 1, 2 ** 29 - 1, 2 ** 29, 2 ** 30, 2 ** 31, 3 << 30, 2 ** 32 - 1] + [rng.randrange(2 ** 32) for _ in range(3000)]:
        c, s = turn_of(frac, scale, inverse)
        angle = 2 * math.pi * frac / 2 ** 32 * (-1 if inverse else 1)
        assert abs(float(c) - scale * math.cos(angle)) < bound and abs(float(s) - scale * math.sin(angle)) < bound
