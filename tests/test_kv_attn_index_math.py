"""The index arithmetic of the attention over 8-bit KV rows, restated in Python
and checked against plain definitions (the GPU tests check the kernel itself):

- work shares: the units of a launch (token, row tile, 64 positions) split over
  CTAs are each taken once, and every row tile is either whole in one CTA or cut
  into pieces whose record names exactly the CTAs and slots that hold them;
- the tile: a lane's 16 codes go to two 16-byte units, eight lanes of a store
  cover all banks, every value lands once, and the row order of the output
  accumulators maps back to the values;
- the softmax's lanes: the positions and heads they own, their weights' place in
  the swizzled operand, and the head a cross-lane reduction leaves in each lane.
"""
import random

KPOS, HT = 64, 64


def share_begin(total, ctas, c):
    each = total // ctas
    return each * c + min(c, total - each * ctas)


def walk(units, hg, total, ctas, c):
    """(token, row tile, unit, units of the tile, first here, last here) of CTA c."""
    u0, u1 = share_begin(total, ctas, c), share_begin(total, ctas, c + 1)
    at, out = 0, []
    for t, n in enumerate(units):
        for g in range(hg):
            for i in range(n):
                if u0 <= at < u1:
                    out.append((t, g, i, n))
                at += 1
    res = []
    for k, (t, g, i, n) in enumerate(out):
        res.append((t, g, i, n, k == 0 or i == 0, i == n - 1 or k + 1 == len(out), k))
    return res


def cut_record(units, hg, total, ctas, c):
    """The record CTA c leaves: (token, row tile, end) of the row tile that began
    in it and goes on in the next, or None."""
    u0, u1 = share_begin(total, ctas, c), share_begin(total, ctas, c + 1)
    if u1 <= u0:
        return None
    at = 0
    for t, n in enumerate(units):
        if at <= u1 - 1 < at + n * hg:
            g = (u1 - 1 - at) // n
            first = at + g * n
            return (t, g, first + n) if first + n > u1 and first >= u0 else None
        at += n * hg
    raise AssertionError


def test_shares_cover_every_unit_once_and_cut_tiles_are_joined():
    rng = random.Random(0)
    for trial in range(300):
        hg = rng.choice([1, 2])
        units = [rng.choice([1, 1, 2, 5, 32, 400]) for _ in range(rng.choice([1, 2, 7, 40]))]
        total, ctas = sum(units) * hg, rng.choice([1, 2, 3, 8, 152])
        seen, whole, pieces = [], set(), {}
        for c in range(ctas):
            for t, g, i, n, first, last, k in walk(units, hg, total, ctas, c):
                seen.append((t, g, i))
                if last:
                    began = k >= i
                    if i == n - 1 and began:
                        whole.add((t, g))
                    else:
                        pieces.setdefault((t, g), set()).add((c, 1 if began else 0))
        assert len(seen) == total and len(set(seen)) == total
        joined = {}
        for c in range(1, ctas):
            rec = cut_record(units, hg, total, ctas, c - 1)
            if rec is None:
                continue
            t, g, end = rec
            count = 2
            while c + count - 1 < ctas and share_begin(total, ctas, c + count - 1) < end:
                count += 1
            assert (t, g) not in joined
            joined[(t, g)] = {(c - 1, 1)} | {(c - 1 + k, 0) for k in range(1, count)}
        assert joined == pieces
        assert whole | set(pieces) == {(t, g) for t in range(len(units)) for g in range(hg)}
        assert not whole & set(pieces)


def sw(r, u):
    return r * 128 + ((u ^ (r & 7)) << 4)


def value_of(c, row):
    return 128 * c + 16 * ((row >> 3) & 7) + 8 * (row >> 6) + (row & 7)


def test_tile_layout():
    region = KPOS * 128
    place = {}
    for warp in range(8):
        for k in range(2):
            for c in range(4):
                for b in range(2):
                    addr = []
                    for lane in range(32):
                        r0, j = 8 * warp + (lane >> 3), lane & 7
                        at0 = sw(r0, j)
                        at = ((at0 ^ 64) + 512) if k else at0
                        row = r0 + 4 * k
                        assert at == sw(row, j)
                        at += c * 2 * region + b * region
                        addr.append(at)
                        for x in range(8):
                            # the lane's codes 16j + 8b + x of quarter c
                            key = (at + 2 * x)
                            assert key not in place
                            place[key] = (row, 128 * c + 16 * j + 8 * b + x)
                    for e in range(0, 32, 8):       # eight lanes of a 16-byte store: all 32 banks
                        assert len({(a % 128) // 16 for a in addr[e:e + 8]}) == 8
    assert len(place) == KPOS * 512
    # accumulator row 64b + 8j + x of quarter c reads region 2c + b, column 8j + x
    for c in range(4):
        for m in range(128):
            reg, col = 2 * c + (m >> 6), m & 63
            for row in (0, 5, 63):
                at = reg * region + sw(row, col >> 3) + 2 * (col & 7)
                assert place[at] == (row, value_of(c, m))
        assert sorted(value_of(c, m) for m in range(128)) == list(range(128 * c, 128 * c + 128))
    # four consecutive rows are four consecutive values (the joined output's stores)
    assert all(value_of(c, 4 * l + x) == value_of(c, 4 * l) + x for c in range(4) for l in range(32) for x in range(4))


def test_softmax_lanes():
    owned, weights = set(), {}
    for warp in range(8):
        qw, sub = warp & 3, warp >> 2
        banks = {}
        for lane in range(32):
            pos, h0 = 16 * qw + (lane >> 2), 32 * sub + 2 * (lane & 3)
            p_at = sw(pos, 4 * sub) + 4 * (lane & 3)
            for k in range(2):
                for i in range(4):
                    at = (p_at ^ (i << 4)) + k * 1024
                    banks.setdefault((k, i), []).append((at // 4) % 32)
                    for b in range(2):
                        p, h = pos + 8 * k, h0 + 8 * i + b
                        owned.add((p, h))
                        assert at + 2 * b == sw(p, h >> 3) + 2 * (h & 7)
                        weights[at + 2 * b] = (p, h)
        assert all(len(set(v)) == 32 for v in banks.values())
    assert len(owned) == KPOS * HT == len(weights)


def test_reduction_leaves_each_head_in_one_lane():
    # v[lane][j]: value of head 8 (j >> 1) + 2 (lane & 3) + (j & 1), tagged by its lane
    v = [[{(8 * (j >> 1) + 2 * (lane & 3) + (j & 1), lane)} for j in range(8)] for lane in range(32)]

    def step(v, o, half):
        out = []
        for lane in range(32):
            up = (lane & o) != 0
            row = []
            for i in range(half):
                keep = v[lane][i + half] if up else v[lane][i]
                other = v[lane ^ o]
                send = other[i + half] if up else other[i]      # what the partner sends to this lane
                row.append(keep | send)
            out.append(row)
        return out

    v = step(v, 16, 4)
    v = step(v, 8, 2)
    v = step(v, 4, 1)
    heads = []
    for lane in range(32):
        got = v[lane][0]
        head = 8 * (lane >> 3) + 2 * (lane & 3) + ((lane >> 2) & 1)
        assert {h for h, _ in got} == {head} and len(got) == 8
        heads.append(head)
    assert sorted(heads) == list(range(32))
