"""A model of the barriers of the attention over 8-bit KV rows, run over random
interleavings on the CPU.

Every warp of a CTA is a coroutine that stops at each wait; the tensor core is
two queues (scores, values) whose products start some time after their issue and
end some time after that. The model checks that

- a parity wait passes on exactly the phase it means, and an arrival counts
  towards the phase it is meant for;
- the products find all eight warps' tiles, queries and weights of their own
  unit, from their start to their end;
- nobody rewrites rows, tiles, queries, scores or weights that are still needed,
  and the output accumulators are touched (rescaled, read out) only between the
  products of the units before and those after.

With one barrier for the weights, not one by unit parity, the model finds the
fault that this had: four softmax warps a unit ahead complete the other four's
phase.
"""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "sparse_attention_indexer_qli_gb300", "csrc", "qli_kv_attn.cu")
LOADERS, SOFTMAX, ROWS = 8, 8, 2


def slots():
    return int(re.search(r"constexpr int kSlots = (\d+);", open(SRC).read()).group(1))


class Fault(AssertionError):
    pass


def need(ok, what):
    if not ok:
        raise Fault(what)


class Barrier:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.done = name, count, count, 0

    def arrive(self, phase):
        need(self.done == phase, "%s: an arrival for phase %d in phase %d" % (self.name, phase, self.done))
        self.pending -= 1
        if self.pending == 0:
            self.done, self.pending = self.done + 1, self.count

    def ready(self, phase):
        return (self.done & 1) != (phase & 1)

    def passed(self, phase):
        need(self.done == phase + 1, "%s: waited for phase %d, %d done" % (self.name, phase, self.done))


class Named:
    """A named barrier of four warps; the vote is or'ed."""

    def __init__(self):
        self.waiting, self.generation, self.vote, self.result = 0, 0, False, False

    def join(self, vote=False):
        self.waiting, self.vote = self.waiting + 1, self.vote or vote
        mine = self.generation
        if self.waiting == 4:
            self.waiting, self.result, self.vote = 0, self.vote, False
            self.generation += 1
        return mine


def simulate(tiles, seed, by_parity=True):
    """tiles: units of each row tile of the CTA's share."""
    rng = random.Random(seed)
    K = slots()
    first, last, seg = [], [], []
    for s, n in enumerate(tiles):
        for i in range(n):
            first.append(i == 0), last.append(i == n - 1), seg.append(s)
    N = len(first)
    pair = lambda name, c: [Barrier("%s%d" % (name, i), c) for i in range(2)]  # noqa: E731
    full = [pair("full%d_" % b, LOADERS) for b in range(2)]
    empty = [pair("empty%d_" % b, 1) for b in range(2)]
    sfull, sfree = pair("sfull", 1), pair("sfree", SOFTMAX)
    rowfull = [Barrier("rowfull%d" % i, ROWS) for i in range(K)]
    rowfree = [Barrier("rowfree%d" % i, LOADERS + SOFTMAX) for i in range(K)]
    qfull, qempty = Barrier("qfull", LOADERS), Barrier("qempty", 1 + SOFTMAX)
    pready = pair("pready", SOFTMAX) if by_parity else [Barrier("pready", SOFTMAX)] * 2
    pphase = (lambda n: n // 2) if by_parity else (lambda n: n)
    bars = [Named(), Named()]
    row = [[None] * ROWS for _ in range(K)]
    tile = [[[None] * LOADERS for _ in range(2)] for _ in range(2)]
    q, sl2 = [None] * LOADERS, [[None] * LOADERS for _ in range(2)]
    S, P = [None, None], [[None] * SOFTMAX for _ in range(2)]
    began, ended = {"s": 0, "v": 0}, {"s": 0, "v": 0}
    vhalf = [0]                                   # halves of the value products done
    written = []                                  # (row tile, warp) outputs
    queue = {"s": [], "v": []}

    def rows(w):
        for m in range(N):
            k = m % K
            yield rowfree[k], m // K - 1
            row[k][w] = m
            rowfull[k].arrive(m // K)

    def loader(w):
        def queries(n):
            yield qempty, seg[n] - 1
            need(ended["s"] >= n, "queries rewritten under their products")
            q[w] = sl2[seg[n] & 1][w] = seg[n]
            qfull.arrive(seg[n])

        def load(n):
            yield rowfull[n % K], n // K
            need(row[n % K] == [n] * ROWS, "rows of another unit")
            rowfree[n % K].arrive(n // K)

        for n in range(-1, N):
            if n >= 0:
                for f in range(2):
                    yield empty[n & 1][f], n // 2 - 1
                    need(n < 2 or vhalf[0] >= 2 * (n - 2) + f + 1, "a tile rewritten under its products")
                    tile[n & 1][f][w] = n
                    full[n & 1][f].arrive(n // 2)
            if n + 1 == N:
                return
            steps = [load(n + 1)] + ([queries(n + 1)] if first[n + 1] else [])
            for step in (steps if n >= 0 else steps[::-1]):
                yield from step

    def scores():
        for n in range(N):
            if first[n]:
                yield qfull, seg[n]
            yield sfree[n & 1], n // 2 - 1
            for f in range(2):
                yield full[n & 1][f], n // 2
                queue["s"].append((n, f))

    def values():
        for n in range(N):
            yield pready[n & 1], pphase(n)
            queue["v"] += [(n, 0), (n, 1)]

    def tensor(kind):
        while ended[kind] < N:
            yield lambda: bool(queue[kind])
            n, f = queue[kind].pop(0)

            def operands():
                need(tile[n & 1][f] == [n] * LOADERS, "%s: a tile of another unit" % kind)
                if kind == "s":
                    need(q == [seg[n]] * LOADERS, "queries of another row tile")
                else:
                    need(P[n & 1] == [n] * SOFTMAX, "weights of another unit: %r" % P[n & 1])
            if f == 0:
                began[kind] = n + 1
            operands()
            if kind == "s":
                S[n & 1] = None
            yield None
            operands()
            if kind == "v":
                vhalf[0] += 1
            if f == 1:
                ended[kind] = n + 1
            if kind == "v":
                empty[n & 1][f].arrive(n // 2)
            elif f == 1:
                S[n & 1] = n
                sfull[n & 1].arrive(n // 2)
                if last[n]:
                    qempty.arrive(seg[n])

    def softmax(w):
        bar = bars[w // 4]
        for n in range(N):
            b = n & 1
            if first[n]:
                yield qfull, seg[n]
                qempty.arrive(seg[n])
            yield rowfull[n % K], n // K
            need(row[n % K] == [n] * ROWS and sl2[seg[n] & 1] == [seg[n]] * LOADERS, "factors of another unit")
            yield sfull[b], n // 2
            need(S[b] == n, "scores of another unit")
            sfree[b].arrive(n // 2)
            yield empty[b][1], n // 2 - 1
            # whether a reference moves: the same for the warps of a barrier
            rises = random.Random((seed, n, w // 4).__hash__()).random() < 0.3 or first[n]
            g = bar.join(rises and w % 4 == n % 4)
            yield lambda: bar.generation != g
            if bar.result and not first[n]:
                yield empty[b ^ 1][1], (n - 1) // 2
                need(ended["v"] == n and began["v"] == n, "accumulators rescaled beside products")
            need(n < 2 or ended["v"] >= n - 1, "weights rewritten under their products")
            P[b][w] = n
            pready[b].arrive(pphase(n))
            rowfree[n % K].arrive(n // K)
            if last[n]:
                yield empty[b][1], n // 2
                need(ended["v"] == n + 1 and began["v"] == n + 1, "accumulators read beside products")
                written.append((seg[n], w))
                g = bar.join()
                yield lambda: bar.generation != g

    actors = ([rows(w) for w in range(ROWS)] + [loader(w) for w in range(LOADERS)] + [scores(), values()] +
              [tensor("s"), tensor("v")] + [softmax(w) for w in range(SOFTMAX)])
    speed = [rng.choice([1, 1, 3, 10]) for _ in actors]
    if rng.random() < 0.5:                        # one half of the softmax warps slow
        for w in range(4):
            speed[-1 - w] = 0.3
    live = {i: next(a, "end") for i, a in enumerate(actors)}
    live = {i: c for i, c in live.items() if c != "end"}
    while live:
        can = [i for i, c in live.items() if c is None or (c() if callable(c) else c[0].ready(c[1]))]
        need(can, "nobody can go on")
        i = rng.choices(can, [speed[j] for j in can])[0]
        if isinstance(live[i], tuple):
            live[i][0].passed(live[i][1])
        c = next(actors[i], "end")
        if c == "end":
            del live[i]
        else:
            live[i] = c
    need(sorted(written) == [(s, w) for s in range(len(tiles)) for w in range(SOFTMAX)], "outputs missing")


SHARES = [[1], [1, 1, 1], [2, 2], [3], [9], [1, 4, 1, 2], [5, 7], [1] * 6, [12]]


@pytest.mark.parametrize("tiles", SHARES, ids=["-".join(map(str, t)) for t in SHARES])
def test_protocol(tiles):
    for seed in range(60):
        simulate(tiles, seed)


def test_model_finds_weights_without_parity():
    faults = 0
    for seed in range(60):
        try:
            simulate([9], seed, by_parity=False)
        except Fault:
            faults += 1
    assert faults > 0
