"""The barrier protocol of the attention kernels (csrc/pe_attention.cuh), replayed
on the CPU: loading warp, issuing warps, softmax or gradient groups as actors that
a random scheduler steps, loads and products that finish at random times, and
barriers that are waited for by the parity of a phase, as mbarriers are.

Checked in every step: a product reads the tiles and the probabilities it is meant
to, nothing is overwritten before its reader is done, and no run gets stuck.  Two
planted mistakes (one barrier for both groups, whose parity a group may take for
that of two phases before; a ring slot given back before the product is done) show
that the model sees such faults."""
from __future__ import annotations

import random

import pytest


class Fault(AssertionError):
    pass


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.done = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.done = self.count, self.done + 1

    def over(self, parity):
        """What a wait by parity sees: the phase before the current one has that parity."""
        return (self.done & 1) != parity


class Run:
    """Actors are generators that yield a condition to wait for; `later` holds events
    in flight, one queue per engine (a queue keeps its order, queues do not)."""

    def __init__(self, seed):
        self.rng, self.actors, self.queues = random.Random(seed), [], {}

    def later(self, queue, event):
        self.queues.setdefault(queue, []).append(event)

    def go(self):
        waiting = [(a, None) for a in self.actors]
        weights = [self.rng.choice([1, 1, 4, 20]) for _ in waiting]      # some actors are slow in this run
        for _ in range(200000):
            ready = [i for i, (a, c) in enumerate(waiting) if a is not None and (c is None or c())]
            busy = [q for q, e in self.queues.items() if e]
            if not ready and not busy:
                if any(a is not None for a, _ in waiting):
                    raise Fault("stuck")
                return
            if busy and (not ready or self.rng.random() < self.speed):
                self.queues[self.rng.choice(busy)].pop(0)()
                continue
            i = self.rng.choices(ready, [weights[j] for j in ready])[0]
            a = waiting[i][0]
            try:
                waiting[i] = (a, next(a))
            except StopIteration:
                waiting[i] = (None, None)
        raise Fault("no end")


def need(ok, what):
    if not ok:
        raise Fault(what)


class Slot:
    def __init__(self, n, at=0):
        self.n, self.at, self.phase = n, at, 0

    def next(self, by=1):
        self.at += by
        if self.at >= self.n:
            self.at, self.phase = self.at - self.n, self.phase ^ 1


def backward(seed, mode, n, stages, sweeps=1, mistake=None):
    """mode: "own" (queries), "shared" or "alias" (keys).  `n` streamed tiles."""
    R = Run(seed)
    R.speed = R.rng.choice([0.05, 0.3, 0.7])
    total, second = n * sweeps, n * (sweeps - 1)
    full, empty = [Barrier(1) for _ in range(stages)], [Barrier(1) for _ in range(stages)]
    s_full, d_full, acc_done = ([Barrier(c) for _ in range(2)] for c in (1, 1, 1))
    s_free = [Barrier(1) for _ in range(2)]
    one = Barrier(1)                                  # the planted mistake: one barrier for both groups
    acc_full, off_full = Barrier(1), Barrier(2)
    ring, score, score_read = [None] * stages, [None, None], [True, True]
    place, place_read = {}, {}
    key = lambda b: "both" if mode == "shared" else b  # noqa: E731
    summed = []

    def loader():
        r = Slot(stages)
        for f in range(total):
            at, ph = r.at, r.phase
            yield lambda: empty[at].over(ph ^ 1)
            ring[at] = None

            def land(at=at, f=f):
                ring[at] = f
                full[at].arrive()
            R.later(("load", R.rng.randrange(3)), land)
            r.next()

    def scores(b):
        r = Slot(stages, b)
        for j in range(b, total, 2):
            k, at, ph = j >> 1, r.at, r.phase
            yield lambda: full[at].over(ph)
            if k:
                yield lambda: s_free[b].over((k - 1) & 1)

            def product(j=j, at=at):
                need(ring[at] == j, "scores read another tile")
                need(score_read[b], "scores overwritten before they were read")
                if mode == "alias":
                    need(place_read.get(b, True), "p and ds overwritten by scores")
                score[b], score_read[b] = j, False
            R.later(("mma", b), product)
            R.later(("mma", b), s_full[b].arrive)
            r.next(2)

    def group(g):
        met = sweeps == 1
        for j in range(g, total, 2):
            k = j >> 1
            if j >= second and not met:
                off_full.arrive()
                yield lambda: off_full.over(0)
                met = True
            yield lambda: s_full[g].over(k & 1)
            need(score[g] == j and not score_read[g], "group read other scores")
            score_read[g] = True
            if mode != "alias":
                s_free[g].arrive()
            yield None
            if mode == "shared" and j > 0:
                if mistake == "one barrier":
                    yield lambda: one.over((j - 1) & 1)
                else:
                    yield lambda: acc_done[1 - g].over(((j - 1) >> 1) & 1)
            elif mode == "own" and k > 0:
                yield lambda: acc_done[g].over((k - 1) & 1)
            if j >= second:
                need(place_read.get(key(g), True), "p and ds overwritten before the sums read them")
                place[key(g)], place_read[key(g)] = j, False
            d_full[g].arrive()
        if not met:
            off_full.arrive()
            yield lambda: off_full.over(0)
        yield lambda: acc_full.over(0)
        need(summed == list(range(second, total)), "results read before every tile was added")

    def sums():
        r = Slot(stages)
        for j in range(total):
            b, at, ph = j & 1, r.at, r.phase
            yield lambda: full[at].over(ph)
            yield lambda: d_full[b].over((j >> 1) & 1)
            if j < second:
                acc_done[b].arrive()
                empty[at].arrive()
            else:
                def product(j=j, b=b, at=at):
                    need(ring[at] == j, "sums read another tile")
                    need(place.get(key(b)) == j and not place_read[key(b)], "sums read other p and ds")
                    place_read[key(b)] = True
                    summed.append(j)
                if mistake == "early":
                    empty[at].arrive()
                R.later(("mma", 2), product)
                free = s_free[b] if mode == "alias" else (one if mistake == "one barrier" else acc_done[b])
                R.later(("mma", 2), free.arrive)
                if mistake != "early":
                    R.later(("mma", 2), empty[at].arrive)
                if j + 1 == total:
                    R.later(("mma", 2), acc_full.arrive)
            r.next()

    R.actors = [loader(), scores(0), scores(1), group(0), group(1), sums()]
    R.go()
    need(len(summed) == n, "a tile was not added")


def forward(seed, n0, n1, stages):
    """Two query tiles that meet n0 and n1 key tiles (n1 = None: no second tile)."""
    R = Run(seed)
    R.speed = R.rng.choice([0.05, 0.3, 0.7])
    tiles = [n0] if n1 is None else [n0, n1]
    n_max = max(tiles)
    full, empty = [Barrier(1) for _ in range(stages)], [Barrier(len(tiles)) for _ in range(stages)]
    s_full, s_free, p_full, pv_done, turn = ([Barrier(1) for _ in range(2)] for _ in range(5))
    ring, score, read, prob, used = [None] * stages, [None, None], [True, True], [None, None], [True, True]
    out = [[], []]
    order = [("k", 0)] + [x for j in range(n_max) for x in ([("k", j + 1)] if j + 1 < n_max else []) + [("v", j)]]

    def loader():
        r = Slot(stages)
        for what in order[:2 * n_max]:
            at, ph = r.at, r.phase
            yield lambda: empty[at].over(ph ^ 1)
            ring[at] = None

            def land(at=at, what=what):
                ring[at] = what
                full[at].arrive()
            R.later(("load", R.rng.randrange(3)), land)
            r.next()

    def mma(t):
        n, r = tiles[t], Slot(stages)

        def issue(j):
            def product(at=r.at, j=j):
                need(ring[at] == ("k", j), "scores read another tile")
                need(read[t], "scores overwritten before they were read")
                score[t], read[t] = j, False
            R.later(("mma", t), product)
            R.later(("mma", t), s_full[t].arrive)
            R.later(("mma", t), empty[r.at].arrive)
        if not n_max:
            return
        yield lambda: full[r.at].over(r.phase)
        issue(0) if n else empty[r.at].arrive()
        r.next()
        for j in range(n_max):
            if j + 1 < n_max:
                yield lambda: full[r.at].over(r.phase)
                if j + 1 < n:
                    yield lambda: s_free[t].over(j & 1)
                issue(j + 1) if j + 1 < n else empty[r.at].arrive()
                r.next()
            yield lambda: full[r.at].over(r.phase)
            if j < n:
                yield lambda: p_full[t].over(j & 1)

                def product(at=r.at, j=j):
                    need(ring[at] == ("v", j), "product read another tile")
                    need(prob[t] == j and not used[t], "product read other probabilities")
                    used[t] = True
                    out[t].append(j)
                R.later(("mma", t), product)
                R.later(("mma", t), pv_done[t].arrive)
                R.later(("mma", t), empty[r.at].arrive)
            else:
                empty[r.at].arrive()
            r.next()

    def softmax(t):
        n, other = tiles[t], tiles[1 - t] if len(tiles) > 1 else 0
        for j in range(n):
            yield lambda: s_full[t].over(j & 1)
            need(score[t] == j and not read[t], "softmax read other scores")
            read[t] = True
            s_free[t].arrive()
            yield None
            if j and R.rng.random() < 0.3:            # the output is rescaled
                yield lambda: pv_done[t].over((j - 1) & 1)
                need(out[t] == list(range(j)), "output rescaled in the middle of a product")
            k = j if t else j - 1
            if 0 <= k < other:
                yield lambda: turn[t].over(k & 1)
            turn[1 - t].arrive()
            if j:
                yield lambda: pv_done[t].over((j - 1) & 1)
            need(used[t], "probabilities overwritten before their product")
            prob[t], used[t] = j, False
            p_full[t].arrive()
        if n:
            yield lambda: pv_done[t].over((n - 1) & 1)
        need(out[t] == list(range(n)), "output read before every tile was added")

    R.actors = [loader()] + [mma(t) for t in range(len(tiles))] + [softmax(t) for t in range(len(tiles))]
    R.go()


@pytest.mark.parametrize("mode,stages", [("own", 4), ("own", 8), ("shared", 4), ("shared", 8), ("alias", 4), ("own", 2)])
def test_backward_protocol(mode, stages):
    for seed in range(120):
        n = seed % 17 + 1
        backward(seed, mode, n, stages, sweeps=2 if mode == "own" and n <= 4 else 1)


@pytest.mark.parametrize("stages", [5, 8])
def test_forward_protocol(stages):
    for seed in range(150):
        n0 = seed % 13
        forward(seed, n0, None if seed % 3 == 0 else max(n0 + seed % 4 - 1, 0), stages)


@pytest.mark.parametrize("stages", [4, 8])
def test_forward_protocol_of_one_tile(stages):
    for seed in range(100):
        forward(seed, seed % 19, None, stages)


def test_the_model_sees_planted_mistakes():
    def caught(**kw):
        for seed in range(400):
            try:
                backward(seed, n=16, stages=8, **kw)
            except Fault:
                return True
        return False
    assert caught(mode="shared", mistake="one barrier")
    assert caught(mode="own", mistake="early")
