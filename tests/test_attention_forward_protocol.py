"""The forward attention kernel's barriers (csrc/pe_attention.cuh) replayed on the CPU
warp by warp: four softmax warps a tile that arrive on the tile's barriers each, a
turn barrier for each of the four pairs of warps that share an SM quarter, and
mistakes planted in every rule that keeps data from being overwritten or a wait from
having no end.  (test_attention_protocol has the backward kernels, and the forward
one with a tile's warps as one actor.)"""
from __future__ import annotations

import pytest

from tests.test_attention_protocol import Barrier, Fault, Run, Slot, need

WARPS = 4


def forward(seed, n0, n1, stages, mistake=None):
    """Two query tiles that meet n0 and n1 key tiles (n1 = None: no second tile)."""
    R = Run(seed)
    R.speed = R.rng.choice([0.05, 0.3, 0.7])
    tiles = [n0] if n1 is None else [n0, n1]
    n_max = max(tiles)
    full, empty = [Barrier(1) for _ in range(stages)], [Barrier(len(tiles)) for _ in range(stages)]
    s_full, pv_done = ([Barrier(1) for _ in range(2)] for _ in range(2))
    s_free, p_full = ([Barrier(1 if mistake == "one warp arrives" else WARPS) for _ in range(2)] for _ in range(2))
    turn = [[Barrier(1) for _ in range(WARPS)] for _ in range(2)]
    ring, out = [None] * stages, [[], []]
    score, read = [None, None], [set(range(WARPS)), set(range(WARPS))]     # whose scores; which warps have read them
    prob = [[None] * WARPS for _ in range(2)]                              # the key tile of each warp's probabilities
    used = [set(range(WARPS)), set(range(WARPS))]
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
                need(len(read[t]) == WARPS, "scores overwritten before every warp had read them")
                score[t], read[t] = j, set()
            if mistake == "early slot":
                empty[r.at].arrive()
            R.later(("mma", t), product)
            R.later(("mma", t), s_full[t].arrive)
            if mistake != "early slot":
                R.later(("mma", t), empty[r.at].arrive)
        if not n_max:
            return
        yield lambda: full[r.at].over(r.phase)
        issue(0) if n else empty[r.at].arrive()
        r.next()
        for j in range(n_max):
            if j + 1 < n_max:
                yield lambda: full[r.at].over(r.phase)
                if j + 1 < n and mistake != "scores unasked":
                    yield lambda: s_free[t].over(j & 1)
                issue(j + 1) if j + 1 < n else empty[r.at].arrive()
                r.next()
            yield lambda: full[r.at].over(r.phase)
            if j < n:
                yield lambda: p_full[t].over(j & 1)

                def product(at=r.at, j=j):
                    need(ring[at] == ("v", j), "product read another tile")
                    need(prob[t] == [j] * WARPS and not used[t], "product read other probabilities")
                    used[t] = set(range(WARPS))
                    out[t].append(j)
                R.later(("mma", t), product)
                R.later(("mma", t), pv_done[t].arrive)
                R.later(("mma", t), empty[r.at].arrive)
            elif mistake != "slot kept":
                empty[r.at].arrive()
            r.next()

    def softmax(t, w):
        n, other = tiles[t], tiles[1 - t] if len(tiles) > 1 else 0
        if mistake == "turns without end":
            other = n_max + 1 if len(tiles) > 1 else 0
        for j in range(n):
            yield lambda: s_full[t].over(j & 1)
            need(score[t] == j and w not in read[t], "softmax read other scores")
            read[t].add(w)
            s_free[t].arrive()
            yield None
            if j and R.rng.random() < 0.3:            # the output is rescaled
                if mistake != "rescaled at once":
                    yield lambda: pv_done[t].over((j - 1) & 1)
                need(out[t] == list(range(j)), "output rescaled in the middle of a product")
            k = j if t else j - 1
            if 0 <= k < other:
                yield lambda: turn[t][w].over(k & 1)
            turn[1 - t][w].arrive()
            if j and mistake != "stored at once":
                yield lambda: pv_done[t].over((j - 1) & 1)
            need(w in used[t], "probabilities overwritten before their product")
            prob[t][w] = j
            used[t].discard(w)
            p_full[t].arrive()
        if n:
            yield lambda: pv_done[t].over((n - 1) & 1)
        need(out[t] == list(range(n)), "output read before every tile was added")

    R.actors = [loader()] + [mma(t) for t in range(len(tiles))] + [softmax(t, w) for t in range(len(tiles)) for w in range(WARPS)]
    R.go()


def tiles_of(seed):
    n0 = seed % 11
    return n0, None if seed % 3 == 0 else max(n0 + seed % 4 - 1, 0)


@pytest.mark.parametrize("stages", [4, 5, 8])
def test_forward_protocol_warp_by_warp(stages):
    for seed in range(90):
        forward(seed, *tiles_of(seed), stages)
    for seed in range(10):
        forward(seed, 1, 9, stages)


@pytest.mark.parametrize("mistake", ["early slot", "one warp arrives", "scores unasked", "slot kept", "rescaled at once",
                                     "stored at once", "turns without end"])
def test_planted_mistakes_are_seen(mistake):
    for seed in range(200):
        try:
            # (a slot that is kept is missed only by a tile that needs many more keys)
            forward(seed, *((1, 9) if mistake == "slot kept" else tiles_of(seed)), 4, mistake)
        except Fault:
            return
    raise AssertionError("not seen")
