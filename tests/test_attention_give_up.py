"""How a block of the attention kernels (csrc/pe_attention.cuh) ends when one of its
bounded waits gives up, replayed on the CPU: roles as actors that a random scheduler
steps, loads and products that finish at random times, and waits that run out at
random.  A role whose wait runs out, or that sees in a wait that another's has, stops;
roles that have begun loads or products wait for them before they end, and when all
have ended the block gives its memory back.

Checked: when it does, no load and no product is in flight, whichever role gave up
and whichever had ended before.  A form whose roles wait for their own only if a wait
of theirs failed is caught: a loading warp that has begun its last load and ended
sees no wait fail."""
from __future__ import annotations

import random

import pytest


class Barrier:
    def __init__(self, count=1):
        self.count, self.pending, self.done = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.done = self.count, self.done + 1

    def over(self, parity):
        return (self.done & 1) != parity


class Block:
    """Roles are generators that yield (condition, whether it may give up) and get
    whether the condition came true."""

    def __init__(self, seed, n, stages, always):
        self.rng, self.n, self.stages, self.always = random.Random(seed), n, stages, always
        self.abort = False
        self.flight = {"load": [], "mma": []}        # events that arrive later, in order per engine
        self.full, self.empty = ([Barrier() for _ in range(stages)] for _ in range(2))
        self.first, self.s_full, self.s_free, self.p_full, self.done, self.drain = (Barrier() for _ in range(6))

    def loader(self):
        if self.n == 0:
            return
        self.flight["load"].append(self.first.arrive)
        f, ok = 0, True
        while f < 2 * self.n:                        # scores' and sums' operands by turns
            s, ph = f % self.stages, f // self.stages & 1
            ok = yield lambda: self.empty[s].over(ph ^ 1), True
            if not ok:
                break
            self.flight["load"].append(self.full[s].arrive)
            f += 1
        if self.always or not ok:
            yield lambda: self.first.over(0), False
            for i in range(max(f - self.stages, 0), f):
                yield lambda: self.full[i % self.stages].over(i // self.stages & 1), False

    def products(self):
        if self.n and not (yield lambda: self.first.over(0), True):
            return False
        f = 0
        for j in range(self.n):
            for what in "sp":
                s, ph = f % self.stages, f // self.stages & 1
                if not (yield lambda: self.full[s].over(ph), True):
                    return False
                if what == "s":
                    if j and not (yield lambda: self.s_free.over((j - 1) & 1), True):
                        return False
                    self.flight["mma"] += [self.s_full.arrive, self.empty[s].arrive]
                else:
                    if not (yield lambda: self.p_full.over(j & 1), True):
                        return False
                    self.flight["mma"] += [self.done.arrive, self.empty[s].arrive]
                f += 1
        return True

    def issuer(self):
        ok = yield from self.products()
        if self.always or not ok:
            self.flight["mma"].append(self.drain.arrive)         # a commit, behind every product issued
            yield lambda: self.drain.over(0), False

    def group(self):
        for j in range(self.n):
            if not (yield lambda: self.s_full.over(j & 1), True):
                return
            self.s_free.arrive()
            if j and not (yield lambda: self.done.over((j - 1) & 1), True):
                return
            self.p_full.arrive()
        if self.n:
            yield lambda: self.done.over((self.n - 1) & 1), True

    def run(self):
        """What is in flight when the last role has ended."""
        roles = {"loader": self.loader(), "issuer": self.issuer(), "group": self.group()}
        waiting = {}
        for name, r in list(roles.items()):
            try:
                waiting[name] = next(r)
            except StopIteration:
                del roles[name]
        patience = self.rng.choice([0.0, 0.002, 0.02, 0.2])
        slow = self.rng.choice([0.1, 0.4, 0.7])
        for _ in range(100000):
            if not roles:
                return {q: len(e) for q, e in self.flight.items()}
            busy = [q for q, e in self.flight.items() if e]
            if busy and self.rng.random() < slow:
                self.flight[self.rng.choice(busy)].pop(0)()
                continue
            name = self.rng.choice(sorted(roles))
            cond, may_give_up = waiting[name]
            came = cond()
            if not came and may_give_up and self.rng.random() < patience:
                self.abort = True
            if not came and not (may_give_up and self.abort):
                continue
            try:
                waiting[name] = roles[name].send(came)
            except StopIteration:
                del roles[name]
        raise AssertionError("the block does not end")


@pytest.mark.parametrize("stages", [2, 4, 5, 8])
def test_nothing_is_in_flight_when_a_block_ends(stages):
    gave_up = 0
    for seed in range(1500):
        b = Block(seed, seed % 9, stages, always=True)
        assert not any(b.run().values()), seed
        gave_up += b.abort
    assert 300 < gave_up < 1400                       # both ways of ending are met


def test_a_role_that_had_ended_leaves_loads_and_products_in_flight():
    """The form in which a role waits for its own only if a wait of its own failed."""
    left = {"load": 0, "mma": 0}
    for seed in range(3000):
        b = Block(seed, seed % 4 + 1, 8, always=False)
        flight = b.run()
        if b.abort:
            for q in left:
                left[q] += flight[q] > 0
    assert left["load"] > 0 and left["mma"] > 0, left
