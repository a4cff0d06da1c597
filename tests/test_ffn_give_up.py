"""The end of a paired product that gave up (host arithmetic only; no GPU).

Two CTAs fill a ring of NS stages; stage i of the run lies in place i % NS.  Both CTAs'
copies of a stage complete on one barrier of the first CTA, which that CTA arms (one
arrival, the bytes of both halves) as it issues its own half.  A CTA refills a place once
the MMAs have read it, and they read it once both halves have landed.  On a give-up each
CTA stops at any stage, so the two may have issued unequal numbers.  The first CTA then
walks over the last NS stages that either has issued: a stage that it never armed itself it
arms for the partner's half alone, from one whose other half never comes it takes that half's
bytes off, and it waits for the stage's phase.

These tests restate the barrier (one arrival and the bytes due, a phase that ends when both
are in) and that walk, let two CTAs run and stop in random order, and check that the wait for
each stage returns exactly when the last copy into it has landed: not before, and not never.
"""
import random

import pytest


class Barrier:
    def __init__(self):
        self.phase, self.arrived, self.tx = 0, False, 0

    def _end(self):
        if self.arrived and self.tx == 0:
            self.phase, self.arrived = self.phase + 1, False

    def arm(self, n):
        assert not self.arrived, "armed twice in a phase"
        self.tx += n
        self.arrived = True
        self._end()

    def complete(self, n):
        self.tx -= n
        self._end()

    def passed(self, i, ns):
        """What a wait for the parity of stage i's phase sees."""
        return (self.phase & 1) != ((i // ns) & 1)


def run_and_stop(rng, ns, total):
    """Barriers, stages issued by either CTA, copies still on their way [(stage, half)]."""
    bars = [Barrier() for _ in range(ns)]
    issued, read, flying = [0, 0], 0, []
    for _ in range(rng.randrange(6 * total)):
        r = rng.randrange(4)
        if r < 2 and issued[r] < total and issued[r] < read + ns:
            i = issued[r]
            if r == 0:
                bars[i % ns].arm(2)
            flying.append((i, r))
            issued[r] += 1
        elif r == 2 and flying:
            i, _ = flying.pop(rng.randrange(len(flying)))
            bars[i % ns].complete(1)
        elif r == 3 and read < min(issued) and bars[read % ns].passed(read, ns):
            read += 1
    return bars, issued, flying


def settle(bars, issued, flying, ns, rng, walk):
    """The first CTA's walk; copies land in random order while it waits."""
    mine, other = issued
    most = max(issued)
    for i in range(max(0, most - ns), most):
        if walk:
            if i >= mine:
                bars[i % ns].arm(1)
            if i >= other:
                bars[i % ns].complete(1)
        while not bars[i % ns].passed(i, ns):
            if not flying:
                return False  # would wait for a copy that does not exist
            j, _ = flying.pop(rng.randrange(len(flying)))
            bars[j % ns].complete(1)
        assert not [f for f in flying if f[0] == i], "the wait returned before a copy landed"
    return not flying


@pytest.mark.parametrize("ns", [4, 6])
def test_every_copy_is_waited_for(ns):
    rng = random.Random(ns)
    unequal = stuck = 0
    for _ in range(4000):
        bars, issued, flying = run_and_stop(rng, ns, rng.randrange(1, 5 * ns))
        assert abs(issued[0] - issued[1]) <= ns
        unequal += issued[0] != issued[1]
        state = rng.getstate()
        copy = [Barrier() for _ in bars]
        for a, b in zip(copy, bars):
            a.__dict__.update(b.__dict__)
        # without settling what was never issued the same waits do not end
        try:
            stuck += not settle(copy, issued, list(flying), ns, rng, walk=False)
        except AssertionError:
            stuck += 1
        rng.setstate(state)
        assert settle(bars, issued, flying, ns, rng, walk=True)
        # every phase that was begun has ended: nothing is due on any barrier
        assert all(b.tx == 0 and not b.arrived for b in bars)
    assert unequal > 500 and stuck > 500
