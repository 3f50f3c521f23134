"""The way out of the many-row product after a wait that ran out, as a model on the CPU.

A pair of CTAs feeds one tensor core: both producers' copies of a block complete on the even CTA's mbarrier, the MMA
warp's commits arrive in both CTAs.  When a role gives up, the others stop at blocks of their own, and nothing may be
in flight when a CTA leaves.  The model runs the roles in random order, lets any wait that is not yet satisfied run
out, and checks after the wind-down that every copy, MMA and arrival has landed.  mbarriers are modelled by their
definition: a phase is complete when its arrivals and its bytes are, and a wait names a parity only.
"""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.tx, self.phase = count, count, 0, 0

    def _turn(self):
        if self.pending == 0 and self.tx == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def arrive(self, expect=0):
        self.tx += expect
        self.pending -= 1
        assert self.pending >= 0
        self._turn()

    def bytes(self, n):
        self.tx -= n
        self._turn()

    def done(self, parity):          # what a wait for `parity` sees
        return self.phase % 2 != parity


class Pair:
    def __init__(self, rng, stages, accs, blocks, give_up):
        self.rng, self.S, self.A, self.N, self.p = rng, stages, accs, blocks, give_up
        self.full = [Barrier(1) for _ in range(stages)]                       # of the even CTA
        self.empty = [[Barrier(1) for _ in range(stages)] for _ in range(2)]
        self.t_full = [[Barrier(1) for _ in range(accs)] for _ in range(2)]
        self.t_empty = [Barrier(2) for _ in range(accs)]                      # one warp of each CTA stands for all
        self.copies, self.mmas, self.arrivals = [], [], []                    # in flight
        self.landed = set()
        self.issued, self.computed, self.failed = [0, 0], 0, False

    # what happens by itself
    def hardware(self):
        r = self.rng
        kind = r.choice(["copy", "mma", "arrival"])
        if kind == "copy" and self.copies:
            rank, u = self.copies.pop(r.randrange(len(self.copies)))
            self.landed.add((rank, u))
            self.full[u % self.S].bytes(1)
        elif kind == "mma" and self.mmas:                                     # in order
            u = self.mmas.pop(0)
            for cta in range(2):
                self.arrivals += [self.empty[cta][u % self.S], self.t_full[cta][u % self.A]]
        elif kind == "arrival" and self.arrivals:
            self.arrivals.pop(r.randrange(len(self.arrivals))).arrive()

    def copy(self, rank, u):
        """Asks for block u: its stage must be free of MMAs and of the copies of the block before it."""
        assert u - self.S not in self.mmas
        assert u < self.S or all((c, u - self.S) in self.landed for c in range(2))
        if rank == 0:
            self.full[u % self.S].arrive(expect=2)
        self.copies.append((rank, u))

    def wait(self, bar, parity):
        """Waits, or gives up: yields until done, returns whether it is."""
        while not bar.done(parity):
            if self.rng.random() < self.p:
                self.failed = True
                return False
            yield
        return True

    def producer(self, rank):
        for u in range(self.N):
            if not (yield from self.wait(self.empty[rank][u % self.S], (u // self.S) % 2 ^ 1)):
                return
            self.copy(rank, u)
            self.issued[rank] = u + 1
            yield
        for u in range(self.N, self.N + self.S):                              # the last uses of the stages
            if not (yield from self.wait(self.empty[rank][u % self.S], (u // self.S) % 2 ^ 1)):
                return

    def tensor(self):
        for u in range(self.N):
            if not (yield from self.wait(self.full[u % self.S], (u // self.S) % 2)):
                return
            if not (yield from self.wait(self.t_empty[u % self.A], (u // self.A) % 2 ^ 1)):
                return
            assert all((c, u) in self.landed for c in range(2))
            self.mmas.append(u)
            self.computed = u + 1
            yield

    def reader(self, rank):
        for u in range(self.N):
            if not (yield from self.wait(self.t_full[rank][u % self.A], (u // self.A) % 2)):
                return
            self.t_empty[u % self.A].arrive()
            yield

    def run(self):
        roles = [self.producer(0), self.producer(1), self.tensor(), self.reader(0), self.reader(1)]
        speed = self.rng.choice([1.0, 0.2, 0.03])                             # of the memory and the tensor core
        while roles:
            if self.rng.random() < speed:
                self.hardware()
            role = self.rng.choice(roles)
            try:
                next(role)
            except StopIteration:
                roles.remove(role)

    def last(self, bars, uses):
        for u in range(max(0, uses - len(bars)), uses):
            limit = 100000
            while not bars[u % len(bars)].done((u // len(bars)) % 2):
                self.hardware()
                limit -= 1
                assert limit, "a wait of the wind-down is never satisfied"

    def wind_down(self):
        for cta in range(2):                       # a cluster barrier: both before the copies below
            self.last(self.empty[cta], self.computed)
            self.last(self.t_full[cta], self.computed)
        assert not self.mmas
        uses = max(self.issued)
        assert uses - min(self.issued) <= self.S
        order = [0, 1]
        self.rng.shuffle(order)
        for rank in order:
            for u in range(self.issued[rank], uses):
                self.copy(rank, u)
        self.last(self.full, uses)


@pytest.mark.parametrize("give_up", [0.0, 0.003, 0.03, 0.3])
@pytest.mark.parametrize("stages,accs,blocks", [(5, 2, 1), (5, 2, 4), (6, 4, 40), (5, 2, 23)])
def test_nothing_is_in_flight_when_a_pair_leaves(stages, accs, blocks, give_up):
    rng = random.Random(stages * 1000 + blocks * 10 + int(give_up * 1000))
    failed = uneven = flying = 0
    for _ in range(150):
        p = Pair(rng, stages, accs, blocks, give_up)
        p.run()
        if p.failed:
            failed += 1
            uneven += p.issued[0] != p.issued[1]
            flying += bool(p.copies)
            p.wind_down()
        assert not p.copies and not p.mmas
        if p.failed or give_up == 0:
            assert not p.arrivals
    assert (failed > 0) == (give_up > 0)
    if give_up >= 0.03 and blocks > stages:        # the model meets what the wind-down is for
        assert uneven > 0 and flying > 0
