"""The prompt attention kernel's hand-offs, walked through on the CPU.

Its roles (copies, two MMA issuers, the guard, two softmax groups) and the tensor cores' queue are coroutines over
barriers that behave as the hardware's: an mbarrier knows the parity of its phase only, a named barrier its count.  A
scheduler runs them in random order and the walk checks that every product finds the operands it is meant for, that
nothing is overwritten while it is needed, that all come to an end, and, where a wait gives up, that nobody is left
at a barrier without a limit."""

import random

import pytest

STAGES = 5


class Mbar:
    """count arrivals complete a phase; a waiter sees parities only."""

    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.pending = self.count
            self.phase += 1

    def done(self, parity):
        return (self.phase & 1) != parity


class Named:
    """A named barrier of one waiter and one arriver a round (each stands for its warps)."""

    def __init__(self):
        self.arrived = 0

    def arrive(self):
        self.arrived += 1
        assert self.arrived == 1, "arrived twice in a round"

    def sync(self):
        while not self.arrived:
            yield
        self.arrived = 0


class Walk:
    def must(self, holds):  # (once a wait has given up, results no longer count)
        assert holds or self.abort or self.give_up

    def __init__(self, items, seed, give_up=None):
        # items: (tiles of group 0, of group 1, first guarded tile)
        self.items, self.rng, self.give_up, self.abort, self.waits = items, random.Random(seed), give_up, False, 0
        bars = lambda n, count: [Mbar(count) for _ in range(n)]
        self.full, self.held, self.guarded, self.empty = bars(STAGES, 1), bars(STAGES, 1), bars(STAGES, 1), bars(STAGES, 2)
        self.qfull, self.qempty, self.sfull, self.ofull, self.ofree = (bars(2, 1) for _ in range(5))
        self.turn, self.p = [Named(), Named()], [Named(), Named()]
        self.stage, self.q, self.s, self.o = [None] * STAGES, [None, None], [None, None], [None, None]
        self.queue, self.copies, self.out = [], [], []

    # a bounded wait: gives up when the walk's give_up-th one comes, or once somebody has
    def wait(self, bar, parity):
        self.waits += 1
        if self.waits == self.give_up:
            return False
        while not bar.done(parity):
            if self.abort:
                return False
            yield
        return True

    def all_tiles(self, item):
        return item[1] or item[0]

    def producer(self):
        at, rounds, qn = 0, 0, [0, 0]
        for u, item in enumerate(self.items):
            everything = self.all_tiles(item)
            loads = [("K", 0)] + [x for t in range(everything) for x in ([("V", t)] + ([("K", t + 1)] if t + 1 < everything else []))]
            for n, (kind, t) in enumerate(loads):
                for a in ((0,) if n == 0 else (1,) if n == 1 else ()):
                    if item[a]:
                        if not (yield from self.wait(self.qempty[a], (qn[a] & 1) ^ 1)):
                            self.abort = True
                            return
                        self.copies.append((self.q, a, ("Q", u, a), self.qfull[a]))
                        qn[a] += 1
                if not (yield from self.wait(self.empty[at], (rounds & 1) ^ 1)):
                    self.abort = True
                    return
                bar = self.held[at] if kind == "V" and t >= item[2] else self.full[at]
                self.copies.append((self.stage, at, (kind, u, t), bar))
                at += 1
                if at == STAGES:
                    at, rounds = 0, rounds + 1

    def issuer(self, a):
        st, f, g, qn, ok = 0, [0] * STAGES, [0] * STAGES, 0, True
        if a == 1:
            self.turn[0].arrive()
        for u, item in enumerate(self.items):
            tiles, everything = item[a], self.all_tiles(item)

            def landed(guard):
                nonlocal st, ok
                at, phase = st, (g if guard else f)
                if ok:
                    ok = yield from self.wait((self.guarded if guard else self.full)[at], phase[at])
                phase[at] ^= 1
                st = (st + 1) % STAGES
                return at

            k = yield from landed(False)
            if tiles and ok:
                ok = yield from self.wait(self.qfull[a], qn & 1)
            yield from self.turn[a].sync()
            if ok and tiles:
                self.queue.append(("S", a, u, 0, k))
                self.queue.append(("commit", self.sfull[a]))
                if tiles == 1:
                    self.queue.append(("commit", self.qempty[a]))
            self.turn[a ^ 1].arrive()
            if ok and not tiles:
                self.empty[k].arrive()
            for t in range(everything):
                v = yield from landed(t >= item[2])
                more = t + 1 < everything
                if more:
                    k = yield from landed(False)
                if t == 0 and tiles and ok:
                    ok = yield from self.wait(self.ofree[a], (qn & 1) ^ 1)
                if not ok:
                    self.abort = True
                if t < tiles:
                    yield from self.p[a].sync()
                yield from self.turn[a].sync()
                if ok and t < tiles:
                    self.queue.append(("PV", a, u, t, v))
                    if t + 1 < tiles:
                        self.queue.append(("S", a, u, t + 1, k))
                    self.queue.append(("commit", self.sfull[a] if t + 1 < tiles else self.ofull[a]))
                    if t + 2 == tiles:
                        self.queue.append(("commit", self.qempty[a]))
                self.turn[a ^ 1].arrive()
                if ok and t >= tiles:
                    self.empty[v].arrive()
                if ok and more and t + 1 >= tiles:
                    self.empty[k].arrive()
            qn += tiles > 0
        if a == 0:
            yield from self.turn[0].sync()

    def guard(self):
        load, phase = 0, [0] * STAGES
        for u, item in enumerate(self.items):
            for t in range(item[2], self.all_tiles(item)):
                st = (load + 2 * t + 1) % STAGES
                if not (yield from self.wait(self.held[st], phase[st])):
                    self.abort = True
                    return
                phase[st] ^= 1
                self.must(self.stage[st] == ("V", u, t))
                self.stage[st] = ("V", u, t, "seen")
                self.guarded[st].arrive()
            load += 2 * self.all_tiles(item)

    def softmax(self, a):
        st, sn, on, ok = 0, 0, 0, True
        for u, item in enumerate(self.items):
            tiles, everything = item[a], self.all_tiles(item)

            def released():
                nonlocal st
                if ok:
                    self.empty[st].arrive()
                st = (st + 1) % STAGES

            if not tiles:
                st = (st + 2 * everything) % STAGES
                continue
            for t in range(tiles):
                if ok:
                    ok = yield from self.wait(self.sfull[a], sn & 1)
                sn += 1
                if not ok:
                    self.abort = True
                if t > 0:
                    released()
                released()
                if ok:
                    self.must(self.s[a] == ("S", u, t))
                    yield
                    self.must(self.s[a] == ("S", u, t))
                    self.s[a] = ("P", u, t)
                self.p[a].arrive()
                while self.p[a].arrived:
                    yield
            if ok:
                ok = yield from self.wait(self.ofull[a], on & 1)
            on += 1
            if not ok:
                self.abort = True
            released()
            st = (st + 2 * (everything - tiles)) % STAGES
            if not ok:
                continue
            self.must(self.o[a] == (u, tiles))
            yield
            self.must(self.o[a] == (u, tiles))
            self.out.append((u, a))
            self.ofree[a].arrive()

    def engines(self):
        """Copies land in any order, the tensor cores work through their queue; `idle` tells whether anything moved."""
        if self.copies and self.rng.random() < 0.5:
            to, at, what, bar = self.copies.pop(self.rng.randrange(len(self.copies)))
            to[at] = what
            bar.arrive()
            return True
        if self.queue:
            op = self.queue.pop(0)
            if op[0] == "commit":
                op[1].arrive()
            elif op[0] == "S":
                _, a, u, t, k = op
                self.must(self.q[a] == ("Q", u, a) and self.stage[k] == ("K", u, t))
                self.s[a] = ("S", u, t)
            else:
                _, a, u, t, v = op
                seen = ("V", u, t, "seen") if t >= self.items[u][2] else ("V", u, t)
                self.must(self.s[a] == ("P", u, t) and self.stage[v] == seen)
                self.must(t == 0 or self.o[a] == (u, t))
                self.o[a] = (u, t + 1)
            return True
        return bool(self.copies)

    def run(self):
        roles = [self.producer(), self.issuer(0), self.issuer(1), self.guard(), self.softmax(0), self.softmax(1)]
        quiet = 0
        while roles:
            moved = self.engines()
            role = self.rng.choice(roles)
            before = (self.waits, self.abort, len(self.queue), len(self.copies), len(self.out))
            try:
                next(role)
            except StopIteration:
                roles.remove(role)
                moved = True
            quiet = 0 if moved or before != (self.waits, self.abort, len(self.queue), len(self.copies), len(self.out)) else quiet + 1
            assert quiet < 4000, "nobody moves any more"
        while self.engines():
            pass
        return self


def _items(rng):
    items = []
    for _ in range(rng.randrange(1, 6)):
        kind = rng.randrange(4)
        one = rng.randrange(1, 6)
        tiles = (one, 0) if kind == 0 else (one, one) if kind < 3 else (one, one + 1)
        items.append((*tiles, rng.randrange(max(0, one - 2), one)))
    return items


@pytest.mark.parametrize("seed", range(150))
def test_every_product_finds_its_operands(seed):
    rng = random.Random(seed)
    walk = Walk(_items(rng), seed).run()
    assert not walk.abort
    assert sorted(walk.out) == [(u, a) for u, item in enumerate(walk.items) for a in (0, 1) if item[a]]
    assert not walk.queue and not walk.copies


@pytest.mark.parametrize("seed", range(60))
def test_a_wait_that_gives_up_leaves_nobody_behind(seed):
    rng = random.Random(1000 + seed)
    items = _items(rng)
    waits = Walk(items, seed).run().waits
    for give_up in sorted({rng.randrange(1, waits + 1) for _ in range(12)} | {1, waits}):
        Walk(items, seed, give_up).run()
