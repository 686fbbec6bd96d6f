"""The prompt attention kernel's hand-offs where the tensor cores keep the documented order only.

Tensor instructions of one accumulator and shape run in the order they are issued in, a commit waits for all that its
thread has issued, and nothing else is promised.  The walk of test_prompt_protocol with such tensor cores, for both of
the kernel's instances: heads of 128 (a ring of 5 stages, weights over their own scores) and of 64 (8 stages, weights
in columns of their own)."""

import os
import random
import re

import pytest

import test_prompt_protocol as protocol
from test_prompt_protocol import Mbar, Walk, _items

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tree_speculative_decoding_split_gb300", "csrc",
                      "prompt_attention.cu")
INSTANCES = {128: (5, True), 64: (8, False)}  # head size: stages, weights over their scores


class Scores(list):
    """Score columns of the groups; weights go to columns of their own."""

    def __init__(self, weights):
        super().__init__([None, None])
        self.weights = weights

    def __setitem__(self, a, what):
        if what[0] == "P":
            self.weights[a] = what
        else:
            super().__setitem__(a, what)


class Loose(Walk):
    """Tensor cores that run what is queued in any order that is allowed, behind the issuers as they once were."""

    def __init__(self, items, seed, give_up=None, over=True):
        super().__init__(items, seed, give_up)
        self.over, self.pread = over, [Mbar(1), Mbar(1)]
        self.weights = [None, None]
        if not over:
            self.s = Scores(self.weights)

    def issuer_of(self, op):
        if op[0] != "commit":
            return op[1]
        return next(a for bars in (self.sfull, self.ofull, self.qempty, self.pread) for a in (0, 1) if bars[a] is op[1])

    def may_run(self, i):
        op, a = self.queue[i], self.issuer_of(self.queue[i])
        ahead = [x for x in self.queue[:i] if self.issuer_of(x) == a and x[0] != "commit"]
        return not ahead if op[0] == "commit" else all(x[0] != op[0] for x in ahead)

    def engines(self):
        if self.copies and self.rng.random() < 0.5:
            to, at, what, bar = self.copies.pop(self.rng.randrange(len(self.copies)))
            to[at] = what
            bar.arrive()
            return True
        if self.queue:
            op = self.queue.pop(self.rng.choice([i for i in range(len(self.queue)) if self.may_run(i)]))
            if op[0] == "commit":
                op[1].arrive()
            elif op[0] == "S":
                _, a, u, t, k = op
                self.must(self.q[a] == ("Q", u, a) and self.stage[k] == ("K", u, t))
                self.s[a] = ("S", u, t)
            else:
                _, a, u, t, v = op
                seen = ("V", u, t, "seen") if t >= self.items[u][2] else ("V", u, t)
                self.must((self.s if self.over else self.weights)[a] == ("P", u, t) and self.stage[v] == seen)
                self.must(t == 0 or self.o[a] == (u, t))
                self.o[a] = (u, t + 1)
            return True
        return bool(self.copies)


class Ordered(Loose):
    """The issuers as the kernel has them."""

    def issuer(self, a):
        stages = protocol.STAGES
        st, f, g, qn, pn, ok = 0, [0] * stages, [0] * stages, 0, 0, True
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
                st = (st + 1) % stages
                return at

            k = yield from landed(False)
            if tiles and ok:
                ok = yield from self.wait(self.qfull[a], qn & 1)
                if ok and self.over and qn > 0:
                    ok = yield from self.wait(self.ofull[a], (qn - 1) & 1)
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
                        if self.over:
                            self.queue.append(("commit", self.pread[a]))
                            ok = yield from self.wait(self.pread[a], pn & 1)
                            pn += 1
                        if ok:
                            self.queue.append(("S", a, u, t + 1, k))
                            self.queue.append(("commit", self.sfull[a]))
                            if t + 2 == tiles:
                                self.queue.append(("commit", self.qempty[a]))
                    else:
                        self.queue.append(("commit", self.ofull[a]))
                self.turn[a ^ 1].arrive()
                if ok and t >= tiles:
                    self.empty[v].arrive()
                if ok and more and t + 1 >= tiles:
                    self.empty[k].arrive()
            if not ok:
                self.abort = True
            qn += tiles > 0
        if a == 0:
            yield from self.turn[0].sync()


@pytest.fixture(params=sorted(INSTANCES))
def over(request, monkeypatch):
    stages, over = INSTANCES[request.param]
    monkeypatch.setattr(protocol, "STAGES", stages)
    return over


@pytest.mark.parametrize("seed", range(150))
def test_every_product_finds_its_operands(over, seed):
    rng = random.Random(seed)
    walk = Ordered(_items(rng), seed, over=over).run()
    assert not walk.abort
    assert sorted(walk.out) == [(u, a) for u, item in enumerate(walk.items) for a in (0, 1) if item[a]]
    assert not walk.queue and not walk.copies


@pytest.mark.parametrize("seed", range(60))
def test_a_wait_that_gives_up_leaves_nobody_behind(over, seed):
    rng = random.Random(1000 + seed)
    items = _items(rng)
    waits = Ordered(items, seed, over=over).run().waits
    for give_up in sorted({rng.randrange(1, waits + 1) for _ in range(12)} | {1, waits}):
        Ordered(items, seed, give_up, over=over).run()


def test_weights_under_scores_that_do_not_wait_are_found(monkeypatch):
    """The walk sees the mistake: weights over their own scores and no wait ahead of the next ones."""
    monkeypatch.setattr(protocol, "STAGES", 5)
    found = 0
    for seed in range(40):
        try:
            Loose([(4, 4, 3), (3, 3, 2)], seed).run()
        except AssertionError:
            found += 1
    assert found


def test_the_kernel_takes_these_steps():
    code = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    code = re.sub(r"\s+", " ", code)
    stages = {128: INSTANCES[128][0], 64: INSTANCES[64][0]}
    assert f"kStages = D == 128 ? {stages[128]} : {stages[64]};" in code and "kOver = D == 128;" in code
    assert "kColP = kOver ? kColS : 384, kWideP = kOver ? kKeys : kKeys / 2;" in code
    issuer = code[code.index("const int a = warp - 1;"):code.index("uint32_t at_load = 0, phase = 0;")]
    first, steps = issuer[:issuer.index("for (int t = 0; t < w.all; ++t)")], issuer[issuer.index("for (int t = 0; t < w.all; ++t)"):]
    assert first.index("wait(&qfull[a]") < first.index("if (C::kOver && q_n > 0) ok = ok && wait(&ofull[a], (q_n - 1) & 1, &s_abort);") < \
        first.index("named_bar_sync(kBarTurn + a, 64);") < first.index("if (ok && tiles > 0 && lane == 0) { scores(k); umma_commit(&sfull[a]);")
    order = ["landed(t >= w.edge)", "wait(&ofree[a]", "named_bar_sync(kBarP + a, 160);", "named_bar_sync(kBarTurn + a, 64);", "umma_bf16_tmem_a(tO, tP",
             "if (C::kOver) { umma_commit(&pread[a]); ok = wait(&pread[a], p_n++ & 1, &s_abort); } if (ok) { scores(k); umma_commit(&sfull[a]); "
             "if (t + 2 == tiles) umma_commit(&qempty[a]); }", "umma_commit(&ofull[a]);", "named_arrive(kBarTurn + (a ^ 1), 64);"]
    at = [steps.index(x) for x in order]
    assert at == sorted(at) and steps.count("scores(") == 1 and first.count("scores(k)") == 1
    counts = {"full[s]": 1, "held[s]": 1, "empty[s]": 2, "guarded[s]": 1, "qfull[a]": 1, "qempty[a]": 1, "sfull[a]": 1, "pread[a]": 1, "ofull[a]": 1,
              "ofree[a]": 4}
    assert all(f"mbar_init(&{bar}, {n});" in code for bar, n in counts.items())
