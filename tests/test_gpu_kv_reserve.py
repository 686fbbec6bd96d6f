"""Block tables, free list and slot map against the oracle, to the bit."""

import numpy as np
import pytest
import torch

import oracle
import tree_speculative_decoding_split_gb300 as st
import kv8_helpers as K8

pytestmark = pytest.mark.gpu


class Blocks:
    """The same state for the oracle (lists) and for the device."""

    def __init__(self, rng, lens, bs, max_blocks, spare):
        self.bs, self.max_blocks = bs, max_blocks
        held = [-(-int(n) // bs) for n in lens]
        self.nb = sum(held) + spare
        order = rng.permutation(self.nb).tolist()
        self.table = []
        for h in held:
            self.table.append(order[:h])
            order = order[h:]
        self.free = order

    def device(self, dev):
        t = np.full((len(self.table), self.max_blocks), -1, np.int32)
        for b, row in enumerate(self.table):
            t[b, : len(row)] = row
        f = np.full(self.nb, -1, np.int32)
        f[: len(self.free)] = self.free
        i = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        return dict(block_table=torch.from_numpy(t).to(dev), n_blocks=i([len(r) for r in self.table]),
                    free_list=torch.from_numpy(f).to(dev), free_count=i([len(self.free)]))

    def compare(self, s):
        torch.cuda.synchronize()
        table, n = s["block_table"].cpu().numpy(), s["n_blocks"].tolist()
        for b, row in enumerate(self.table):
            assert n[b] == len(row) and table[b, : n[b]].tolist() == row and (table[b, n[b]:] == -1).all(), b
        count = int(s["free_count"].item())
        assert s["free_list"][:count].tolist() == self.free


def _call(s, lens, add, bs, cap=None, **kw):
    dev = s["block_table"].device
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    i = lambda x: torch.tensor([int(v) for v in x], dtype=torch.int32, device=dev)  # noqa: E731
    slots, starts = st.kv_reserve(i(lens), i(add), block_size=bs, slot_cap=cap, dev_status=status, **s, **kw)
    torch.cuda.synchronize()
    return slots, starts, int(status.item())


def _slots(answer, add, cap):
    want = []
    for a, n in zip(answer, add):
        want += a if a is not None else [-1] * int(n)
    return want + [-1] * (cap - len(want))


@pytest.mark.parametrize("B,bs,top,new", [(1, 16, 2100, 63), (1, 256, 0, 1), (3, 64, 100, 0), (32, 16, 4000, 63),
                                          (64, 32, 50, 255), (65, 16, 300, 20), (200, 64, 500, 700), (1500, 16, 60, 40),
                                          (8192, 128, 300, 3)])
def test_growth_and_shrinking(B, bs, top, new):
    dev = K8.dev()
    rng = np.random.default_rng(B + bs)
    lens = rng.integers(0, top + 1, B)
    add = rng.integers(0, new + 1, B)
    blocks = Blocks(rng, lens, bs, -(-(top + new) // bs) + 3, int(-(-(add + bs) // bs).sum()) + 5)
    s = blocks.device(dev)
    for grow in (add, np.zeros(B, int), add[::-1].copy()):
        cap = int(grow.sum()) + 3
        answer = oracle.reserve(lens, grow, blocks.table, blocks.free, bs)
        slots, starts, status = _call(s, lens, grow, bs, cap=cap)
        assert status == 0
        assert starts.tolist() == np.concatenate([[0], np.cumsum(grow)]).tolist()
        assert slots.tolist() == _slots(answer, grow, cap)
        blocks.compare(s)


@pytest.mark.parametrize("B", [6, 100])
def test_one_gives_while_another_takes(B):
    """Lengths that fall and rise in the same call, with an empty free list: blocks change hands."""
    dev = K8.dev()
    rng = np.random.default_rng(B)
    lens = rng.integers(100, 400, B)
    blocks = Blocks(rng, lens, 16, 64, 0)
    s = blocks.device(dev)
    after = rng.permutation(lens)
    after[0] = 1
    answer = oracle.reserve(after, np.ones(B, int), blocks.table, blocks.free, 16)
    slots, _, status = _call(s, after, np.ones(B, int), 16, cap=B)
    served = [a is not None for a in answer]
    assert status == (0 if all(served) else 7)
    assert slots.tolist() == _slots(answer, np.ones(B, int), B)
    blocks.compare(s)


@pytest.mark.parametrize("B", [5, 90])
def test_too_few_blocks_serves_a_prefix_of_the_requests(B):
    dev = K8.dev()
    rng = np.random.default_rng(B)
    lens = np.full(B, 10)
    add = np.array([30 + 16 * (b % 3) if b != 2 else 0 for b in range(B)])
    blocks = Blocks(rng, lens, 16, 8, B)
    s = blocks.device(dev)
    lens[B - 1] = 0  # gives its block back although requests before it go without
    answer = oracle.reserve(lens, np.where(np.arange(B) == B - 1, 0, add), blocks.table, blocks.free, 16)
    add[B - 1] = 0
    slots, _, status = _call(s, lens, add, 16, cap=int(add.sum()))
    assert status == 7 and any(a is None for a in answer)
    assert slots.tolist() == _slots(answer, add, int(add.sum()))
    blocks.compare(s)


@pytest.mark.parametrize("B", [4, 70])
@pytest.mark.parametrize("kind", ["len", "count", "held", "table"])
def test_bad_requests_are_left_alone(B, kind):
    dev = K8.dev()
    rng = np.random.default_rng(B)
    lens, add = np.full(B, 20), np.full(B, 20)
    blocks = Blocks(rng, lens, 16, 4, 4 * B)
    s = blocks.device(dev)
    held = blocks.table[1]
    bad_lens, bad_add = lens.copy(), add.copy()
    if kind == "len":
        bad_lens[1] = -3
    if kind == "count":
        bad_add[1] = 64   # wants more than max_blocks
    if kind == "held":
        s["n_blocks"][1] = 9
    if kind == "table":
        s["block_table"][1, 1] = blocks.nb  # (slot 20 lies in it)
        held = held[:1] + [blocks.nb]
        blocks.table[1] = held
    others = [b for b in range(B) if b != 1 or kind == "table"]
    table = [blocks.table[b] for b in others]
    answer = oracle.reserve(lens[others], add[others], table, blocks.free, 16)
    full = [None] * B
    for b, a, t in zip(others, answer, table):
        full[b], blocks.table[b] = a, t
    if kind == "table":
        full[1] = [x if x < blocks.nb * 16 else -1 for x in full[1]]
    cap = int(bad_add.sum())
    slots, _, status = _call(s, bad_lens, bad_add, 16, cap=cap)
    assert status == 7
    assert slots.tolist() == _slots(full, bad_add, cap)
    if kind == "held":
        s["n_blocks"][1] = len(held)
    blocks.compare(s)


@pytest.mark.parametrize("B", [4, 70])
@pytest.mark.parametrize("kind", ["count_high", "count_low", "overfull", "cap"])
def test_a_broken_list_or_short_map_changes_nothing(B, kind):
    dev = K8.dev()
    rng = np.random.default_rng(B)
    lens, add = np.full(B, 40), np.full(B, 20)
    blocks = Blocks(rng, lens, 16, 8, 4 * B)
    s = blocks.device(dev)
    cap = 20 * B
    if kind == "count_high":
        s["free_count"][0] = blocks.nb + 1
    if kind == "count_low":
        s["free_count"][0] = -1
    if kind == "overfull":  # blocks given back that the list says are free already
        s["free_count"][0] = blocks.nb
        lens, add = np.zeros(B, int), np.zeros(B, int)
    if kind == "cap":
        cap -= 1
    before = {k: v.clone() for k, v in s.items()}
    slots, starts, status = _call(s, lens, add, 16, cap=cap)
    assert status == 7 and (slots == -1).all() and (starts == 0).all()
    for k in s:
        assert torch.equal(s[k], before[k]), k


def test_without_a_slot_map():
    dev = K8.dev()
    rng = np.random.default_rng(1)
    blocks = Blocks(rng, [100, 3], 64, 8, 9)
    s = blocks.device(dev)
    oracle.reserve([100, 3], [200, 64], blocks.table, blocks.free, 64)
    slots, starts, status = _call(s, [100, 3], [200, 64], 64)
    assert slots is None and status == 0 and starts.tolist() == [0, 200, 264]
    blocks.compare(s)
