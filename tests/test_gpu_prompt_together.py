"""The prompt calls one after another, as prompts are admitted: positions, rotation, attention, key weights, the rows
that a budget leaves, and from there the 8-bit cache and decoding over it; eager and as one captured graph."""

import math

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import EPS, attention, check_attention, kept, key_weights, rows, starts

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, BS, BUDGET, FIRST, LAST, WINDOW = 4, 8, 2, 128, 16, 96, 4, 16, 32
LENS = [40, 700, 97, 301]
MAX_ROWS = 1400


class Admission:
    """Buffers of one layer, all on the device, and the calls in their order."""

    def __init__(self):
        dev = "cuda"
        i32 = dict(dtype=torch.int32, device=dev)
        self.qkv = torch.zeros((MAX_ROWS, HQ + 2 * HKV, D), dtype=torch.bfloat16, device=dev)
        self.row_start, self.pos0 = torch.zeros(B + 1, **i32), torch.zeros(B, **i32)
        self.turns = st.rope_table(D, 10000.0, "bands", 8.0, 256, 1.0, 4.0).to(dev)
        self.num_blocks = B * (BUDGET // BS + 3) + 5
        self.k_cache, self.v_cache = (torch.zeros((self.num_blocks, HKV, BS, D), device=dev).to(torch.float8_e4m3fn) for _ in "kv")
        self.k_scale, self.v_scale = (torch.ones((self.num_blocks, HKV), device=dev) for _ in "kv")
        self.seq_len, self.n_blocks = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.table = torch.full((B, BUDGET // BS + 3), -1, **i32)
        self.free = torch.arange(self.num_blocks - 1, -1, -1, **i32)
        self.free_count = torch.full((1,), self.num_blocks, **i32)
        self.status = torch.zeros(1, **i32)
        self.tok = torch.zeros((B, 1, HQ + 2 * HKV, D), dtype=torch.bfloat16, device=dev)
        self.one, self.root = torch.ones(B, **i32), torch.full((B, 1), -1, **i32)

    def run(self):
        s = dict(dev_status=self.status)
        q, k, v = self.qkv[:, :HQ], self.qkv[:, HQ:HQ + HKV], self.qkv[:, HQ + HKV:]
        pos = torch.full((MAX_ROWS,), -1, dtype=torch.int32, device="cuda")
        st.rope_positions(self.pos0, row_start=self.row_start, positions=pos, **s)
        q_rot, k_rot = torch.zeros_like(q, memory_format=torch.contiguous_format), torch.zeros_like(k, memory_format=torch.contiguous_format)
        st.rope(q, k, pos, self.turns, q_out=q_rot, k_out=k_rot)
        out, lse = st.prompt_attention(q_rot, k_rot, v, self.row_start, **s)
        weight = st.prompt_key_weights(q_rot, k_rot, lse, self.row_start, WINDOW, **s)
        k_keep, v_keep, index, keep_start, n_keep = st.kv_keep(k_rot, v, weight, self.row_start, BUDGET, first=FIRST, last=LAST,
                                                               rows_out=B * BUDGET, **s)
        st.kv_reserve(self.seq_len, n_keep, self.table, self.n_blocks, self.free, self.free_count, BS, **s)
        length = st.kv8_append(k_keep, v_keep, self.k_cache, self.v_cache, self.k_scale, self.v_scale, self.seq_len, self.table,
                               row_start=keep_start, **s)
        # one new token of every request: its position goes on from the prompt's whole length
        at = st.rope_positions(self.pos0 + self.row_start[1:] - self.row_start[:-1], parent=self.root, n_nodes=self.one, **s)
        tq, tk = st.rope(self.tok[:, :, :HQ], self.tok[:, :, HQ:HQ + HKV], at, self.turns)
        tv = self.tok[:, :, HQ + HKV:].contiguous()
        answer, answer_lse = st.tree_attention_kv8(tq, tk, tv, self.k_cache, self.v_cache, self.k_scale, self.v_scale, length,
                                                   self.one, self.root, self.table, **s)
        return dict(pos=pos, q=q_rot, k=k_rot, v=v, out=out, lse=lse, weight=weight, k_keep=k_keep, v_keep=v_keep, index=index,
                    keep_start=keep_start, n_keep=n_keep, length=length, at=at, tq=tq, tk=tk, tv=tv, answer=answer)

    def fill(self, seed, lens):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.qkv.copy_(rows(gen, MAX_ROWS, HQ + 2 * HKV, D))
        self.tok.copy_(rows(gen, B, HQ + 2 * HKV, D).view(B, 1, HQ + 2 * HKV, D))
        self.row_start.copy_(starts(lens))
        self.pos0.copy_(torch.tensor([0, 5, 77, 123456], dtype=torch.int32))

    def reset(self):
        self.n_blocks.zero_()
        self.table.fill_(-1)
        self.free.copy_(torch.arange(self.num_blocks - 1, -1, -1, dtype=torch.int32))
        self.free_count.fill_(self.num_blocks)


def _check(a, r, lens):
    start = a.row_start
    n = int(start[-1])
    assert int(a.status) == 0
    pos = [p + j for p, m in zip(a.pos0.tolist(), lens) for j in range(m)]
    assert r["pos"][:n].tolist() == pos and (r["pos"][n:] == -1).all()
    assert r["at"].flatten().tolist() == [p + m for p, m in zip(a.pos0.tolist(), lens)]
    check_attention((r["out"][:n], r["lse"][:n]), r["q"][:n], r["k"][:n], r["v"][:n], start)
    want, off = key_weights(r["q"][:n], r["k"][:n], r["lse"][:n], start, WINDOW)
    assert ((r["weight"][:, :n].double() - want).abs() <= off + 1e-37).all()
    chosen = kept(r["weight"].cpu(), start.cpu(), BUDGET, FIRST, LAST)
    assert r["n_keep"].tolist() == [min(m, BUDGET) for m in lens] and torch.equal(r["length"], r["n_keep"])
    total = int(r["keep_start"][-1])
    assert r["index"][:total].tolist() == [list(x) for h in chosen for x in zip(*h)]
    # the answers against attention over what the cache holds: the kept rows' codes and the token itself
    for b, m in enumerate(r["length"].tolist()):
        blocks = a.table[b, :(m + BS - 1) // BS].long()
        for h in range(HQ):
            g = h // (HQ // HKV)

            def whole(cache, scale, own):
                old = cache[blocks, g].double() * scale[blocks, g].double()[:, None, None]
                return torch.cat([old.reshape(-1, D)[:m], own[b, :, g].double()])
            k, v = whole(a.k_cache, a.k_scale, r["tk"]), whole(a.v_cache, a.v_scale, r["tv"])
            src = r["k_keep"][r["keep_start"][b]:r["keep_start"][b] + m, g].double()
            # e4m3: half a step, 2^-4 of the value, or of the smallest normal number under the block's scale
            assert ((k[:m] - src).abs() <= 2.0 ** -4 * src.abs() + 2.0 ** -10 * float(a.k_scale.max())).all()
            p = torch.softmax(k @ r["tq"][b, 0, h].double() / math.sqrt(D), 0)
            got, exact, size = r["answer"][b, 0, h].double(), p @ v, p @ v.abs()
            assert ((got - exact).abs() <= 2 * EPS * size).all()


def test_prompts_are_admitted_and_decoded():
    a = Admission()
    a.fill(1, LENS)
    _check(a, a.run(), LENS)


def test_one_captured_graph_for_other_prompts():
    a = Admission()
    a.fill(2, LENS)
    a.run()
    a.reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = a.run()
    for seed, lens in ((3, LENS), (4, [1, 1, 1, 1]), (5, [0, 1300, 95, 5]), (6, [96, 97, 0, 1000])):
        a.reset()
        a.fill(seed, lens)
        graph.replay()
        _check(a, r, lens)


def test_two_graphs_on_two_streams():
    both = [Admission(), Admission()]
    graphs, results = [], []
    for i, a in enumerate(both):
        a.fill(7 + i, LENS)
        a.run()
        a.reset()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(a.run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(3):
        for a in both:
            a.reset()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
    for a, r in zip(both, results):
        _check(a, r, LENS)
