"""The 8-bit cache's calls together, as a decoding loop makes them: blocks reserved, prompts appended, then rounds
of tree attention, acceptance, appending of the accepted path and giving back of blocks, eager and from one captured
graph, every state against the oracle."""

import types

import numpy as np
import pytest
import torch

import oracle
import tree_speculative_decoding_split_gb300 as st
import kv8_helpers as K8

pytestmark = pytest.mark.gpu


class Loop:
    def __init__(self, rng, prompts, N, G, Hkv, d, bs, vocab=16):
        self.dev, self.rng, self.N, self.bs, self.d, self.Hkv = K8.dev(), rng, N, bs, d, Hkv
        self.B, self.Hq, self.vocab = len(prompts), G * Hkv, vocab
        self.max_blocks = -(-(max(prompts) + 8 * N) // bs)
        self.nb = sum(-(-(n + 8 * N) // bs) for n in prompts) + 3
        dev, i32 = self.dev, torch.int32
        f8 = torch.float8_e4m3fn
        shape = (self.nb, Hkv, bs, d)
        self.pools = [torch.full(shape, 0x7F, dtype=torch.uint8, device=dev).view(f8) for _ in range(2)]
        self.scales = [torch.full(shape[:2], float("nan"), device=dev) for _ in range(2)]
        self.table = torch.full((self.B, self.max_blocks), -1, dtype=i32, device=dev)
        self.n_blocks = torch.zeros(self.B, dtype=i32, device=dev)
        free = rng.permutation(self.nb).astype(np.int32)
        self.free = torch.from_numpy(free).to(dev)
        self.free_count = torch.full((1,), self.nb, dtype=i32, device=dev)
        self.seq_len = torch.zeros(self.B, dtype=i32, device=dev)
        self.status = torch.zeros(1, dtype=i32, device=dev)
        self.room = torch.full((self.B,), N, dtype=i32, device=dev)
        self.none = torch.zeros_like(self.room)
        self.weight = K8.bf16(rng.standard_normal((vocab, self.Hq * d)))[0].to(dev)
        # the same for the oracle
        self.o_free, self.o_table = free.tolist(), [[] for _ in prompts]
        self.o_cache = [np.full(shape, 0x7F, np.uint8) for _ in range(2)]
        self.o_scale = [np.full(shape[:2], np.nan) for _ in range(2)]
        self.o_len = [0] * self.B
        self._prompt(prompts)
        self.inputs()
        self.static = {k: v.to(dev) for k, v in self.fresh.items()}

    def reserve(self, add, slot_cap=None):
        return st.kv_reserve(self.seq_len, add, self.table, self.n_blocks, self.free, self.free_count, self.bs, slot_cap,
                             dev_status=self.status)

    def _prompt(self, prompts):
        total = sum(prompts)
        rows = [K8.bf16(self.rng.standard_normal((total, self.Hkv, self.d))) for _ in range(2)]
        add = torch.tensor(prompts, dtype=torch.int32, device=self.dev)
        _, starts = self.reserve(add, total)
        new_len = st.kv8_append(rows[0][0].to(self.dev), rows[1][0].to(self.dev), *self.pools, *self.scales, self.seq_len,
                                self.table, row_start=starts, dev_status=self.status)
        self.seq_len.copy_(new_len)
        oracle.reserve(self.o_len, prompts, self.o_table, self.o_free, self.bs)
        at = np.concatenate([[0], np.cumsum(prompts)])
        for b in range(self.B):
            for c in range(2):
                oracle.append_rows(rows[c][1][at[b]: at[b + 1]], self.o_cache[c], self.o_scale[c], 0, self.o_table[b], self.bs)
        self.o_len = list(prompts)
        self.compare()

    def inputs(self):
        """Another round's queries, tree and tokens; nodes behind n_nodes are padding."""
        r, B, N = self.rng, self.B, self.N
        n = r.integers(max(1, N // 2), N + 1, B)
        n[0], n[-1] = 1, N
        self.qs = K8.Queries(r, B, N, self.Hq, self.Hkv, self.d, n_nodes=n)
        self.qs.kt_t[1, n[1]:] = float("nan")
        self.qs.vt_t[1, n[1]:] = float("nan")
        self.fresh = dict(q=self.qs.q_t, k=self.qs.kt_t, v=self.qs.vt_t, n=torch.from_numpy(self.qs.n_nodes),
                          parent=torch.from_numpy(self.qs.parent),
                          tokens=torch.from_numpy(r.integers(0, self.vocab, (B, N)).astype(np.int32)))

    def round(self):
        s = self.static
        self.reserve(self.room)
        out, lse = st.tree_attention_kv8(s["q"], s["k"], s["v"], *self.pools, *self.scales, self.seq_len, s["n"], s["parent"],
                                         self.table, dev_status=self.status)
        r = st.verify_accept(out.view(self.B, self.N, -1), self.weight, s["tokens"], s["parent"], s["n"], "greedy",
                             dev_status=self.status)
        new_len = st.kv8_append(s["k"], s["v"], *self.pools, *self.scales, self.seq_len, self.table, path=r["path"],
                                accept_len=r["accept_len"], dev_status=self.status)
        before = self.seq_len.clone()
        self.seq_len.copy_(new_len)
        self.reserve(self.none)
        self.out = (out, lse, r["path"], r["accept_len"], before)

    def compare(self):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        assert self.seq_len.tolist() == self.o_len
        table, n = self.table.cpu().numpy(), self.n_blocks.tolist()
        for b, row in enumerate(self.o_table):
            assert n[b] == len(row) and table[b, : n[b]].tolist() == row and (table[b, n[b]:] == -1).all(), b
        count = int(self.free_count.item())
        assert self.free[:count].tolist() == self.o_free
        for b, row in enumerate(self.o_table):
            for c in range(2):
                got = self.pools[c].view(torch.uint8)[row].cpu().numpy()
                assert np.array_equal(got, self.o_cache[c][row]), (b, c)
                assert np.array_equal(self.scales[c][row].cpu().numpy(), self.o_scale[c][row].astype(np.float32)), (b, c)

    def check(self):
        """The round just made, against the oracle's state before it, which it then brings up to date."""
        torch.cuda.synchronize()
        out, lse, path, accept = (x.double().cpu().numpy() for x in self.out[:4])
        cache = types.SimpleNamespace(lens=self.o_len, bs=self.bs, Hkv=self.Hkv, vs=self.o_scale[1],
                                      table=[np.array(t + [0], np.int64) for t in self.o_table])
        cache.values = lambda b: tuple(oracle.gather_kv8(self.o_cache[c], self.o_scale[c], self.o_table[b], self.bs,
                                                         self.o_len[b]) for c in range(2))
        K8.check(cache, self.qs, out, lse)
        oracle.reserve(self.o_len, [self.N] * self.B, self.o_table, self.o_free, self.bs)
        for b in range(self.B):
            nodes = path[b, : int(accept[b]) + 1].astype(int)
            assert nodes[0] == 0 and (self.qs.parent[b, nodes[1:]] == nodes[:-1]).all()
            for c, rows in ((0, self.qs.kt), (1, self.qs.vt)):
                oracle.append_rows(rows[b, nodes], self.o_cache[c], self.o_scale[c], self.o_len[b], self.o_table[b], self.bs)
            self.o_len[b] += len(nodes)
        oracle.reserve(self.o_len, [0] * self.B, self.o_table, self.o_free, self.bs)
        self.compare()
        return int(accept.sum())


@pytest.mark.parametrize("N,G,Hkv,d,bs,prompts", [(63, 4, 2, 128, 16, [130, 3, 700, 64]), (7, 2, 2, 128, 64, [64, 1, 300]),
                                                  (1, 4, 2, 64, 32, [31, 32, 100, 9, 500]),
                                                  (255, 2, 1, 64, 128, [200, 127, 1, 1000, 40])])
def test_decoding_rounds(N, G, Hkv, d, bs, prompts):
    """Two eager rounds, then one captured round replayed four times with other queries, trees and lengths."""
    rng = np.random.default_rng(N + bs)
    loop = Loop(rng, prompts, N, G, Hkv, d, bs)

    def next_inputs():
        loop.inputs()
        for k, v in loop.fresh.items():
            loop.static[k].copy_(v)

    accepted = 0
    for i in range(2):
        if i:
            next_inputs()
        loop.round()
        accepted += loop.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop.round()
    for _ in range(4):
        next_inputs()
        graph.replay()
        accepted += loop.check()
    assert accepted > 0 or N == 1


def _plain(rng, N=3):
    """Arguments of a plain attention and append call."""
    dev = K8.dev()
    cache = K8.Cache(rng, [70, 5], 2, 128, 16, max_len=96)
    qs = K8.Queries(rng, 2, N, 4, 2, 128)
    c = cache.device(dev)
    pools = [c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"]]
    lens = torch.tensor(cache.lens, dtype=torch.int32, device=dev)
    attend = [qs.q_t.to(dev), qs.kt_t.to(dev), qs.vt_t.to(dev), *pools, lens, torch.from_numpy(qs.n_nodes).to(dev),
              torch.from_numpy(qs.parent).to(dev), c["block_table"]]
    append = [attend[1], attend[2], *pools, lens, c["block_table"]]
    path = dict(path=torch.tensor([[0, -1, -1]] * 2, dtype=torch.int32, device=dev),
                accept_len=torch.zeros(2, dtype=torch.int32, device=dev))
    return attend, append, path


def test_both_ways_of_marshalling_agree():
    """A plain call goes through the native marshalling, one with a stream, a workspace or a scale that is no float
    through the interpreted one: the same answers, and given outputs come back themselves."""
    attend, append, path = _plain(np.random.default_rng(1))
    native = st._native()
    order = attend[:7] + [attend[10]] + attend[7:10]
    assert native.attend(*order, None, None, 0.1, None) is not None
    out, lse = st.tree_attention_kv8(*attend, scale=1.0)
    here = torch.cuda.current_stream()
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    for kw in (dict(stream=here), dict(workspace=ws), dict(scale=1)):
        again = st.tree_attention_kv8(*attend, **{"scale": 1.0, **kw})
        torch.cuda.synchronize()
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    mine = torch.empty_like(out), torch.empty_like(lse)
    back = st.tree_attention_kv8(*attend, scale=1.0, out=mine[0], lse=mine[1])
    assert back[0] is mine[0] and back[1] is mine[1] and torch.equal(mine[0], out) and torch.equal(mine[1], lse)
    states = []
    for kw in (dict(), dict(stream=here), dict(new_len=torch.empty(2, dtype=torch.int32, device="cuda"))):
        pools = [x.clone() for x in append[2:6]]
        new_len = st.kv8_append(*append[:2], *pools, *append[6:], **path, **kw)
        torch.cuda.synchronize()
        assert new_len.tolist() == [71, 6] and kw.get("new_len", new_len) is new_len
        states.append(pools)
    for pools in states[1:]:
        for a, b in zip(pools, states[0]):
            assert torch.equal(a.view(torch.uint8) if a.dim() == 4 else a, b.view(torch.uint8) if b.dim() == 4 else b)


@pytest.mark.parametrize("i,change,error", [
    (0, lambda t: t.float(), TypeError), (0, lambda t: t.transpose(1, 2), ValueError), (1, lambda t: t[:, :2], ValueError),
    (1, lambda t: t[:, :2].contiguous(), ValueError), (2, lambda t: t.half(), TypeError), (3, lambda t: t.cpu(), ValueError),
    (4, lambda t: t[:-1], ValueError), (5, lambda t: t.double(), TypeError), (6, lambda t: t[:, :1], ValueError),
    (7, lambda t: t.long(), TypeError), (8, lambda t: t[:1], ValueError), (9, lambda t: t[:, :2].contiguous(), ValueError),
    (10, lambda t: t[0], ValueError), (7, lambda t: t.tolist(), TypeError)])
def test_refused_tensors(i, change, error):
    attend, append, path = _plain(np.random.default_rng(2))
    attend[i] = change(attend[i])
    with pytest.raises(error):
        st.tree_attention_kv8(*attend)
    where = {1: 0, 2: 1, 3: 2, 4: 3, 5: 4, 6: 5, 7: 6, 10: 7}.get(i)
    if where is not None and i != 1:
        append[where] = attend[i]
        with pytest.raises((error, AttributeError)):
            st.kv8_append(*append, **path)


def test_refusals_by_the_library():
    attend, append, path = _plain(np.random.default_rng(3))
    pools = [torch.zeros((4, 2, 48, 128), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)] * 2
    scales = [torch.ones((4, 2), device="cuda")] * 2
    with pytest.raises(st.SpecError, match="UNSUPPORTED"):
        st.tree_attention_kv8(*attend[:3], *pools, *scales, *attend[7:])
    with pytest.raises(st.SpecError, match="UNSUPPORTED"):
        st.kv8_append(*append[:2], *pools, *scales, *append[6:], **path)
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(st.SpecError, match="UNSUPPORTED"):
        st.kv_reserve(i, i, i.view(2, 1).clone(), i.clone(), i.clone(), i[:1].clone(), 48)
    with pytest.raises(ValueError):
        st.kv_reserve(i[:1], i, i.view(2, 1).clone(), i.clone(), i.clone(), i[:1].clone(), 16)


@pytest.mark.parametrize("N", [1, 40])
def test_graphs_that_share_a_workspace(N):
    """Two captured calls with one workspace of the caller's, replayed in turn after other lengths have been written:
    the answers of eager calls."""
    dev = K8.dev()
    rng = np.random.default_rng(4 + N)
    ws = torch.empty(1 << 27, dtype=torch.uint8, device=dev)
    calls, outs, graphs = [], [], []
    for lens in ([2600, 31], [64, 5000, 700]):
        cache = K8.Cache(rng, lens, 2, 128, 32)
        qs = K8.Queries(rng, len(lens), N, 8, 2, 128)
        c = cache.device(dev)
        calls.append([qs.q_t.to(dev), qs.kt_t.to(dev), qs.vt_t.to(dev), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"],
                      torch.tensor(lens, dtype=torch.int32, device=dev), torch.from_numpy(qs.n_nodes).to(dev),
                      torch.from_numpy(qs.parent).to(dev), c["block_table"]])
    for call in calls:
        st.tree_attention_kv8(*call, workspace=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(st.tree_attention_kv8(*call, workspace=ws))
    for shorter in (0, 7, 29):
        for call in calls:
            call[7].sub_(shorter)
        want = [st.tree_attention_kv8(*call) for call in calls]
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for (out, lse), (o, e) in zip(want, outs):
            assert torch.equal(out, o) and torch.equal(lse, e)
