"""Shared plumbing of the 8-bit cache's GPU tests: random caches built by the oracle, their device copies,
and the attention's error bound.

The bound of one output element (attention), against 64 bits, where p are the exact weights:
* the output's own rounding to bf16: 2^-8 |out| (half a step);
* each weight enters the product rounded: to bf16 for tree keys (2^-8 of it), else, multiplied by its
  block's V scale, to f16 (2^-11 of it, or 2^-25 in a unit that puts the row's largest such product w at 1/2
  or above: 2^-24 w); the product multiplies the code, v / scale; so at most 2^-8 A + 2^-20 w C1,
  A = sum p |v|, C1 = sum of the prefix's |codes| (2^-20 where 2^-24 would do);
* a score that is off by dx moves a weight by a factor exp(dx): 2 dx A more.  dx: the query's elements
  are kept to 2^-17 of the row's largest, so |dx| <= scale 2^-17 qmax K1, K1 = max over the keys of
  sum |k|; the float32 sums of at most 256 products add 2^-16 of scale sum |q k| at most;
* float32 sums over the keys and the joining of splits: 2^-14 A.
The LSE is off by dx, and by 2^-20 of itself for the exponentials, logarithms and sums."""

import numpy as np
import torch

import oracle
import tree_speculative_decoding_split_gb300 as st
from gen import trees as T
import gpu_helpers as H


class Cache:
    """Random 8-bit pools with the blocks of every request scattered over them."""

    def __init__(self, rng, lens, Hkv, d, bs, max_len=None, extra=5, scale_spread=2, pow2=True, stale=True):
        self.lens, self.bs, self.Hkv, self.d = [int(x) for x in lens], bs, Hkv, d
        B = len(self.lens)
        self.max_blocks = max(1, -(-int(max_len or max(self.lens)) // bs))
        held = [-(-n // bs) for n in self.lens]
        nb = sum(held) + extra
        order = rng.permutation(nb)
        self.table = np.full((B, self.max_blocks), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at: at + n]
            at += n
        shape = (nb, Hkv, bs, d)
        self.k = oracle.e4m3_encode(rng.standard_normal(shape) * 64)
        self.v = oracle.e4m3_encode(rng.standard_normal(shape) * 64)
        e = rng.integers(-scale_spread, scale_spread + 1, (2, nb, Hkv)).astype(np.float64)
        f = 1.0 if pow2 else rng.uniform(1, 2, (2, nb, Hkv))
        self.ks, self.vs = ((2.0 ** (e - 6)) * f).astype(np.float32)
        if stale:  # what lies behind a prefix may be anything
            for b, n in enumerate(self.lens):
                if n % bs:
                    self.k[self.table[b, n // bs], :, n % bs:] = 0x7F
                    self.v[self.table[b, n // bs], :, n % bs:] = 0xFF

    def device(self, dev):
        f8 = torch.float8_e4m3fn
        return dict(k_cache=torch.from_numpy(self.k).to(dev).view(f8), v_cache=torch.from_numpy(self.v).to(dev).view(f8),
                    k_scale=torch.from_numpy(self.ks).to(dev), v_scale=torch.from_numpy(self.vs).to(dev),
                    block_table=torch.from_numpy(self.table).to(dev))

    def values(self, b):
        args = (self.table[b], self.bs, self.lens[b])
        return (oracle.gather_kv8(self.k, self.ks.astype(np.float64), *args),
                oracle.gather_kv8(self.v, self.vs.astype(np.float64), *args))


def bf16(x):
    """float64 array rounded to bf16 values, as a torch tensor and as float64."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t, t.double().numpy()


class Queries:
    def __init__(self, rng, B, N, Hq, Hkv, d, n_nodes=None, parents=None, spread=1.0):
        self.n_nodes = np.full(B, N, np.int32) if n_nodes is None else np.asarray(n_nodes, np.int32)
        self.parent = np.full((B, N), -1, np.int32)
        for b in range(B):
            n = int(self.n_nodes[b])
            par = parents[b] if parents is not None else T.random_bfs_tree(rng, n, 8)[0]
            self.parent[b, :n] = par[:n]
        q = rng.standard_normal((B, N, Hq, d)) * spread
        q[..., 3] *= 4
        self.q_t, self.q = bf16(q)
        self.kt_t, self.kt = bf16(rng.standard_normal((B, N, Hkv, d)))
        self.vt_t, self.vt = bf16(rng.standard_normal((B, N, Hkv, d)))


def attend(dev, cache, qs, scale=0.0, status=None, **kw):
    c = cache.device(dev) if isinstance(cache, Cache) else cache
    lens = torch.tensor(cache.lens, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev) if status is None else status
    out, lse = st.tree_attention_kv8(qs.q_t.to(dev), qs.kt_t.to(dev), qs.vt_t.to(dev), c["k_cache"], c["v_cache"],
                                     c["k_scale"], c["v_scale"], lens, torch.from_numpy(qs.n_nodes).to(dev),
                                     torch.from_numpy(qs.parent).to(dev), c["block_table"], scale=scale,
                                     dev_status=status, **kw)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), int(status.item())


def exact(cache, qs, b, scale=0.0):
    """(out, lse, out bound, lse bound) of request b, [N][Hq][d] and [N][Hq]; rows of padding are 0."""
    n, (N, Hq, d) = int(qs.n_nodes[b]), qs.q.shape[1:]
    L = cache.lens[b]
    k0, v0 = cache.values(b)
    s = scale if scale > 0 else 1 / np.sqrt(d)
    mask = oracle.tree_mask(qs.parent[b], n, L)
    blocks = cache.table[b][np.arange(L) // cache.bs]
    slot_vs = cache.vs.astype(np.float64)[blocks].T  # [Hkv][L]
    O, E = np.zeros((N, Hq, d)), np.zeros((N, Hq, d))
    LSE, EL = np.zeros((N, Hq)), np.zeros((N, Hq))
    G = Hq // cache.Hkv
    for g in range(cache.Hkv):
        K = np.concatenate([k0[g], qs.kt[b, :n, g]])
        V = np.concatenate([v0[g], qs.vt[b, :n, g]])
        for h in range(g * G, (g + 1) * G):
            Q = qs.q[b, :n, h]
            x = np.where(mask, s * (Q @ K.T), -np.inf)
            m = x.max(1, keepdims=True)
            w = np.exp(x - m)
            tot = w.sum(1, keepdims=True)
            O[:n, h] = (w @ V) / tot
            LSE[:n, h] = (m + np.log(tot))[:, 0]
            A = (w @ np.abs(V)) / tot
            vs = slot_vs[g]
            top = (w[:, :L] * vs).max(1, keepdims=True) if L else np.zeros((n, 1))
            floor = top * (np.abs(v0[g]) / vs[:, None]).sum(0) if L else 0
            dx = s * (2.0 ** -17 * np.abs(Q).max(1, keepdims=True) * np.abs(K).sum(1).max()
                      + 2.0 ** -16 * (np.abs(Q) @ np.abs(K).T).max(1, keepdims=True))
            E[:n, h] = (2.0 ** -8 * np.abs(O[:n, h]) + (2.0 ** -8 + 2.0 ** -14 + 2 * dx) * A
                        + 2.0 ** -20 * floor / tot)
            EL[:n, h] = dx[:, 0] + 2.0 ** -20 * (np.abs(LSE[:n, h]) + 1)
    return O, LSE, E, EL


def check(cache, qs, out, lse, scale=0.0, requests=None):
    for b in range(len(cache.lens)) if requests is None else requests:
        O, LSE, E, EL = exact(cache, qs, b, scale)
        n = int(qs.n_nodes[b])
        assert (out[b, n:] == 0).all() and (lse[b, n:] == 0).all(), b
        bad = np.abs(out[b] - O) > E
        assert not bad.any(), (b, np.abs(out[b] - O).max(), np.argwhere(bad)[:3].tolist())
        bad = np.abs(lse[b] - LSE) > EL
        assert not bad.any(), (b, np.abs(lse[b] - LSE).max(), np.argwhere(bad)[:3].tolist())


def dev():
    return H.dev()
