"""Plain 64-bit forms of the prompt calls, and inputs for their tests."""

import math

import torch

EPS = 2.0 ** -8  # half a step of bf16, relative


def starts(lens, dev="cuda", front=0):
    """row_start of requests of these lengths, the first one `front` rows in."""
    at = [front]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=dev)


def rows(gen, n, heads, d, dtype=torch.bfloat16, spread=1.0):
    return (torch.randn((n, heads, d), generator=gen, device="cuda") * spread).to(dtype)


def fused(gen, n, hq, hkv, d, pad=0, dtype=torch.bfloat16):
    """q, k, v as views of one projection's rows, with `pad` heads behind them that nothing reads (NaN)."""
    x = rows(gen, n, hq + 2 * hkv + pad, d, dtype)
    x[:, hq + 2 * hkv:] = math.nan
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]


def attention(q, k, v, row_start, scale=None):
    """out, lse, and for every output the bound's terms: sum p |v| and the largest sum |q_c k_c| of its row."""
    n_rows, hq, d = q.shape
    g = hq // k.shape[1]
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = torch.zeros((n_rows, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.zeros((n_rows, hq), dtype=torch.float64, device=q.device)
    mag, size = torch.zeros_like(out), torch.zeros_like(lse)
    at = row_start.tolist()
    for lo, hi in zip(at[:-1], at[1:]):
        if hi == lo:
            continue
        late = torch.ones((hi - lo, hi - lo), dtype=torch.bool, device=q.device).triu_(1)
        for h in range(hq):
            x, y, z = q[lo:hi, h].double(), k[lo:hi, h // g].double(), v[lo:hi, h // g].double()
            s = (x @ y.T * scale).masked_fill_(late, -math.inf)
            size[lo:hi, h] = (x.abs() @ y.abs().T).masked_fill_(late, 0).amax(1)
            lse[lo:hi, h] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[lo:hi, h, None])
            out[lo:hi, h] = p @ z
            mag[lo:hi, h] = p @ z.abs()
    return out, lse, mag, size


def score_error(size, scale, d):
    """How far a float32 score may be off, in units of the exponent: d additions, each off by 2^-23 of the sum of
    magnitudes (additions that cut instead of rounding), and two more roundings of the scaled score."""
    return size * scale * (d + 2) * 2.0 ** -23


def check_attention(got, q, k, v, row_start, scale=None):
    out, lse = got
    d = q.shape[2]
    want, want_lse, mag, size = attention(q, k, v, row_start, scale)
    lo, hi = int(row_start[0]), int(row_start[-1])
    err = score_error(size, 1 / math.sqrt(d) if scale is None else scale, d)
    n = (hi - lo) or 1
    # weights as bf16, the sums of up to n float32 terms, exponentials of scores that are off
    weight = EPS + 2 * err + (n + 8) * 2.0 ** -23
    bound = (1 + EPS) * mag * weight[..., None] + EPS * want.abs() + 1e-30
    assert ((out.double() - want).abs() <= bound)[lo:hi].all(), ((out.double() - want).abs() / bound)[lo:hi].max()
    bound = err + (n + 8) * 2.0 ** -23 + want_lse.abs() * 2.0 ** -23
    assert ((lse.double() - want_lse).abs() <= bound)[lo:hi].all(), ((lse.double() - want_lse).abs() / bound)[lo:hi].max()


def key_weights(q, k, lse, row_start, window, scale=None):
    """weight [Hkv][n_rows], and the same sums of p times what a score and its lse may be off by."""
    n_rows, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    weight = torch.zeros((hkv, n_rows), dtype=torch.float64, device=q.device)
    off = torch.zeros_like(weight)
    at = row_start.tolist()
    for lo, hi in zip(at[:-1], at[1:]):
        n = hi - lo
        w = min(window, n)
        if n == 0:
            continue
        late = torch.arange(n, device=q.device) > torch.arange(n - w, n, device=q.device)[:, None]
        for h in range(hq):
            x, y = q[hi - w:hi, h].double(), k[lo:hi, h // g].double()
            norm = lse[hi - w:hi, h].double()[:, None]
            p = torch.exp((x @ y.T) * scale - norm).masked_fill_(late, 0)
            size = x.abs() @ y.abs().T
            weight[h // g, lo:hi] += p.sum(0)
            # a score, lse times log2(e), and their difference; the exponential itself and the sum's terms
            e = score_error(size, scale, d) + norm.abs() * 2.0 ** -22 + (g * w + 8) * 2.0 ** -23
            off[h // g, lo:hi] += (p * e).sum(0)
    return weight, off


def kept(weight, row_start, budget, first, last):
    """For every request, [Hkv][n_keep] rows kept: python lists."""
    answer = []
    at = row_start.tolist()
    for lo, hi in zip(at[:-1], at[1:]):
        n = hi - lo
        heads = []
        for h in range(weight.shape[0]):
            if n <= budget:
                heads.append(list(range(n)))
                continue
            w = weight[h, lo:hi].tolist()
            cand = range(first, n - last)
            order = sorted(cand, key=lambda j: (w[j] != w[j], -w[j] if w[j] == w[j] else 0.0, j))
            heads.append(list(range(first)) + sorted(order[:budget - first - last]) + list(range(n - last, n)))
        answer.append(heads)
    return answer
