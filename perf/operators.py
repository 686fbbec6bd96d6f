"""Cases, plain forms and exact values of the 8-bit paged KV cache's operators.

Three operators that one verification round over a paged 8-bit cache runs one after another:

  reserve   the block tables grow to hold every request's new rows (blocks come off a free list on
            the device) and the slot of every new row is written out; after the round the tables
            shrink again.  One pass is the growth and the shrinking, so the state ends as it began.
  append    new K/V rows (a prompt's, or the accepted path's rows of the draft tree) become e4m3
            codes with one power-of-two scale for each block and KV head.
  attend    tree attention of bf16 query rows over the 8-bit prefix and the tree's own bf16 K/V; a
            tree of one node is single-token decoding.

``run`` computes them with elementary torch operations, or, where ``own`` is true, with the
framework's kernels.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
SCALE_EXP_MIN, SCALE_EXP_MAX = -64, 120


# ---- sizes ---------------------------------------------------------------------------------------

def _spread(lo, hi, count):
    """`count` lengths from lo to hi, evenly spaced, the long ones not all at one end."""
    if count == 1:
        return [hi]
    even = [lo + (hi - lo) * i // (count - 1) for i in range(count)]
    return even[::2] + even[1::2][::-1]


def _lens(c):
    return _spread(c["lo"], c["hi"], c["batch"])


def _new_rows(c):
    """Rows that every request adds: a tree's nodes, an accepted path, or a prompt."""
    if c["op"] == "append" and c["form"] == "path":
        return [1 + (5 * b + 2) % c["new_hi"] for b in range(c["batch"])]
    return _spread(c["new_lo"], c["new_hi"], c["batch"])


def _nodes(c):
    n = c["nodes"]
    return [n - (3 * b) % (n // 4 + 1) for b in range(c["batch"])] if c["ragged"] else [n] * c["batch"]


def _trees(c):
    """Parent arrays [batch][nodes] (-1 for the root and for padding): random recursive trees, siblings
    and parents close together, as a draft numbered breadth-first has them."""
    rng = random.Random(c["nodes"] * 1009 + c["batch"])
    rows = []
    for n in _nodes(c):
        par = [-1] + [max(0, (i - 1) // 2 - rng.randrange(0, 2)) for i in range(1, n)]
        rows.append(par + [-1] * (c["nodes"] - n))
    return rows


def _blocks(slots, bs):
    return (slots + bs - 1) // bs


def listed():
    return [
        # the round of one request: 63 tree slots behind a 2K prefix, blocks of 16
        {"name": "reserve_round_b1", "op": "reserve", "batch": 1, "lo": 2048, "hi": 2048, "new_lo": 63, "new_hi": 63, "bs": 16},
        # the same for a batch of 32 at 4K
        {"name": "reserve_round_b32", "op": "reserve", "batch": 32, "lo": 3900, "hi": 4300, "new_lo": 40, "new_hi": 63, "bs": 16},
        # admission of 512 prompts of 1 to 4K tokens at once, blocks of 64: a slot for each of a million rows
        {"name": "reserve_admit_b512", "op": "reserve", "batch": 512, "lo": 0, "hi": 0, "new_lo": 1, "new_hi": 4095, "bs": 64},
        # accepted paths of a batch of 32 after a round: a handful of rows each, blocks half full
        {"name": "append_path_b32", "op": "append", "form": "path", "dtype": "bf16", "batch": 32, "lo": 3900, "hi": 4300,
         "nodes": 63, "new_hi": 7, "hkv": 8, "d": 128, "bs": 16},
        # eight prompts of 0.5K to 8K tokens, appended behind shared system prompts of odd lengths
        {"name": "append_prompt_b8", "op": "append", "form": "rows", "dtype": "bf16", "batch": 8, "lo": 0, "hi": 301,
         "new_lo": 512, "new_hi": 8192, "hkv": 8, "d": 128, "bs": 64},
        # a long-context batch of 32K to 128K rows from float32 projections, heads of 64
        {"name": "append_long_f32", "op": "append", "form": "rows", "dtype": "f32", "batch": 4, "lo": 0, "hi": 0,
         "new_lo": 32768, "new_hi": 131072, "hkv": 8, "d": 64, "bs": 256},
        # single-token decoding of one request: latency
        {"name": "decode_b1_l2k", "op": "attend", "batch": 1, "lo": 2048, "hi": 2048, "nodes": 1, "ragged": False, "hq": 32,
         "hkv": 8, "d": 128, "bs": 64},
        # single-token decoding of a batch of 32 at ragged lengths around 4K
        {"name": "decode_b32_l4k", "op": "attend", "batch": 32, "lo": 2111, "hi": 6081, "nodes": 1, "ragged": False, "hq": 32,
         "hkv": 8, "d": 128, "bs": 16},
        # the 63-node tree of one request at 2K
        {"name": "tree63_b1_l2k", "op": "attend", "batch": 1, "lo": 2048, "hi": 2048, "nodes": 63, "ragged": False, "hq": 32,
         "hkv": 8, "d": 128, "bs": 64},
        # 63-node trees of a batch of 32 at 4K
        {"name": "tree63_b32_l4k", "op": "attend", "batch": 32, "lo": 4096, "hi": 4096, "nodes": 63, "ragged": False, "hq": 32,
         "hkv": 8, "d": 128, "bs": 64},
        # ragged trees of up to 127 nodes, eight requests of 0.5K to 8K tokens, heads of 64
        {"name": "tree127_b8_d64", "op": "attend", "batch": 8, "lo": 512, "hi": 8192, "nodes": 127, "ragged": True, "hq": 16,
         "hkv": 8, "d": 64, "bs": 32},
        # the long-context layer: 255-node trees, prefixes of 32K to 128K, 64 query heads
        {"name": "tree255_b4_l128k", "op": "attend", "batch": 4, "lo": 32768, "hi": 131072, "nodes": 255, "ragged": False,
         "hq": 64, "hkv": 8, "d": 128, "bs": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["reserve", "append", "append", "attend", "attend", "attend"])
    bs = rng.choice([16, 32, 64, 128, 256])
    if op == "reserve":
        hi = _log(rng, 1, 8192)
        batch = _log(rng, 1, 512)
        new = _log(rng, 1, max(1, min(8192, (1 << 20) // batch)))
        return {"op": op, "batch": batch, "lo": rng.randrange(0, hi + 1), "hi": hi, "new_lo": rng.randrange(0, new + 1),
                "new_hi": new, "bs": bs}
    d, hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    if op == "append":
        hi = _log(rng, 1, 8192)
        c = {"op": op, "form": rng.choice(["path", "rows"]), "dtype": rng.choice(["bf16", "bf16", "f32"]),
             "batch": _log(rng, 1, 32), "lo": rng.randrange(0, hi + 1), "hi": hi, "hkv": hkv, "d": d, "bs": bs}
        if c["form"] == "path":
            c["nodes"] = _log(rng, 2, 255)
            c["new_hi"] = rng.randrange(1, min(c["nodes"], 12) + 1)
        else:
            c["new_hi"] = _log(rng, 1, 131072 // c["batch"])
            c["new_lo"] = rng.randrange(0, c["new_hi"] + 1)
        return c
    nodes = 1 if rng.random() < 0.4 else _log(rng, 2, 255)
    batch = _log(rng, 1, 32)
    hi = _log(rng, 1, 131072 // batch)
    return {"op": op, "batch": batch, "lo": rng.randrange(0, hi + 1), "hi": hi, "nodes": nodes,
            "ragged": rng.random() < 0.5, "hq": hkv * rng.choice([1, 2, 4, 5, 8]), "hkv": hkv, "d": d, "bs": bs}


# ---- inputs --------------------------------------------------------------------------------------

def _ints(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _rows(gen, shape, d, hkv, dev):
    """K or V rows [..., hkv, d] as a layer makes them: unit variance, each head at its own magnitude,
    a few channels several times the others."""
    x = torch.randn(shape, generator=gen, device=dev)
    channel = torch.ones(d, device=dev)
    channel[::23] = 4.0
    head = 0.5 + torch.arange(hkv, device=dev, dtype=torch.float32)[:, None] / hkv
    return x.mul_(head * channel)


def _pool(gen, c, num_blocks, dev):
    """A filled e4m3 pool [num_blocks][hkv][bs][d] and its scales [num_blocks][hkv]."""
    x = _rows(gen, (num_blocks, c["bs"], c["hkv"], c["d"]), c["d"], c["hkv"], dev).transpose(1, 2).contiguous()
    scale = _scale_of(x.abs().amax(dim=(2, 3)))
    return (x / scale[:, :, None, None]).to(torch.float8_e4m3fn), scale


def _table(gen, blocks, max_blocks, num_blocks, dev):
    """Block table [batch][max_blocks] (-1 behind each request's own), blocks in random order."""
    order = torch.randperm(num_blocks, generator=gen, device=dev).to(torch.int32)
    have = torch.tensor(blocks, device=dev)
    start = torch.cumsum(have, 0) - have
    col = torch.arange(max_blocks, device=dev)
    at = (start[:, None] + col).clamp_(max=num_blocks - 1)
    return torch.where(col < have[:, None], order[at], torch.full_like(order[:1], -1)), order


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens, bs, batch = _lens(c), c["bs"], c["batch"]
    s = {"case": c, "seq_len": _ints(lens, dev)}
    if c["op"] == "reserve":
        new = _new_rows(c)
        held = [_blocks(n, bs) for n in lens]
        full = [_blocks(n + m, bs) for n, m in zip(lens, new)]
        num_blocks = sum(full) + 64
        s["num_blocks"], s["slots"] = num_blocks, sum(new)
        s["table"], order = _table(gen, held, max(full) + 2, num_blocks, dev)
        s["n_blocks"] = _ints(held, dev)
        s["n_new"] = _ints(new, dev)
        s["none_new"] = torch.zeros_like(s["n_new"])
        # the free list: the blocks that no table names, behind them room for the others
        s["free"] = torch.cat([order[sum(held):], torch.full_like(order[:sum(held)], -1)])
        s["free_count"] = _ints([num_blocks - sum(held)], dev)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
        return s
    hkv, d = c["hkv"], c["d"]
    if c["op"] == "append":
        new = _new_rows(c)
        full = [_blocks(n + m, bs) for n, m in zip(lens, new)]
        dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        num_blocks = sum(full) + 8
        s["table"], _ = _table(gen, full, max(full) + 2, num_blocks - 1, dev)  # the last block stays unused
        s["k_cache"], s["k_scale"] = _pool(gen, c, num_blocks, dev)
        s["v_cache"], s["v_scale"] = _pool(gen, c, num_blocks, dev)
        if c["form"] == "path":
            shape = (batch, c["nodes"], hkv, d)
            path = [sorted(random.Random(seed * 977 + b).sample(range(1, c["nodes"]), m - 1)) for b, m in enumerate(new)]
            s["path"] = _ints([[0] + p + [-1] * (c["new_hi"] - 1 - len(p)) for p in path], dev)
            s["accept_len"] = _ints([m - 1 for m in new], dev)
        else:
            shape = (sum(new), hkv, d)
            s["row_start"] = _ints([sum(new[:b]) for b in range(batch + 1)], dev)
        s["k_new"] = _rows(gen, shape, d, hkv, dev).to(dtype)
        s["v_new"] = _rows(gen, shape, d, hkv, dev).to(dtype)
        s["units"] = max(_blocks(n + m, bs) - n // bs for n, m in zip(lens, new))
        return s
    full = [_blocks(n, bs) for n in lens]
    num_blocks = sum(full) + 8
    s["table"], _ = _table(gen, full, max(full) + _blocks(256, bs), num_blocks, dev)
    s["k_cache"], s["k_scale"] = _pool(gen, c, num_blocks, dev)
    s["v_cache"], s["v_scale"] = _pool(gen, c, num_blocks, dev)
    n, hq = c["nodes"], c["hq"]
    s["k_tree"] = _rows(gen, (batch, n, hkv, d), d, hkv, dev).to(torch.bfloat16)
    s["v_tree"] = _rows(gen, (batch, n, hkv, d), d, hkv, dev).to(torch.bfloat16)
    s["q"] = torch.randn((batch, n, hq, d), generator=gen, device=dev).to(torch.bfloat16)
    s["n_nodes"], s["parent"] = _ints(_nodes(c), dev), _ints(_trees(c), dev)
    s["longest"] = max(lens)
    return s


# ---- the plain forms -----------------------------------------------------------------------------

def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s, its exponent held to [-64, 120]; amax = m 2^k with
    m in [1/2, 1), and 448 = 0.875 * 2^9."""
    m, k = torch.frexp(amax)
    e = torch.where(m > 0.875, k - 8, k - 9)
    e = torch.where(amax > 0, e, torch.full_like(e, SCALE_EXP_MIN)).clamp(SCALE_EXP_MIN, SCALE_EXP_MAX)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)    # 2^e by its bits


def _reserve(table, n_blocks, free, free_count, seq_len, n_new, bs):
    """The tables hold ceil((seq_len + n_new) / bs) blocks afterwards; changes the four first arguments."""
    want = (seq_len + n_new + bs - 1) // bs
    rel, need = (n_blocks - want).clamp(min=0), (want - n_blocks).clamp(min=0)
    rel_start, need_start = torch.cumsum(rel, 0) - rel, torch.cumsum(need, 0) - need
    released = rel.sum()
    col = torch.arange(table.shape[1], device=table.device)
    num = free.shape[0]
    # blocks given back go on top of the free list, the first of them last
    gone = (col >= want[:, None]) & (col < n_blocks[:, None])
    to = free_count + released - 1 - (rel_start[:, None] + col - want[:, None])
    longer = torch.cat([free, free[:1]])
    longer.scatter_(0, torch.where(gone, to, num).reshape(-1).long(), table.reshape(-1))
    free.copy_(longer[:num])
    top = free_count + released
    # blocks taken come off its top, in the order of the requests; all that a request wants, or none
    ok = torch.cumsum(need, 0) <= top
    taken = ok[:, None] & (col >= n_blocks[:, None]) & (col < want[:, None])
    at = (top - 1 - (need_start[:, None] + col - n_blocks[:, None])).clamp(0, num - 1)
    table.copy_(torch.where(taken, free[at.long()], torch.where(gone, -1, table)))
    n_blocks.copy_(torch.where(ok, want, n_blocks))
    free_count.copy_(top - torch.where(ok, need, 0).sum())
    return ok


def _run_reserve(s):
    c = s["case"]
    bs = c["bs"]
    if own:
        import tree_speculative_decoding_split_gb300 as st
        slot_map, row_start = st.kv_reserve(s["seq_len"], s["n_new"], s["table"], s["n_blocks"], s["free"], s["free_count"],
                                            bs, s["slots"], dev_status=s["status"])
        st.kv_reserve(s["seq_len"], s["none_new"], s["table"], s["n_blocks"], s["free"], s["free_count"], bs, 0,
                      dev_status=s["status"])
    else:
        ok = _reserve(s["table"], s["n_blocks"], s["free"], s["free_count"], s["seq_len"], s["n_new"], bs)
        ends = torch.cumsum(s["n_new"], 0)
        row_start = torch.cat([torch.zeros_like(ends[:1]), ends]).to(torch.int32)
        row = torch.arange(s["slots"], device=ends.device)
        b = torch.searchsorted(ends, row, right=True).clamp(max=c["batch"] - 1)
        pos = s["seq_len"][b] + row - row_start[b]
        block = s["table"][b, pos // bs].long()
        slot_map = torch.where(ok[b], block * bs + pos % bs, -1)
        _reserve(s["table"], s["n_blocks"], s["free"], s["free_count"], s["seq_len"], s["none_new"], bs)
    return {"slot_map": slot_map, "row_start": row_start, "table": s["table"], "n_blocks": s["n_blocks"], "free": s["free"],
            "free_count": s["free_count"]}


def _append(new, source, is_new, is_old, block, cache, scale):
    """Codes of the blocks [batch][units] that rows are added to: `source` names the row of `new` at
    every place of a block, is_new and is_old say what a place holds afterwards."""
    batch, units, bs = source.shape
    hkv, d = cache.shape[1], cache.shape[3]
    x = torch.where(is_new[..., None, None], new.reshape(-1, hkv, d)[source].float(), 0.0)
    s_new = _scale_of(x.abs().amax(dim=(2, 4)))                     # [batch][units][hkv]
    s_old = scale[block]
    s_all = torch.where(is_old.any(2)[..., None], torch.maximum(s_old, s_new), s_new)
    s_all = torch.where(is_new.any(2)[..., None], s_all, s_old)
    old = cache[block]                                              # [batch][units][hkv][bs][d]
    again = (old.float() * (s_old / s_all)[..., None, None]).to(torch.float8_e4m3fn)
    codes = (x.transpose(2, 3) / s_all[..., None, None]).to(torch.float8_e4m3fn)
    sel_new, sel_old = is_new[:, :, None, :, None], is_old[:, :, None, :, None]
    put = torch.where(sel_new, codes.view(torch.uint8), torch.where(sel_old, again.view(torch.uint8), old.view(torch.uint8)))
    cache.view(torch.uint8)[block.reshape(-1)] = put.reshape(-1, hkv, bs, d)
    scale[block.reshape(-1)] = s_all.reshape(-1, hkv)


def _run_append(s):
    c = s["case"]
    bs, seq_len = c["bs"], s["seq_len"]
    paths = c["form"] == "path"
    if own:
        import tree_speculative_decoding_split_gb300 as st
        if paths:
            new_len = st.kv8_append(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], seq_len,
                                    s["table"], path=s["path"], accept_len=s["accept_len"])
        else:
            new_len = st.kv8_append(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], seq_len,
                                    s["table"], row_start=s["row_start"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"],
                "new_len": new_len}
    count = s["accept_len"] + 1 if paths else s["row_start"][1:] - s["row_start"][:-1]
    unit = torch.arange(s["units"], device=seq_len.device)
    first = seq_len // bs
    logical = first[:, None] + unit                                 # [batch][units]
    pos = logical[..., None] * bs + torch.arange(bs, device=seq_len.device)
    j = pos - seq_len[:, None, None]
    is_new = (j >= 0) & (j < count[:, None, None])
    is_old = (j < 0) & is_new.any(2, keepdim=True)
    if paths:
        row = torch.gather(s["path"], 1, j.clamp(0, s["path"].shape[1] - 1).reshape(c["batch"], -1).long()).reshape(j.shape)
        source = torch.arange(c["batch"], device=row.device)[:, None, None] * c["nodes"] + row
    else:
        source = s["row_start"][:-1, None, None] + j
    source = torch.where(is_new, source, 0).long()
    block = torch.gather(s["table"], 1, logical.clamp(max=s["table"].shape[1] - 1).long()).long()
    block = torch.where(is_new.any(2), block, s["k_cache"].shape[0] - 1)
    _append(s["k_new"], source, is_new, is_old, block, s["k_cache"], s["k_scale"])
    _append(s["v_new"], source, is_new, is_old, block, s["v_cache"], s["v_scale"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"],
            "new_len": seq_len + count}


def _ancestors(parent, n_nodes):
    """[batch][nodes][nodes]: is column j an ancestor of row i, or i itself.  Paths doubled by products of
    the relation with itself; padding sees and is seen by nothing."""
    batch, n = parent.shape
    at = torch.arange(n, device=parent.device)
    real = at < n_nodes[:, None]
    reach = ((parent[:, :, None] == at) | (at[:, None] == at)).float()
    for _ in range(max(1, (n - 1).bit_length())):
        reach = (reach @ reach).clamp(max=1)
    return (reach > 0) & real[:, :, None] & real[:, None, :]


def _gather(cache, scale, table, longest):
    """The values [batch][hkv][longest][d] that every request's first slots stand for."""
    batch, bs = table.shape[0], cache.shape[2]
    blocks = table[:, :_blocks(longest, bs)].clamp(min=0).long()
    x = cache[blocks].float() * scale[blocks][..., None, None]      # [batch][blocks][hkv][bs][d]
    return x.permute(0, 2, 1, 3, 4).reshape(batch, cache.shape[1], -1, cache.shape[3])[:, :, :longest]


def _run_attend(s):
    c = s["case"]
    if own:
        import tree_speculative_decoding_split_gb300 as st
        out, lse = st.tree_attention_kv8(s["q"], s["k_tree"], s["v_tree"], s["k_cache"], s["v_cache"], s["k_scale"],
                                         s["v_scale"], s["seq_len"], s["n_nodes"], s["parent"], s["table"])
        return {"out": out, "lse": lse}
    batch, n, hq, d = s["q"].shape
    hkv, longest = c["hkv"], s["longest"]
    g = hq // hkv
    k = torch.cat([_gather(s["k_cache"], s["k_scale"], s["table"], longest), s["k_tree"].float().transpose(1, 2)], 2)
    q = s["q"].float().view(batch, n, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(batch, hkv, n * g, d) / math.sqrt(d)
    score = q @ k.transpose(2, 3)                                   # [batch][hkv][n g][longest + n]
    prefix = torch.arange(longest, device=q.device) < s["seq_len"][:, None]
    real = torch.arange(n, device=q.device) < s["n_nodes"][:, None]
    seen = torch.cat([prefix[:, None, :] & real[:, :, None], _ancestors(s["parent"], s["n_nodes"])], 2)
    seen = seen[:, None, :, None, :].expand(batch, 1, n, g, longest + n).reshape(batch, 1, n * g, longest + n)
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(3, keepdim=True).clamp_(min=-3e38)
    score.sub_(top).exp_()
    total = score.sum(3, keepdim=True)
    v = torch.cat([_gather(s["v_cache"], s["v_scale"], s["table"], longest), s["v_tree"].float().transpose(1, 2)], 2)
    out = (score @ v) / total.clamp(min=1e-30)
    lse = torch.where(total > 0, top + torch.log(total), 0.0)

    def rows(x):
        return x.view(batch, hkv, n, g, -1).permute(0, 2, 1, 3, 4).reshape(batch, n, hq, -1)

    return {"out": rows(out).to(torch.bfloat16), "lse": rows(lse)[..., 0].contiguous()}


def run(state):
    return {"reserve": _run_reserve, "append": _run_append, "attend": _run_attend}[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    c, bs = case, case["bs"]
    lens = _lens(c)
    if c["op"] == "reserve":
        new = _new_rows(c)
        grown = sum(_blocks(n + m, bs) - _blocks(n, bs) for n, m in zip(lens, new))
        # lengths, counts and held blocks in and out, twice; a block id from the list to the table and back; the slots
        return {"bytes": 2 * 16 * c["batch"] + 2 * 8 * grown + 8 * sum(new) + 4 * (c["batch"] + 1), "flops": 0}
    hkv, d = c["hkv"], c["d"]
    if c["op"] == "append":
        new = _new_rows(c)
        size = 2 if c["dtype"] == "bf16" else 4
        touched = sum(_blocks(n + m, bs) - n // bs for n, m in zip(lens, new) if m)
        return {"bytes": sum(new) * hkv * d * 2 * (size + 1) + touched * (2 * hkv * 4 + 4), "flops": sum(new) * hkv * d * 2 * 2}
    nodes = _nodes(c)
    rows = sum(nodes)
    pairs = sum(m * n for n, m in zip(lens, nodes)) + rows
    cached = sum(lens) * hkv * d * 2 + sum(_blocks(n, bs) for n in lens) * (2 * hkv * 4 + 4)
    return {"bytes": cached + rows * (c["hq"] * (4 * d + 4) + hkv * d * 4 + 4), "flops": 4 * d * c["hq"] * pairs}


# ---- exact values --------------------------------------------------------------------------------

def _pow2(e):
    """2^e in 64 bits, by its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """x (64 bits, |x| <= 448) at the nearest e4m3 value, ties to even: three bits behind the leading one,
    steps of 2^-9 below 2^-6."""
    exponent = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    exponent = torch.where(_pow2(exponent) > x.abs().clamp(min=2.0 ** -6), exponent - 1, exponent)
    step = _pow2(exponent - 3)
    return torch.round(x / step) * step


def _exact_append(case, seed):
    s = prepare(case, seed)
    c, bs = case, case["bs"]
    lens, new = _lens(c), _new_rows(c)
    answer = {"new_len": None}
    start = [sum(new[:b]) for b in range(c["batch"])]
    table = s["table"].tolist()
    for name in ("k", "v"):
        cache, scale = s[name + "_cache"].double(), s[name + "_scale"].double()
        rows = s[name + "_new"]
        for b in range(c["batch"]):
            mine = rows[b][s["path"][b, :new[b]].long()] if c["form"] == "path" else rows[start[b]:start[b] + new[b]]
            done = 0
            while done < new[b]:
                at = lens[b] + done
                held, room = at % bs, min(bs - at % bs, new[b] - done)
                block = table[b][at // bs]
                x = mine[done:done + room].double().transpose(0, 1)                  # [hkv][room][d]
                amax = x.abs().amax(dim=(1, 2))
                e = torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(SCALE_EXP_MIN, SCALE_EXP_MAX)
                e = torch.where(_pow2(e) * E4M3_MAX < amax, e + 1, e)
                e = torch.where(_pow2(e - 1) * E4M3_MAX >= amax, e - 1, e).clamp(SCALE_EXP_MIN, SCALE_EXP_MAX)
                sc = _pow2(e)
                if held:
                    sc = torch.maximum(sc, scale[block])
                    cache[block, :, :held] = _round_e4m3(cache[block, :, :held] * (scale[block] / sc)[:, None, None])
                cache[block, :, held:held + room] = _round_e4m3(x / sc[:, None, None])
                scale[block] = sc
                done += room
        answer[name + "_cache"], answer[name + "_scale"] = cache, scale
    return {k: answer[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale", "new_len")}


def _exact_attend(case, seed):
    s = prepare(case, seed)
    c, bs = case, case["bs"]
    batch, n, hq, d = s["q"].shape
    hkv = c["hkv"]
    g = hq // hkv
    out = torch.zeros((batch, n, hq, d), dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros((batch, n, hq), dtype=torch.float64, device=s["q"].device)
    parents = _trees(c)
    for b, (length, real) in enumerate(zip(_lens(c), _nodes(c))):
        hidden = torch.ones((real, real), dtype=torch.bool)
        for i in range(real):
            j = i
            while j >= 0:
                hidden[i, j] = False
                j = parents[b][j]
        hidden = hidden.to(out.device).repeat_interleave(g, 0)
        blocks = s["table"][b, :_blocks(length, bs)].long()
        for h in range(hkv):
            def whole(cache, scale, tree):
                old = cache[blocks, h].double() * scale[blocks, h].double()[:, None, None]
                return torch.cat([old.reshape(-1, d)[:length], tree[b, :real, h].double()])
            q = s["q"][b, :real, h * g:(h + 1) * g].double().reshape(real * g, d)
            x = (q @ whole(s["k_cache"], s["k_scale"], s["k_tree"]).T) / math.sqrt(d)
            x[:, length:].masked_fill_(hidden, -math.inf)
            norm = torch.logsumexp(x, 1, keepdim=True)
            o = x.sub_(norm).exp_() @ whole(s["v_cache"], s["v_scale"], s["v_tree"])
            out[b, :real, h * g:(h + 1) * g] = o.view(real, g, d)
            lse[b, :real, h * g:(h + 1) * g] = norm.view(real, g)
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "reserve":
        return None
    if case["op"] == "append":
        return _exact_append(case, seed)
    return _exact_attend(case, seed)
