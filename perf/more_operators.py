"""Cases, plain forms and exact values of the operators that take a prompt to the cache.

Five operators that run one after another when prompts are admitted (and, the first two, before every
attention call of a round):

  positions  the position of every packed prompt row, or of every node of the draft trees (its depth
             below the request's root)
  rope       rotary positions of query and key rows: pairs of channels turned by an angle that is the
             position times a frequency, kept as a 64-bit fraction of a turn
  attend     causal attention over packed prompts with grouped heads, and its log-sum-exp
  weights    the attention weight that every key gets from a prompt's last queries, summed over them and
             over the heads that share the key
  keep       the rows with the largest weights, per request and KV head, up to a budget: the ones that the
             cache is to hold

``run`` computes them with elementary torch operations, or, where ``own`` is true, with the
framework's kernels.
"""

import math
import random

import torch

own = False


# ---- sizes ---------------------------------------------------------------------------------------

def _spread(lo, hi, count):
    """`count` lengths from lo to hi, evenly spaced, the long ones not all at one end."""
    if count == 1:
        return [hi]
    even = [lo + (hi - lo) * i // (count - 1) for i in range(count)]
    return even[::2] + even[1::2][::-1]


def _lens(c):
    return _spread(c["lo"], c["hi"], c["batch"])


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _nodes(c):
    n = c["nodes"]
    return [n - (3 * b) % (n // 4 + 1) for b in range(c["batch"])]


def _trees(c):
    """Parent arrays [batch][nodes] (-1 for the root and for padding), numbered breadth-first."""
    rng = random.Random(c["nodes"] * 1013 + c["batch"])
    rows = []
    for n in _nodes(c):
        par = [-1] + [max(0, (i - 1) // 2 - rng.randrange(0, 2)) for i in range(1, n)]
        rows.append(par + [-1] * (c["nodes"] - n))
    return rows


def _rope_rows(c):
    return c["batch"] * c["nodes"] if c["form"] == "tree" else sum(_lens(c))


def listed():
    return [
        # nodes of 32 draft trees, once per round
        {"name": "positions_tree_b32", "op": "positions", "form": "tree", "batch": 32, "nodes": 63, "far": 4096},
        # the rows of 512 prompts admitted at once behind shared prefixes, a million of them
        {"name": "positions_admit_b512", "op": "positions", "form": "rows", "batch": 512, "lo": 1, "hi": 4095, "far": 2048},
        # one new token of one request, before a layer's attention: latency
        {"name": "rope_token_b1", "op": "rope", "form": "tree", "dtype": "bf16", "batch": 1, "nodes": 1, "far": 131072, "hq": 32,
         "hkv": 8, "d": 128, "rot": 128, "layout": "half", "fused": True},
        # the 63-node trees of a batch of 32
        {"name": "rope_tree_b32", "op": "rope", "form": "tree", "dtype": "bf16", "batch": 32, "nodes": 63, "far": 4096, "hq": 32,
         "hkv": 8, "d": 128, "rot": 128, "layout": "half", "fused": True},
        # prompts of 4K to 16K tokens in float32, neighbouring channels paired, half of each head turned
        {"name": "rope_prompt_f32", "op": "rope", "form": "rows", "dtype": "f32", "batch": 4, "lo": 4096, "hi": 16384, "far": 3000,
         "hq": 16, "hkv": 8, "d": 64, "rot": 32, "layout": "interleaved", "fused": False},
        # one prompt of 500 tokens: latency
        {"name": "attend_b1_l500", "op": "attend", "batch": 1, "lo": 500, "hi": 500, "hq": 32, "hkv": 8, "d": 128},
        # a packed batch of 48 short and middling prompts, heads of 64
        {"name": "attend_b48_d64", "op": "attend", "batch": 48, "lo": 1, "hi": 1800, "hq": 16, "hkv": 8, "d": 64},
        # one long prompt of 64 query heads on 8
        {"name": "attend_b1_l16k", "op": "attend", "batch": 1, "lo": 16384, "hi": 16384, "hq": 64, "hkv": 8, "d": 128},
        # the last 64 tokens of a prompt of 16K look back over it
        {"name": "weights_b1_l16k", "op": "weights", "batch": 1, "lo": 16384, "hi": 16384, "window": 64, "hq": 32, "hkv": 8, "d": 128},
        # the last 37 of eight prompts of 0.5K to 32K tokens, 64 query heads on 8
        {"name": "weights_b8_ragged", "op": "weights", "batch": 8, "lo": 512, "hi": 32768, "window": 37, "hq": 64, "hkv": 8, "d": 128},
        # a budget of 1024 rows for 16 prompts of up to 8K, heads of 64 from float32 projections
        {"name": "keep_b16_f32", "op": "keep", "dtype": "f32", "batch": 16, "lo": 300, "hi": 8192, "budget": 1024, "first": 4,
         "last": 64, "hkv": 8, "d": 64, "fused": False},
        # 4096 rows of a prompt of 128K
        {"name": "keep_b1_l128k", "op": "keep", "dtype": "bf16", "batch": 1, "lo": 131072, "hi": 131072, "budget": 4096, "first": 4,
         "last": 64, "hkv": 8, "d": 128, "fused": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["positions", "rope", "rope", "attend", "attend", "attend", "weights", "weights", "keep", "keep"])
    if op == "positions":
        batch = _log(rng, 1, 512)
        if rng.random() < 0.5:
            return {"op": op, "form": "tree", "batch": batch, "nodes": _log(rng, 1, 255), "far": _log(rng, 1, 131072)}
        hi = _log(rng, 1, (1 << 20) // batch)
        return {"op": op, "form": "rows", "batch": batch, "lo": rng.randrange(0, hi + 1), "hi": hi, "far": _log(rng, 1, 131072)}
    d, hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    if op == "rope":
        c = {"op": op, "form": rng.choice(["tree", "rows"]), "dtype": rng.choice(["bf16", "bf16", "f32"]), "batch": _log(rng, 1, 32),
             "far": _log(rng, 1, 131072), "hq": hq, "hkv": hkv, "d": d, "rot": 16 * rng.randrange(1, d // 16 + 1),
             "layout": rng.choice(["half", "interleaved"]), "fused": rng.random() < 0.5}
        if c["form"] == "tree":
            c["nodes"] = 1 if rng.random() < 0.4 else _log(rng, 2, 255)
        else:
            c["hi"] = _log(rng, 1, 16384 // c["batch"])
            c["lo"] = rng.randrange(0, c["hi"] + 1)
        return c
    if op == "attend":
        hi = _log(rng, 1, 16384)
        batch = _log(rng, 1, max(1, min(48, (1 << 32) // (hi * hi * hq))))
        return {"op": op, "batch": batch, "lo": rng.randrange(0, hi + 1), "hi": hi, "hq": hq, "hkv": hkv, "d": d}
    hi = _log(rng, 2, 32768 if op == "weights" else 131072)
    batch = _log(rng, 1, max(1, min(16, 131072 // hi)))
    lo = rng.randrange(0, hi + 1)
    if op == "weights":
        return {"op": op, "batch": batch, "lo": lo, "hi": hi, "window": _log(rng, 1, 128), "hq": hq, "hkv": hkv, "d": d}
    budget = _log(rng, 1, 4096)
    first = rng.randrange(0, min(8, budget) + 1)
    return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "batch": batch, "lo": lo, "hi": hi, "budget": budget, "first": first,
            "last": rng.randrange(0, min(64, budget - first) + 1), "hkv": hkv, "d": d, "fused": rng.random() < 0.5}


# ---- inputs --------------------------------------------------------------------------------------

def _ints(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _rows(gen, rows, heads, d, dev):
    """Q, K or V rows [rows, heads, d] as a layer makes them: unit variance, each head at its own
    magnitude, a few channels several times the others."""
    x = torch.randn((rows, heads, d), generator=gen, device=dev)
    channel = torch.ones(d, device=dev)
    channel[::23] = 4.0
    head = 0.5 + torch.arange(heads, device=dev, dtype=torch.float32)[:, None] / heads
    return x.mul_(head * channel)


def _qkv(gen, rows, c, dev, fused, dtype):
    """Query, key and value rows; fused: views of one projection's rows."""
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    x = torch.cat([torch.randn((rows, hq, d), generator=gen, device=dev), _rows(gen, rows, hkv, d, dev), _rows(gen, rows, hkv, d, dev)],
                  1).to(dtype)
    parts = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return parts if fused else tuple(p.contiguous() for p in parts)


def _far(c, seed):
    """Where every request's rows begin."""
    rng = random.Random(seed * 7919 + c["batch"])
    return [rng.randrange(0, c["far"] + 1) for _ in range(c["batch"])]


def _turns(rot, dev):
    """Frequencies theta^(-2i/rot), theta = 500000, in 2^-64 turns per position."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    return torch.floor(500000.0 ** (-2.0 * i / rot) / (2.0 * math.pi) * 2.0 ** 64).to(torch.int64).to(dev)


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("positions", "rope"):
        far = _far(c, seed)
        if c["op"] == "positions":
            s["pos0"] = _ints(far, dev)
            if c["form"] == "tree":
                s["parent"], s["n_nodes"] = _ints(_trees(c), dev), _ints(_nodes(c), dev)
            else:
                starts = _starts(_lens(c))
                s["row_start"], s["n_rows"] = _ints(starts, dev), starts[-1]
            return s
        rows = _rope_rows(c)
        s["q"], s["k"], _ = _qkv(gen, rows, c, dev, c["fused"], _dtype(c))
        if c["form"] == "tree":
            shape = (c["batch"], c["nodes"])
            s["q"], s["k"] = s["q"].unflatten(0, shape), s["k"].unflatten(0, shape)
            depth = [[(i + 1).bit_length() - 1 for i in range(c["nodes"])] for _ in far]
            s["positions"] = _ints([[f + e for e in row] for f, row in zip(far, depth)], dev)
        else:
            pos = [torch.arange(f, f + n, dtype=torch.int32) for f, n in zip(far, _lens(c))]
            s["positions"] = torch.cat(pos).to(dev)
        s["turns"] = _turns(c["rot"], dev)
        return s
    lens = _lens(c)
    starts = _starts(lens)
    rows = starts[-1]
    s["row_start"], s["longest"] = _ints(starts, dev), max(lens)
    if c["op"] == "keep":
        both = torch.cat([_rows(gen, rows, c["hkv"], c["d"], dev), _rows(gen, rows, c["hkv"], c["d"], dev)], 1).to(_dtype(c))
        s["k"], s["v"] = both[:, :c["hkv"]], both[:, c["hkv"]:]
        if not c["fused"]:
            s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
        # weights spread over several magnitudes, some of them 0
        w = torch.randn((c["hkv"], rows), generator=gen, device=dev).mul_(2.0).exp_()
        s["weight"] = w.masked_fill_(torch.rand((c["hkv"], rows), generator=gen, device=dev) < 0.1, 0.0)
        s["rows_out"] = sum(min(n, c["budget"]) for n in lens)
        return s
    s["q"], s["k"], s["v"] = _qkv(gen, rows, c, dev, True, torch.bfloat16)
    if c["op"] == "weights":
        # the log-sum-exp that the attention over these prompts left
        s["lse"] = torch.zeros((rows, c["hq"]), dtype=torch.float32, device=dev)
        for at, n in zip(starts, lens):
            w = min(c["window"], n)
            if w == 0:
                continue
            g = c["hq"] // c["hkv"]
            q = s["q"][at + n - w:at + n].float().reshape(w, c["hkv"], g, c["d"]).permute(1, 2, 0, 3)
            x = (q @ s["k"][at:at + n].float().permute(1, 2, 0)[:, None]) / math.sqrt(c["d"])
            late = torch.arange(n, device=dev) > torch.arange(n - w, n, device=dev)[:, None]
            s["lse"][at + n - w:at + n] = torch.logsumexp(x.masked_fill_(late, -math.inf), 3).permute(2, 0, 1).reshape(w, -1)
    return s


# ---- the plain forms -----------------------------------------------------------------------------

def _run_positions(s):
    c = s["case"]
    if own:
        import tree_speculative_decoding_split_gb300 as st
        if c["form"] == "tree":
            return {"positions": st.rope_positions(s["pos0"], parent=s["parent"], n_nodes=s["n_nodes"])}
        return {"positions": st.rope_positions(s["pos0"], row_start=s["row_start"], n_rows=s["n_rows"])}
    if c["form"] == "tree":
        batch, n = s["parent"].shape
        at = torch.arange(n, device=s["parent"].device)
        reach = ((s["parent"][:, :, None] == at) | (at[:, None] == at)).float()
        for _ in range(max(1, (n - 1).bit_length())):   # paths doubled by products of the relation with itself
            reach = (reach @ reach).clamp(max=1)
        depth = (reach.sum(2) - 1).to(torch.int32)
        return {"positions": torch.where(at < s["n_nodes"][:, None], s["pos0"][:, None] + depth, -1)}
    row = torch.arange(s["n_rows"], device=s["pos0"].device, dtype=torch.int32)
    b = torch.searchsorted(s["row_start"][1:], row, right=True)
    return {"positions": s["pos0"][b] + row - s["row_start"][b]}


def _turn(x, cos, sin, rot, layout):
    head = x[..., :rot].float()
    if layout == "half":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([head.to(x.dtype), x[..., rot:]], -1)


def _run_rope(s):
    c = s["case"]
    if own:
        import tree_speculative_decoding_split_gb300 as st
        q, k = st.rope(s["q"], s["k"], s["positions"], s["turns"], layout=c["layout"])
        return {"q": q, "k": k}
    angle = s["positions"].double()[..., None] * s["turns"].double() * (2.0 * math.pi / 2.0 ** 64)
    cos, sin = torch.cos(angle).float()[..., None, :], torch.sin(angle).float()[..., None, :]
    return {"q": _turn(s["q"], cos, sin, c["rot"], c["layout"]), "k": _turn(s["k"], cos, sin, c["rot"], c["layout"])}


def _padded(s, longest):
    """(row of every request's place [batch][longest], is there a row)."""
    j = torch.arange(longest, device=s["row_start"].device)
    n = s["row_start"][1:] - s["row_start"][:-1]
    there = j < n[:, None]
    return torch.where(there, s["row_start"][:-1, None] + j, 0).long(), there


def _run_attend(s):
    c = s["case"]
    if own:
        import tree_speculative_decoding_split_gb300 as st
        out, lse = st.prompt_attention(s["q"], s["k"], s["v"], s["row_start"])
        return {"out": out, "lse": lse}
    rows, hq, d = s["q"].shape
    hkv, longest = c["hkv"], s["longest"]
    g = hq // hkv
    at, there = _padded(s, longest)
    batch = at.shape[0]
    q = (s["q"][at].float() / math.sqrt(d)).view(batch, longest, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, g * longest, d)
    k, v = s["k"][at].float().permute(0, 2, 3, 1), s["v"][at].float().transpose(1, 2)
    score = (q @ k).view(batch, hkv, g, longest, longest)
    place = torch.arange(longest, device=q.device)
    score.masked_fill_(place > place[:, None], -math.inf)
    top = score.amax(4, keepdim=True)
    score.sub_(top).exp_()
    total = score.sum(4, keepdim=True)
    out = (score.view(batch, hkv, g * longest, longest) @ v).view(batch, hkv, g, longest, d) / total
    lse = (top + torch.log(total))[..., 0]
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, longest, hq, d)[there].to(torch.bfloat16)
    lse = lse.permute(0, 3, 1, 2).reshape(batch, longest, hq)[there]
    return {"out": out, "lse": lse}


def _run_weights(s):
    c = s["case"]
    if own:
        import tree_speculative_decoding_split_gb300 as st
        return {"weight": st.prompt_key_weights(s["q"], s["k"], s["lse"], s["row_start"], c["window"])}
    rows, hq, d = s["q"].shape
    hkv, longest, w = c["hkv"], s["longest"], c["window"]
    g = hq // hkv
    at, there = _padded(s, longest)
    batch = at.shape[0]
    n = s["row_start"][1:] - s["row_start"][:-1]
    i = n[:, None] - w + torch.arange(w, device=at.device)             # the window's places [batch][w]
    at_q = torch.where(i >= 0, s["row_start"][:-1, None] + i, 0).long()
    q = (s["q"][at_q].float() / math.sqrt(d)).view(batch, w, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, g * w, d)
    k = s["k"][at].float().permute(0, 2, 3, 1)
    score = (q @ k).view(batch, hkv, g, w, longest)
    lse = s["lse"][at_q].view(batch, w, hkv, g).permute(0, 2, 3, 1)
    seen = (torch.arange(longest, device=q.device) <= i[..., None]) & there[:, None, :] & (i >= 0)[..., None]
    score.sub_(lse[..., None]).masked_fill_(~seen[:, None, None], -math.inf).exp_()
    return {"weight": score.sum((2, 3)).transpose(1, 2)[there].t().contiguous()}


def _run_keep(s):
    c = s["case"]
    if own:
        import tree_speculative_decoding_split_gb300 as st
        k, v, index, keep_start, n_keep = st.kv_keep(s["k"], s["v"], s["weight"], s["row_start"], c["budget"], first=c["first"],
                                                     last=c["last"], rows_out=s["rows_out"])
        return {"k": k, "v": v, "index": index, "keep_start": keep_start, "n_keep": n_keep}
    hkv, longest, budget = c["hkv"], s["longest"], c["budget"]
    at, there = _padded(s, longest)
    n = s["row_start"][1:] - s["row_start"][:-1]
    n_keep = n.clamp(max=budget)
    place = torch.arange(longest, device=at.device)
    held = there & ((place < c["first"]) | (place >= n[:, None] - c["last"]))
    rank = torch.where(held, 2, torch.where(there, 1, 0))[:, None, :].expand(-1, hkv, -1)      # kept anyway, a row, none
    weight = s["weight"][:, at].permute(1, 0, 2)                                               # [batch][hkv][longest]
    order = torch.sort(weight, dim=2, descending=True, stable=True).indices
    order = torch.gather(order, 2, torch.sort(torch.gather(rank, 2, order), dim=2, descending=True, stable=True).indices)
    width = min(budget, longest)
    slot = torch.arange(width, device=at.device)
    there_out = slot < n_keep[:, None]
    best = torch.where(there_out[:, None, :], order[:, :, :width], longest)
    best = torch.sort(best, dim=2).values                                                      # back in the prompt's order
    index = best.transpose(1, 2)[there_out]                                                    # [rows_out][hkv]
    first_row = s["row_start"][:-1, None].expand(-1, width)[there_out]
    head = torch.arange(hkv, device=at.device)
    source = first_row[:, None] + index
    ends = torch.cumsum(n_keep, 0)
    keep_start = torch.cat([torch.zeros_like(ends[:1]), ends]).to(torch.int32)
    return {"k": s["k"][source, head], "v": s["v"][source, head], "index": index.to(torch.int32), "keep_start": keep_start, "n_keep": n_keep}


def run(state):
    return {"positions": _run_positions, "rope": _run_rope, "attend": _run_attend, "weights": _run_weights,
            "keep": _run_keep}[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "positions":
        if c["form"] == "tree":
            return {"bytes": 8 * c["batch"] * (c["nodes"] + 1), "flops": 0}
        return {"bytes": 4 * sum(_lens(c)) + 8 * c["batch"] + 4, "flops": 0}
    size = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "rope":
        rows = _rope_rows(c)
        return {"bytes": rows * ((c["hq"] + c["hkv"]) * c["d"] * size * 2 + 4) + 4 * c["rot"],
                "flops": 3 * rows * (c["hq"] + c["hkv"]) * c["rot"]}
    lens = _lens(c)
    hkv, d = c["hkv"], c["d"]
    if c["op"] == "attend":
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": sum(lens) * (c["hq"] * (4 * d + 4) + hkv * 4 * d) + 4 * len(lens) + 4, "flops": 4 * d * c["hq"] * pairs}
    if c["op"] == "weights":
        w = [min(c["window"], n) for n in lens]
        pairs = sum(m * n - m * (m - 1) // 2 for m, n in zip(w, lens))
        return {"bytes": sum(lens) * hkv * (2 * d + 4) + sum(w) * c["hq"] * (2 * d + 4) + 4 * len(lens) + 4,
                "flops": 2 * d * c["hq"] * pairs}
    kept = sum(min(n, c["budget"]) for n in lens)
    chosen = sum(n for n in lens if n > c["budget"])   # weights of prompts within the budget need not be read
    return {"bytes": chosen * hkv * 4 + kept * hkv * (4 * d * size + 4) + 12 * len(lens) + 8, "flops": 0}


# ---- exact values --------------------------------------------------------------------------------

def _exact_rope(case, seed):
    s = prepare(case, seed)
    c, rot = case, case["rot"]
    # the fraction of a turn: the product modulo 2^64, as 64-bit integers wrap
    turn = (s["positions"].long()[..., None] * s["turns"]).double() * 2.0 ** -64
    z = torch.polar(torch.ones_like(turn), turn * (2.0 * math.pi))[..., None, :]
    answer = {}
    for name in ("q", "k"):
        x = s[name].double()
        i = torch.arange(rot // 2, device=x.device)
        lo, hi = (i, i + rot // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)
        y = torch.complex(x[..., lo], x[..., hi]) * z
        x[..., lo], x[..., hi] = y.real, y.imag
        answer[name] = x
    return answer


def _exact_attend(case, seed):
    s = prepare(case, seed)
    c = case
    rows, hq, d = s["q"].shape
    g = hq // c["hkv"]
    dev = s["q"].device
    out = torch.zeros((rows, hq, d), dtype=torch.float64, device=dev)
    lse = torch.zeros((rows, hq), dtype=torch.float64, device=dev)
    lens = _lens(c)
    for at, n in zip(_starts(lens), lens):
        for h in range(hq):
            k, v = s["k"][at:at + n, h // g].double(), s["v"][at:at + n, h // g].double()
            for i in range(0, n, 4096):
                top = min(n, i + 4096)
                x = (s["q"][at + i:at + top, h].double() @ k[:top].T) / math.sqrt(d)
                x.masked_fill_(torch.ones_like(x, dtype=torch.bool).triu_(i + 1), -math.inf)
                norm = torch.logsumexp(x, 1, keepdim=True)
                out[at + i:at + top, h] = x.sub_(norm).exp_() @ v[:top]
                lse[at + i:at + top, h] = norm[:, 0]
    return {"out": out[:sum(lens)], "lse": lse[:sum(lens)]}


def _exact_weights(case, seed):
    s = prepare(case, seed)
    c = case
    rows, hq, d = s["q"].shape
    g = hq // c["hkv"]
    weight = torch.zeros((c["hkv"], rows), dtype=torch.float64, device=s["q"].device)
    lens = _lens(c)
    for at, n in zip(_starts(lens), lens):
        for i in range(max(0, n - c["window"]), n):
            x = torch.einsum("hgd,jhd->hgj", s["q"][at + i].double().view(c["hkv"], g, d), s["k"][at:at + i + 1].double()) / math.sqrt(d)
            weight[:, at:at + i + 1] += torch.exp(x - s["lse"][at + i].double().view(c["hkv"], g, 1)).sum(1)
    return {"weight": weight[:, :sum(lens)]}


def exact(case, seed):
    if case["op"] in ("positions", "keep"):
        return None
    if case["op"] == "attend" and case["hq"] * case["batch"] * case["hi"] ** 2 > 1 << 34:
        return None
    return {"rope": _exact_rope, "attend": _exact_attend, "weights": _exact_weights}[case["op"]](case, seed)
