"""8-bit paged KV cache: e4m3 codes with a scale per block and KV head, block tables from a stack of
free blocks, and the appending of rows (fp64, one step at a time).

TEST INFRASTRUCTURE ONLY (see the package docstring).

e4m3: one sign, four exponent bits (bias 7), three fraction bits; exponent field 0 holds multiples of
2^-9; the code 0x7f (0xff) is NaN and there is no infinity, so the largest value is 1.75 * 2^8 = 448.
"""

import numpy as np


def _decode_table():
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if c & 127 == 127:
            v = np.nan
        out[c] = -v if c & 128 else v
    return out


E4M3 = _decode_table()


def e4m3_encode(x):
    """Codes nearest to x (ties to the even code), NaN to 0x7f, what passes 448 to 448."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(x), 448.0)
    values = E4M3[:127]
    hi = np.clip(np.searchsorted(values, mag), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = mag - values[lo], values[hi] - mag
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def block_scale(x):
    """The smallest 2^e, -64 <= e <= 120, with max |x| <= 448 * 2^e; infinities and NaN are left out."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    x = x[np.isfinite(x)]
    top = x.max() if x.size else 0.0
    e = -64
    while e < 120 and top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append_rows(rows, cache, scale, start, table, bs):
    """Append rows [n][Hkv][d] of one request at logical slot ``start``, in place: cache uint8
    [num_blocks][Hkv][bs][d], scale float64 [num_blocks][Hkv], table the request's blocks."""
    n = rows.shape[0]
    done = 0
    while done < n:
        held = (start + done) % bs
        take = min(bs - held, n - done)
        blk = int(table[(start + done) // bs])
        for h in range(rows.shape[1]):
            x = rows[done: done + take, h]
            s_new = block_scale(x)
            s = s_new
            if held:
                old = scale[blk, h]
                s = max(old, s_new)
                if s > old:
                    cache[blk, h, :held] = e4m3_encode(E4M3[cache[blk, h, :held]] * (old / s))
            cache[blk, h, held: held + take] = e4m3_encode(x / s)
            scale[blk, h] = s
        done += take


def gather_kv8(cache, scale, table, bs, length):
    """Values [Hkv][length][d] that a request's first ``length`` slots stand for."""
    Hkv, d = cache.shape[1], cache.shape[3]
    out = np.zeros((Hkv, length, d))
    for s in range(length):
        blk = int(table[s // bs])
        out[:, s] = E4M3[cache[blk, :, s % bs]] * scale[blk][:, None]
    return out


def reserve(seq_len, n_new, table, free, bs):
    """Block tables for seq_len + n_new slots.  ``table`` is a list of lists (a request's blocks), ``free``
    a list with the top of the stack at its end; both are changed.  Returns (slots per request or None
    for one that is not served)."""
    want = [-(-(int(a) + int(b)) // bs) for a, b in zip(seq_len, n_new)]
    given = []
    for b, w in enumerate(want):
        given += table[b][w:]
        table[b] = table[b][:w]
    free += given[::-1]
    full = False
    slots = []
    budget = len(free)
    asked = 0
    for b, w in enumerate(want):
        need = w - len(table[b])
        asked += need
        full = asked > budget and need > 0
        if not full:
            for _ in range(need):
                table[b].append(free.pop())
        covered = len(table[b]) * bs >= int(seq_len[b]) + int(n_new[b])
        slots.append([table[b][s // bs] * bs + s % bs for s in range(int(seq_len[b]), int(seq_len[b]) + int(n_new[b]))]
                     if covered else None)
    return slots
