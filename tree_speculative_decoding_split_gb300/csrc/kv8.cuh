// Device helpers shared by the attention kernels over the 8-bit paged cache.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.cuh"

namespace spectree {

constexpr int kKv8Splits = 32;  // per request at most (the merge holds one per lane)

constexpr float kKv8MinScale = 5.4210108624275222e-20f;  // 2^-64
constexpr float kKv8MaxScale = 1.329227995784916e36f;    // 2^120

__device__ __forceinline__ float kv8_clamp_scale(float s) { return fminf(fmaxf(s, kKv8MinScale), kKv8MaxScale); }

// Index of row (node row / G, head h G + row % G) of request b in [B][N][Hq].
__device__ __forceinline__ int kv8_node(const Kv8AttnParams& p, int row) {
  return p.G == 1 ? row : (int)__umulhi((uint32_t)row, p.g_magic);
}
__device__ __forceinline__ size_t kv8_row(const Kv8AttnParams& p, int b, int h, int row) {
  const int i = kv8_node(p, row);
  return ((size_t)b * p.N + i) * p.Hq + h * p.G + (row - i * p.G);
}

// Verdict on request b from its counts alone; `len` is the prefix length every kernel goes on with.
__device__ __forceinline__ int kv8_verdict(const Kv8AttnParams& p, long long* len, int* n) {
  int err = 0;
  if (*n < 1 || *n > p.N) {
    err = SPEC_ERR_BAD_TREE;
    *n = 0;
  }
  if (*len < 0 || *len > p.L_cap) {
    if (!err) err = SPEC_ERR_CAPACITY;
    *len = 0;
  }
  return err;
}

// A CTA's work: node rows of tile `rt` of head h of request b, over split `split` of the n that the request's prefix
// is cut into.
struct Kv8Work {
  int b, h, rt, split, n;
  int steps;      // steps (2^unit_shift keys) per split
  int nodes;
  int err;
  long long L;    // prefix length, 0 when it is refused
  size_t part;    // first row of the CTA's partial results
};

// How prefixes are cut, in whole steps of 2^unit_shift keys.  The grid holds `base` units of Hkv * n_rt CTAs for
// every request, whose CTAs run over row tiles first, then splits, then heads (with heads before splits, decoding
// for 32 requests took 62-66 us instead of 56), and behind them `extra` units for the splits past `base`, in the
// requests' order.  CTAs without a split end at once.
// The lengths are on the device, so every CTA works out the same cut from them:
//   few-rows kernel: `base` splits, more where one of them would be longer than 1.5 even shares of all the steps.  Its
//   CTAs share the memory's bandwidth, so that it only has to keep one long request from running on alone.  Splits
//   past base are then no more than slots / (1.5 * heads) units.  (31 requests of 2K and one of 128K take a tenth less
//   than at two shares; at one share the 32 requests of 2K to 6K take 68 us instead of 57.)
//   tensor-core kernel, where a CTA's speed is its own: c steps at most, the one of ceil(longest / k), for 16 numbers k
//   from 1 to 32, that fits the units with the least cost.  With a split's work w = c + fixed, the whole work W and
//   `slots` CTAs at once, the cost is the lesser of two upper bounds, whole rounds of CTAs times w and
//   (W - w) / slots + w.  One warp evaluates it, two lanes per k.  Over 128 requests c = ceil(all steps / extra)
//   instead, which always fits.
// Against equal splits per request, fixed by the host from the batch's size: 8 trees of 127 nodes at ragged lengths
// 103 -> 66 us, 4 of 255 nodes at up to 128K 2112 -> 1990, 32 requests' tokens at 2K to 6K 56 -> 57.5.
__device__ __forceinline__ int kv8_steps(const Kv8AttnParams& p, int len) {
  return len > 0 && len <= p.L_cap ? (int)(((long long)len + (1 << p.unit_shift) - 1) >> p.unit_shift) : 0;
}
__device__ __forceinline__ int kv8_cut(const Kv8AttnParams& p) {
  const int least = 256 >> p.unit_shift, lane = threadIdx.x & 31;
  float total = 0.f;
  int longest = 1;
#pragma unroll 4
  for (int i = lane; i < p.B; i += 32) {
    const int steps = kv8_steps(p, p.prefix_len[i]);
    total += (float)steps;
    longest = max(longest, steps);
  }
  total = warp_sum(total);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (p.unit_shift == 6 || p.B > 128 || longest > 65535) {
    const float share = p.unit_shift == 6 ? 1.5f * total * (float)(p.Hkv * p.n_rt) * p.inv_slots : total / (float)p.extra;
    return max(least, (int)fminf(ceilf(share * 1.0001f), 1e9f));
  }
  // two lanes per candidate, each over every other request
  const int nth = lane >> 1, k = nth < 8 ? nth + 1 : nth < 12 ? 2 * nth - 6 : 4 * nth - 28;
  const int c = max(least, (longest + k - 1) / k);
  const float rc = __fdividef(1.f, (float)c);
  int units = 0, past = 0;
  for (int i0 = 0; i0 < p.B; i0 += 32) {
    const float steps = (float)(i0 + lane < p.B ? kv8_steps(p, p.prefix_len[i0 + lane]) : 0) - 0.5f;
    const int here = min(32, p.B - i0);
#pragma unroll 4
    for (int i = 0; i < here; i += 2) {
      // max(1, ceil(steps / c)) - 1, exactly: (steps - 1/2) / c keeps 1 / (2 c) >= 2^-17 from every whole number,
      // and below 33 its error is less
      const int n = (int)(__shfl_sync(0xffffffffu, steps, i + (lane & 1)) * rc);
      units += n;
      past += max(0, n + 1 - p.base);  // (a lane past the last request holds -1/2: none)
    }
  }
  units += __shfl_xor_sync(0xffffffffu, units, 1) + p.B;
  past += __shfl_xor_sync(0xffffffffu, past, 1);
  const float heads = (float)(p.Hkv * p.n_rt), w = (float)(c + p.fixed_steps);
  const float work = heads * (total + (float)units * (float)p.fixed_steps) * p.inv_slots;
  float cost = fminf(ceilf((float)units * heads * p.inv_slots) * w, work + w * (1.f - p.inv_slots));
  if (units > p.B) cost += 3.f;  // the merge
  const bool fits = k == 1 || past <= p.extra;
  const uint32_t key = fits ? (__float_as_uint(cost) & ~31u) | (uint32_t)lane : 0xffffffffu;
  return __shfl_sync(0xffffffffu, c, (int)(__reduce_min_sync(0xffffffffu, key) & 31u));
}
__device__ __forceinline__ int kv8_splits(const Kv8AttnParams& p, int steps, int c) {
  if (p.unit_shift == 6) c = max(256 >> 6, min((steps + p.base - 1) / p.base, c));
  c = max(c, (steps + kKv8Splits - 1) / kKv8Splits);
  return steps <= c ? 1 : (steps + c - 1) / c;
}

// What is known of a CTA's work before any length is read: all but the lengths for one of the `base` units of a
// request, nothing (b < 0) for one behind them.
__device__ __forceinline__ Kv8Work kv8_own(const Kv8AttnParams& p) {
  const int per_req = p.base * p.Hkv * p.n_rt, per_head = p.base * p.n_rt;
  Kv8Work w;
  int idx = blockIdx.x;
  w.b = idx / per_req;
  idx -= w.b * per_req;
  w.h = idx / per_head;
  idx -= w.h * per_head;
  w.split = idx / p.n_rt;
  w.rt = idx - w.split * p.n_rt;
  w.part = (size_t)blockIdx.x * p.rows_cta;
  if (w.b >= p.B) w.b = -1;
  return w;
}
// The whole of it, for a warp of the CTA; b < 0 when there is none.
__device__ __forceinline__ Kv8Work kv8_begin(const Kv8AttnParams& p, Kv8Work w) {
  const int lane = threadIdx.x & 31;
  const bool own = w.b >= 0;
  int c = 0x3fffffff, first = 0;
  w.L = own ? p.prefix_len[w.b] : 0;
  w.nodes = own ? p.n_nodes[w.b] : 0;
  // (a request of 256 keys or fewer has one split whatever the others are)
  if ((p.extra > 0 || (p.unit_shift == 7 && p.base > 1)) && !(own && w.L <= 256)) {
    c = kv8_cut(p);
    if (!own) {
      const int heads = p.Hkv * p.n_rt, idx = blockIdx.x - p.B * p.base * heads, unit = idx / heads;
      w.h = (idx - unit * heads) / p.n_rt;
      w.rt = idx - unit * heads - w.h * p.n_rt;
      int before = 0;  // extra units of the requests before
#pragma unroll 1
      for (int i0 = 0; i0 < p.B && w.b < 0; i0 += 32) {
        const int mine = i0 + lane < p.B ? max(0, kv8_splits(p, kv8_steps(p, p.prefix_len[i0 + lane]), c) - p.base) : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += up;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + incl > unit);
        if (hit) {
          const int src = __ffs(hit) - 1;
          w.b = i0 + src;
          first = before + __shfl_sync(0xffffffffu, incl - mine, src);
          w.split = p.base + unit - first;
        } else {
          before += __shfl_sync(0xffffffffu, incl, 31);
        }
      }
      if (w.b < 0) return w;
      w.L = p.prefix_len[w.b];
      w.nodes = p.n_nodes[w.b];
    }
  }
  w.err = kv8_verdict(p, &w.L, &w.nodes);
  const int total = (int)((w.L + (1 << p.unit_shift) - 1) >> p.unit_shift);
  w.n = kv8_splits(p, total, c);
  w.steps = w.n == 1 ? total : (total + w.n - 1) / w.n;
  // for the merge, by the first CTA that knows both
  if (p.used && threadIdx.x == 0 && w.h == 0 && w.rt == 0 && w.split == (w.n > p.base ? p.base : 0))
    p.used[w.b] = make_int2(w.n, first);
  if (w.split >= w.n) w.b = -1;
  return w;
}
// First row of the partial results of split s of a request, for the row tile's CTA of head h.
__device__ __forceinline__ size_t kv8_part(const Kv8AttnParams& p, int b, int h, int rt, int s, int first) {
  const int heads = p.Hkv * p.n_rt;
  const size_t cta = s < p.base ? (size_t)b * p.base * heads + (h * p.base + s) * p.n_rt + rt
                                : (size_t)(p.B * p.base + first + s - p.base) * heads + h * p.n_rt + rt;
  return cta * p.rows_cta;
}

}  // namespace spectree
