// K8: rows into the 8-bit paged cache (spec_kv8_append).
//
// A block of one KV head is bs x d elements with one scale s = 2^e, e the smallest with
// max |x| <= 448 * 2^e; a code is e4m3(x / s).  Both steps need all of a block's new rows, which fit the
// registers of one group of threads: the group loads them once, reduces |x| to the
// maximum, and converts what it holds.  So the rows are read once and the codes written once: HBM-bound.
// A CTA goes through the heads of its block one after another (one head per CTA took 103 us for 35K rows of 8 heads:
// most of it finding the request, block and scale); long runs of rows come by TMA, three rounds ahead.
// Measured: 8 prompts of 35K rows together (bf16, 8 heads, d 128) 43 us = 5.0 TB/s, 0.73 of a plain copy's rate;
// 328K fp32 rows (d 64) 262 us = 6.4 TB/s, 0.94 (one round ahead into registers: 51.7 and 303 us).  The accepted
// paths of 32 requests 10.7 us with a cold cache, 6.5 warm: one launch and four loads in a row.
// A half-full block keeps its larger scale; its old codes are read only when the scale grows.
#include "common.cuh"
#include "kernels.cuh"
#include "pdl.cuh"

namespace spectree {

namespace {

constexpr int kVecs = 4;          // 16-byte source vectors a thread holds (8 where a block needs > 1024 threads)
constexpr long long kFillCtas = 152 * 4;
constexpr int kStages = 3;        // rounds of items in shared memory
constexpr int kMinExp = -64, kMaxExp = 120;

// The exponent of the smallest power of two s with amax <= 448 s (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_exp(uint32_t b) {  // the bits of amax
  if ((b >> 23) == 0) return kMinExp;  // zero and what is below 2^-126
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kMinExp), kMaxExp);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two floats to two e4m3 codes (the first in the low byte), to nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// One 16-byte source vector: 8 bf16 or 4 floats.  Magnitudes are compared as bits (a pair of bf16 at a time):
// their order is that of the numbers, with infinities and NaN on top.
template <bool BF16>
struct Vec {
  static constexpr int kElems = BF16 ? 8 : 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[kElems]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        x[i] = __uint_as_float(w[i]);
      }
    }
  }
  // `top` (bf16: two 16-bit maxima) with the vector's magnitudes
  static __device__ __forceinline__ uint32_t grow(uint32_t top, const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF16)
        top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
      else
        top = max(top, w[i] & 0x7FFFFFFFu);
    }
    return top;
  }
  // the bits of the larger of the two as a float
  static __device__ __forceinline__ uint32_t bits(uint32_t top) {
    return BF16 ? max(top << 16, top & 0xFFFF0000u) : top;
  }
};

// The bits of the vector's largest finite magnitude, and of `top`.
template <bool BF16>
__device__ __noinline__ uint32_t finite_top(uint32_t top, uint4 v) {
  float x[Vec<BF16>::kElems];
  Vec<BF16>::unpack(v, x);
  for (int e = 0; e < Vec<BF16>::kElems; ++e) {
    const uint32_t b = __float_as_uint(x[e]) & 0x7FFFFFFFu;
    if (b < 0x7F800000u) top = max(top, b);
  }
  return top;
}

// kElems codes at `dst` (8 or 4 bytes)
template <int E>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&x)[E]) {
  const uint32_t lo = e4m3x2(x[0], x[1]) | (e4m3x2(x[2], x[3]) << 16);
  if constexpr (E == 8) {
    const uint32_t hi = e4m3x2(x[4], x[5]) | (e4m3x2(x[6], x[7]) << 16);
    *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
  } else {
    *reinterpret_cast<uint32_t*>(dst) = lo;
  }
}

__device__ __forceinline__ int units_before(const int32_t* row_start, int b, int bs_shift) {
  return (row_start[b] >> bs_shift) + 2 * b;
}

struct Request {
  int count;  // rows to append; -1 = refused
  int err;
};

// Checks of request b that do not need its table; every thread of the block calls it (barriers inside).
__device__ __forceinline__ Request check_request(const Kv8AppendParams& p, int b) {
  Request r = {0, 0};
  const long long len = p.seq_len[b];
  int bad = 0;
  if (p.path) {
    const int a = p.accept_len[b];
    if (a < 0 || a >= p.path_cap) {
      r.err = SPEC_ERR_CAPACITY;
    } else {
      r.count = a + 1;
      const int32_t* pth = p.path + (size_t)b * p.path_cap;
      for (int j = threadIdx.x; j <= a; j += blockDim.x) {
        const int v = pth[j];
        if (v >= p.N || (j == 0 ? v != 0 : v <= pth[j - 1])) bad = 1;
      }
    }
  } else {
    r.count = p.row_start[b + 1] - p.row_start[b];
  }
  if (__syncthreads_or(bad)) r.err = SPEC_ERR_BAD_TREE;
  // (lengths are 32-bit numbers, whatever the table has room for)
  if (!r.err && (len < 0 || len + r.count > min((long long)p.max_blocks * p.bs, 0x7fffffffLL))) r.err = SPEC_ERR_CAPACITY;
  if (r.err) r.count = -1;
  return r;
}

// Is a table entry of the blocks that request b's rows go to out of range?  (block-wide)
__device__ __forceinline__ bool bad_table(const Kv8AppendParams& p, int b, long long len, int count) {
  int bad = 0;
  if (count > 0)
    for (long long j = (len >> p.bs_shift) + threadIdx.x; j <= (len + count - 1) >> p.bs_shift; j += blockDim.x) {
      const int blk = p.table[(size_t)b * p.max_blocks + j];
      if (blk < 0 || blk >= p.num_blocks) bad = 1;
    }
  return __syncthreads_or(bad);
}

}  // namespace

// Grid: units x parts.  A unit is one block that rows of a request go to; its items are the 2 * Hkv (head, K
// or V) blocks of codes; a part is a run of them, which the CTA's groups of TG threads take in turn.
// TMA: the packed rows of an item come as one box into a ring in shared memory, kStages rounds ahead, instead of one
// round ahead into registers.
template <bool BF16, int NV, int THREADS, bool TMA>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    kv8_append_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const Kv8AppendParams p, int parts, int tg_shift) {
  constexpr int E = Vec<BF16>::kElems;
  constexpr int kStageBytes = THREADS * NV * 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = TMA ? reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127)) : nullptr;
  __shared__ uint64_t s_full[kStages];
  __shared__ uint32_t s_max[2][32];
  __shared__ int s_gave_up;  // a wait for a box has passed its limit
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int u = blockIdx.x / parts, part = blockIdx.x - u * parts;
  pdl_wait();  // what comes before in the stream may still be ending: nothing of it is read ahead of this
  // ---- the unit's request and block ----
  int b, k;  // request, its k-th touched block
  if (p.path) {
    b = u / p.units_per_req;
    k = u - b * p.units_per_req;
  } else {
    // units are laid out from floor(row_start / bs) + 2 b, which leaves each request at least as many as
    // its rows can touch at any offset; 32-way search, one probe per lane
    int lo = 0, n = p.B;
    while (n > 1) {
      const int step = (n + 31) >> 5;
      const int at = min(lo + lane * step, lo + n - 1);
      const bool le = lane * step < n && units_before(p.row_start, at, p.bs_shift) <= u;
      const unsigned m = __ballot_sync(0xffffffffu, le);
      const int hit = m ? 31 - __clz(m) : 0;
      const int rest = n - hit * step;
      lo += hit * step;
      n = min(step, rest);
    }
    b = lo;
    k = u - units_before(p.row_start, b, p.bs_shift);
    // a row_start that decreases or leaves its range would share units out wrongly: the whole call is refused
    int bad = 0;
    for (int i = tid; i < p.B; i += THREADS) {
      const int r = p.row_start[i], next = p.row_start[i + 1];
      bad |= r < 0 || next < r || next > p.n_rows;
    }
    if (__syncthreads_or(bad)) {
      if (tid == 0 && part == 0 && u < p.B) {
        set_status(p.dev_status, SPEC_ERR_CAPACITY);
        if (p.new_len) p.new_len[u] = p.seq_len[u];
      }
      return;
    }
    if (k < 0) return;  // (rows ahead of the first request's)
  }
  const Request rq = check_request(p, b);
  const int len = p.seq_len[b];
  const bool lead = k == 0 && part == 0;  // this CTA answers for the request
  bool bad = false;
  if (rq.count > 0 && (p.path || lead)) bad = bad_table(p, b, len, rq.count);
  if (lead && tid == 0) {
    if (rq.err || bad) set_status(p.dev_status, rq.err ? rq.err : SPEC_ERR_CAPACITY);
    if (p.new_len) p.new_len[b] = len + (rq.err || bad ? 0 : rq.count);
  }
  if (rq.count <= 0 || (p.path && bad)) return;
  const long long first = ((long long)(len >> p.bs_shift) + k) << p.bs_shift;  // first slot of the block
  if (first >= (long long)len + rq.count) return;
  const int held = max(0, (int)(len - first));                       // slots that hold older rows
  const int end = (int)min((long long)p.bs, len + rq.count - first);  // new rows go to [held, end)
  const int blk = p.table[(size_t)b * p.max_blocks + (first >> p.bs_shift)];
  if (blk < 0 || blk >= p.num_blocks) return;  // (the lead CTA has set the status)

  // ---- this thread's vectors: the same places of every item, counted from the first new row.  Where a group cannot
  // hold all of a block's (a prompt among single tokens), the others are read twice. ----
  const int tg = 1 << tg_shift, groups = blockDim.x >> tg_shift;
  const int t = tid & (tg - 1);
  const int row_shift = 31 - __clz(p.d / E);  // vectors per row: a power of two
  const int row_bytes = p.d * (BF16 ? 2 : 4);
  const long long row0 = p.path ? (long long)b * p.N : (long long)p.row_start[b] + (first - len);
  const int32_t* pth = p.path ? p.path + (size_t)b * p.path_cap + (first - len) : nullptr;
  const int start = held << row_shift, vecs = (end - held) << row_shift;
  auto source = [&](int q) {  // source row of vector q, or -1 behind the last new row
    const int r = held + (q >> row_shift);
    return q < vecs ? (int)(p.path ? row0 + pth[r] : row0 + r) : -1;
  };
  int from[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) from[j] = source(t + j * tg);
  const int items = 2 * p.Hkv, per = (items + parts - 1) / parts;
  const int i0 = part * per, i1 = min(items, i0 + per);
  const size_t cell0 = (size_t)blk * p.Hkv;
  auto vector = [&](int item, int q, int row) {
    const uint8_t* src = static_cast<const uint8_t*>((item & 1) ? p.v_new : p.k_new) + (size_t)(item >> 1) * row_bytes;
    const int col = q & ((1 << row_shift) - 1);
    return __ldcs(reinterpret_cast<const uint4*>(src + row * ((size_t)p.Hkv * row_bytes) + col * 16));
  };
  auto scale_of = [&](int item) { return ((item & 1) ? p.v_scale : p.k_scale) + cell0 + (item >> 1); };
  auto load = [&](int item, uint4 (&v)[NV], float& s_old) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      v[j] = make_uint4(0, 0, 0, 0);
      if (item < i1 && from[j] >= 0) v[j] = vector(item, t + j * tg, from[j]);
    }
    s_old = item < i1 && held ? *scale_of(item) : 0.f;
  };
  uint4 next[NV];
  float s_next;
  const int mine0 = i0 + (tid >> tg_shift);
  const int item_bytes = NV * 16 << tg_shift;
  int asked = 0;  // rounds
  auto fetch = [&](int base, int stage) {  // one thread: the boxes of a round's items
    ++asked;
    const int n = min(groups, i1 - base);
    mbar_arrive_expect_tx(&s_full[stage], (uint32_t)(n * item_bytes));
    for (int g = 0; g < n; ++g)
      tma_load_3d(ring + stage * kStageBytes + g * item_bytes, (base + g) & 1 ? &tmV : &tmK, &s_full[stage], 0,
                  (base + g) >> 1, (int)(row0));
  };
  if constexpr (TMA) {
    if (tid == 0) {
      s_gave_up = 0;
      for (int i = 0; i < kStages; ++i) mbar_init(&s_full[i], 1);
      fence_mbar_init();
      for (int i = 0; i < kStages && i0 + i * groups < i1; ++i) fetch(i0 + i * groups, i);
    }
    __syncthreads();
    s_next = mine0 < i1 && held ? *scale_of(mine0) : 0.f;
  } else {
    load(mine0, next, s_next);
  }
  int stage = 0, phase = 0;
  for (int base = i0, turn = 0; base < i1; base += groups, turn ^= 1) {  // (every thread: barriers inside)
    const int item = base + (tid >> tg_shift);
    uint4 v[NV];
    const float s_old = s_next;
    if constexpr (TMA) {
      // A thread that gives up stays with the others, whose warp's and block's steps follow: behind the barrier all know,
      // and the rounds that are left ask for nothing, wait for nothing and write nothing.
      if (!mbar_wait_bounded(&s_full[stage], phase, &s_gave_up)) s_gave_up = 1;
      const uint4* box = reinterpret_cast<const uint4*>(ring + stage * kStageBytes + (tid >> tg_shift) * item_bytes);
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = from[j] >= 0 ? box[start + t + j * tg] : make_uint4(0, 0, 0, 0);
      const int ahead = item + groups;
      s_next = ahead < i1 && held ? *scale_of(ahead) : 0.f;
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = next[j];
      load(item + groups, next, s_next);
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) top = Vec<BF16>::grow(top, v[j]);
    top = Vec<BF16>::bits(top);
    if (top >= 0x7F800000u) {  // NaN and infinities are left out
      top = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j) top = finite_top<BF16>(top, v[j]);
    }
    if constexpr (!TMA)
      if (item < i1)
#pragma unroll 1
        for (int q = t + NV * tg; q < vecs; q += tg) top = finite_top<BF16>(top, vector(item, q, source(q)));
    top = __reduce_max_sync(0xffffffffu, top);
    if (TMA || tg > 32) {
      if (lane == 0) s_max[turn][warp] = top;
      __syncthreads();
      if constexpr (TMA) {  // the round has been read: its place is free
        if (tid == 0 && base + kStages * groups < i1 && !s_gave_up) fetch(base + kStages * groups, stage);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (tg > 32) {
      const int w0 = (tid >> tg_shift) << (tg_shift - 5);
      top = __reduce_max_sync(0xffffffffu, lane < (tg >> 5) ? s_max[turn][w0 + lane] : 0u);
    }
    if (item >= i1 || (TMA && s_gave_up)) continue;
    uint8_t* codes = ((item & 1) ? p.v_cache : p.k_cache) + (cell0 + (item >> 1)) * ((size_t)p.bs * p.d);
    const float s_new = pow2f(scale_exp(top));
    const bool grown = held && !(s_old >= s_new);
    const float s = held && !grown ? s_old : s_new;
    // x / s: by the reciprocal where s is a power of two (always, unless the caller's own scale stays)
    if ((__float_as_uint(s) & 0x7FFFFFu) == 0u && s >= 5.4210108624275222e-20f &&
        s <= 1.329227995784916e36f) {  // 2^-64 .. 2^120
      const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));
      const float2 inv2 = make_float2(inv, inv);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (from[j] < 0) continue;
        float x[E];
        Vec<BF16>::unpack(v[j], x);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 y = __fmul2_rn(make_float2(x[e], x[e + 1]), inv2);
          x[e] = y.x;
          x[e + 1] = y.y;
        }
        store_codes<E>(codes + (size_t)(start + t + j * tg) * E, x);
      }
    } else {
#pragma unroll 1
      for (int j = 0; j < NV; ++j) {
        uint4 w = make_uint4(0, 0, 0, 0);
        int row = -1;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (i == j) {
            w = v[i];
            row = from[i];
          }
        if (row < 0) continue;
        float x[E];
        Vec<BF16>::unpack(w, x);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = x[e] / s;
        store_codes<E>(codes + (size_t)(start + t + j * tg) * E, x);
      }
    }
    if constexpr (!TMA)
#pragma unroll 1
      for (int q = t + NV * tg; q < vecs; q += tg) {
        float x[E];
        Vec<BF16>::unpack(vector(item, q, source(q)), x);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = x[e] / s;
        store_codes<E>(codes + (size_t)(start + q) * E, x);
      }
    if (grown) {  // the old rows' codes in the new scale
      const float ratio = s_old / s;
#pragma unroll 1
      for (int c = t; c < held << row_shift; c += tg) {
        float x[E];
        const uint32_t* w = reinterpret_cast<const uint32_t*>(codes + (size_t)c * E);
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const uint32_t q = w[e / 4];
          const float2 a = from_e4m3x2(q & 0xFFFFu), z = from_e4m3x2(q >> 16);
          x[e] = a.x * ratio; x[e + 1] = a.y * ratio; x[e + 2] = z.x * ratio; x[e + 3] = z.y * ratio;
        }
        store_codes<E>(codes + (size_t)c * E, x);
      }
    }
    if (t == 0) *scale_of(item) = s;
  }
  if constexpr (TMA)
    if (tid == 0 && s_gave_up) {
      set_status(p.dev_status, SPEC_ERR_TIMEOUT);
      for (int i = 0; i < kStages; ++i)  // what is in flight lands first (again with a limit)
        if (asked > i) mbar_wait_bounded(&s_full[(asked - 1 - i) % kStages], ((asked - 1 - i) / kStages) & 1, nullptr);
    }
}

namespace {

struct AppendShape {
  int tg_shift, threads, parts, nv;
  bool boxes;  // packed rows by TMA
  long long units;
};

AppendShape append_shape(const Kv8AppendParams& p) {
  AppendShape s;
  // A group holds a block's new rows: of a path, all there can be; of packed rows a whole block, or, where the
  // requests have few on average (tokens, one each), about as many as that.  One row for each of 512 requests (bf16,
  // d 128, blocks of 64): 17.5 us, as whole blocks by TMA 34, into registers 40; 16 rows each: by TMA 36, into
  // registers 44.  (fp32, blocks of 256, one row each: 17.5 and 261.)
  long long rows = p.bs;
  if (p.path) rows = p.path_cap < p.N ? p.path_cap : p.N;
  else if (p.n_rows < (long long)p.B * p.bs / 8) rows = (p.n_rows + p.B - 1) / p.B;
  const bool whole = rows >= p.bs;
  int fit = 1;
  while (fit < rows && fit < p.bs) fit <<= 1;
  const int vecs = fit * p.d / (p.is_bf16 ? 8 : 4);  // up to 8192 (256 x 128 fp32)
  s.nv = vecs > 1024 * kVecs ? 2 * kVecs : kVecs;
  s.boxes = !p.path && whole && p.n_rows > 0 && s.nv == kVecs;
  s.tg_shift = 5;
  while ((s.nv << s.tg_shift) < vecs) ++s.tg_shift;
  const int tg = 1 << s.tg_shift;
  s.threads = tg > 256 ? tg : 256;
  // as many parts per unit as keep every SM busy, down to one for long prompts
  const int groups = s.threads / tg, most = (2 * p.Hkv + groups - 1) / groups;
  s.units = p.path ? (long long)p.B * p.units_per_req : (p.n_rows >> p.bs_shift) + 2ll * p.B;
  const long long want = (kFillCtas + s.units - 1) / s.units;
  s.parts = want < 1 ? 1 : want > most ? most : (int)want;
  return s;
}

}  // namespace

unsigned kv8_append_grid(const Kv8AppendParams& p) {
  const AppendShape s = append_shape(p);
  const long long g = s.units * s.parts;
  return g > 0x7fffffffLL ? 0u : (unsigned)g;
}

cudaError_t launch_kv8_append(const CUtensorMap* tm, const Kv8AppendParams& p, cudaStream_t stream) {
  const AppendShape s = append_shape(p);
  const unsigned grid = kv8_append_grid(p);
  static const CUtensorMap none = {};
  cudaError_t err = cudaSuccess;
  auto go = [&](auto kernel, size_t smem = 0) {
    if (smem) err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err == cudaSuccess)
      err = launch_dependent(kernel, dim3(grid), dim3(s.threads), smem, stream, tm ? tm[0] : none, tm ? tm[1] : none, p,
                             s.parts, s.tg_shift);
  };
  const size_t ring = 128 + (size_t)kStages * s.threads * kVecs * 16;
  if (p.is_bf16) {
    if (s.threads == 256) {
      if (tm) go(kv8_append_kernel<true, kVecs, 256, true>, ring);
      else go(kv8_append_kernel<true, kVecs, 256, false>);
    } else if (s.threads == 512) {
      if (tm) go(kv8_append_kernel<true, kVecs, 512, true>, ring);
      else go(kv8_append_kernel<true, kVecs, 512, false>);
    } else {
      if (tm) go(kv8_append_kernel<true, kVecs, 1024, true>, ring);
      else go(kv8_append_kernel<true, kVecs, 1024, false>);
    }
  } else {
    if (s.threads == 256) {
      if (tm) go(kv8_append_kernel<false, kVecs, 256, true>, ring);
      else go(kv8_append_kernel<false, kVecs, 256, false>);
    } else if (s.threads == 512) {
      if (tm) go(kv8_append_kernel<false, kVecs, 512, true>, ring);
      else go(kv8_append_kernel<false, kVecs, 512, false>);
    } else if (s.nv == kVecs) {
      if (tm) go(kv8_append_kernel<false, kVecs, 1024, true>, ring);
      else go(kv8_append_kernel<false, kVecs, 1024, false>);
    } else {
      go(kv8_append_kernel<false, 2 * kVecs, 1024, false>);
    }
  }
  return err;
}

bool kv8_append_boxes(const Kv8AppendParams& p) { return append_shape(p).boxes; }

}  // namespace spectree
