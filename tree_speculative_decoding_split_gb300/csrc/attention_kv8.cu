// K9: tree attention over the 8-bit paged cache, for few rows per KV head (single tokens, short drafts),
// and the merge of its key splits.
//
// Row (node i, query head j) against key s of block c: x = (q . k8) * kscale_c * scale (log2 units), weights
// 2^x, out = sum 2^x vscale_c v8 / sum 2^x.  The V scale is folded into the exponent: with
// y = x + log2(vscale_c) and a running reference m of y, P' = 2^(y - m) multiplies the codes themselves and
// the sum adds P' / vscale_c.  So no code is ever rescaled: e4m3 becomes f16 exactly, on the way from
// shared memory to the registers of m16n8k16.  Keys (then dimensions) are on M and the few rows on N = 8:
//   S^T = K Q^T,   O^T += V^T P^T,
// with P^T from S^T by one 8 x 8 transposition in registers per 8 keys.
//
// With 16 rows or fewer a key's 2 d bytes carry 4 d * 16 products at most, far below what the tensor
// cores need to be busy: the kernel is bound by HBM.  What matters is bytes in flight, so every warp
// runs its own ring of TMA boxes of 16 keys and its own softmax state over every fourth box of the
// split, without any barrier between warps; the four states are joined at the end.
// The tree's weights enter their product as a pair of bf16 numbers (to 2^-16 of them), the prefix's as f16.
// Measured: 32 requests of 4 rows over 2K to 6K keys (8 KV heads, d 128) 57 us = 4.7 TB/s of codes, 0.69 of a plain
// copy's rate; one request at 2K 18.9 us with a cold cache, 14.6 warm, most of it latency (two launches, and three
// loads that hang on one another ahead of the first keys).  With two 8-row tiles the registers (246) leave two CTAs
// an SM; three with a few spilled take as long, four twice as long.
#include "common.cuh"
#include "kernels.cuh"
#include "kv8.cuh"
#include "pdl.cuh"

namespace spectree {

namespace {

constexpr int kWarps = 4;
constexpr int kStagesR = 3;      // boxes of 16 keys (K and V) in flight per warp
constexpr float kLazy = 8.f;     // the reference maximum may be 2^8 behind: P' <= 256, far inside f16

// RN: 8-row tiles per CTA
template <int D, int RN>
struct RowsCfg {
  static constexpr int kRows = 8 * RN;
  static constexpr int kBox = 16 * D;                 // bytes of 16 keys of K (or V)
  static constexpr int kRing = kWarps * kStagesR * 2 * kBox;
  static constexpr int kJoin = kWarps * kRows * (D + 4) * 4;  // O of every warp, rows padded
  static constexpr int kSmem = 1024 + (kRing > kJoin ? kRing : kJoin);
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit elements held two per lane (row lane / 4).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// two e4m3 codes (the low or high half of `w`) to f16, exactly
template <int HALF>
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (HALF == 0)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ bool bf16_pair_finite(uint32_t w) {
  return (w & 0x7F80u) != 0x7F80u && (w & 0x7F800000u) != 0x7F800000u;
}

// Softmax state of a lane's rows 2t and 2t + 1 of every 8-row tile; m is equal in the lanes that share them, l
// covers this lane's keys only.
template <int RN>
struct RowState {
  float m[RN][2], l[RN][2];
};

// y[tile][key g, g + 8 | row 2t, 2t + 1]: this lane's scores (log2 units, V scale included).  Moves the
// references when a score has run ahead of one, then returns P' and adds it to the sums.  `rebase`, at the
// first prefix keys behind tree keys: references move down as well, as f16 weights need one near their own
// largest, however small the prefix's V scales are (the tree's bf16 weights bear any).
template <int RN, int NT>
__device__ __forceinline__ void softmax_step(float (&y)[RN][4], RowState<RN>& st, float (&o)[RN][NT][4], float inv_vs,
                                             bool rebase) {
  bool ahead = rebase;
#pragma unroll
  for (int n = 0; n < RN; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r) ahead = ahead || fmaxf(y[n][r], y[n][2 + r]) - st.m[n][r] > kLazy;
  if (__any_sync(0xffffffffu, ahead)) {
#pragma unroll
    for (int n = 0; n < RN; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float v = fmaxf(y[n][r], y[n][2 + r]);
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
        // each row by its own scores alone, so that no row's rounding depends on its neighbours
        const float m = st.m[n][r];
        // (down by 64 at most, also where 64 is less than a step of m)
        const float mn = v - m > kLazy || (rebase && v > -INFINITY) ? fmaxf(v, __fsub_ru(m, 64.f)) : m;
        const float f = mn == m ? 1.f : ex2_approx(m - mn);
        st.m[n][r] = mn;
        st.l[n][r] *= f;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          o[n][j][r] *= f;
          o[n][j][2 + r] *= f;
        }
      }
  }
#pragma unroll
  for (int n = 0; n < RN; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float mu = st.m[n][r] == -INFINITY ? 0.f : st.m[n][r];
      y[n][r] = ex2_approx(y[n][r] - mu);
      y[n][2 + r] = ex2_approx(y[n][2 + r] - mu);
      st.l[n][r] = fmaf(y[n][r] + y[n][2 + r], inv_vs, st.l[n][r]);
    }
}

}  // namespace

template <int D, int RN>
__global__ void __launch_bounds__(kWarps * 32, RN == 1 ? 4 : 2)
    attn_kv8_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const Kv8AttnParams p) {
  using C = RowsCfg<D, RN>;
  constexpr int kRowsR = C::kRows;
  constexpr int RUN = D / 4;   // consecutive dimensions of a query or key row that a lane holds
  constexpr int KS = D / 16;   // k steps of K Q^T
  constexpr int NT = D / 16;   // m tiles of V^T P^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t s_full[kWarps][kStagesR];
  __shared__ int s_par[kMaxNodes];
  __shared__ uint32_t s_anc[kRowsR][kAncWords];
  __shared__ float s_m[kWarps][kRowsR], s_l[kWarps][kRowsR];
  __shared__ uint32_t s_odd[kAncWords];  // tree keys with an infinity or NaN in their V row
  __shared__ int s_bad, s_abort;  // a table entry out of range; a wait that gave up
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  Kv8Work sp = kv8_own(p);
  // queries: row g of every 8-row tile, dimensions [RUN t, RUN t + RUN); they and the tree's links are on their way
  // while the lengths are read, where they do not hang on them
  uint4 qv[RN][RUN / 8];
  int par0 = -1;
  auto early = [&]() {
#pragma unroll
    for (int r = 0; r < RN; ++r) {
      const int row = sp.rt * kRowsR + g + 8 * r;
      const bool has = row < p.N * p.G;
      const uint16_t* qrow = p.q + kv8_row(p, sp.b, sp.h, has ? row : 0) * D + RUN * t;
#pragma unroll
      for (int i = 0; i < RUN / 8; ++i)
        qv[r][i] = has ? *reinterpret_cast<const uint4*>(qrow + 8 * i) : make_uint4(0, 0, 0, 0);
    }
    if (tid < p.N) par0 = p.parent[(size_t)sp.b * p.N + tid];
  };
  pdl_wait();  // what comes before in the stream may still be ending: nothing of it is read ahead of this
  pdl_launch_dependents();  // the merge may be launched
  const bool own = sp.b >= 0;
  if (own) early();
  sp = kv8_begin(p, sp);
  if (sp.b < 0) return;
  if (!own) early();
  const int b = sp.b, h = sp.h, rt = sp.rt, split = sp.split, n = sp.nodes;
  const long long L = sp.L;
  int err = sp.err;
  const int row0 = rt * kRowsR, rows = p.N * p.G;
  auto orow_of = [&](int row) { return kv8_row(p, b, h, row); };
  if (lane == 0) {
    for (int s = 0; s < kStagesR; ++s) mbar_init(&s_full[warp][s], 1);
    fence_mbar_init();
  }
  if (tid == 0) s_bad = s_abort = 0;
  if (tid < kAncWords) s_odd[tid] = 0u;
  // ---- this warp's boxes: box c0 + warp + 4 i of 16 keys.  Their first table entries, scales and copies are on
  // their way while the tree is checked.
  const bool tree = split == sp.n - 1;  // the last split takes the tree's keys
  const int nbox = (int)((L + 15) >> 4);
  const int c0 = (split * sp.steps) << (p.unit_shift - 4);
  const int c1 = min(nbox, c0 + (sp.steps << (p.unit_shift - 4)));
  const int mine = c0 + warp < c1 ? (c1 - c0 - warp + kWarps - 1) / kWarps : 0;
  uint8_t* ring = base + warp * (kStagesR * 2 * C::kBox);
  // table entries, and K scale, log2 and reciprocal of the V scale, of 32 boxes at a time, one per lane:
  // `e` for the boxes being requested, `c` for those being worked on
  int blk_e = -1;
  float ks_e = 0.f, iv_e = 0.f, ks_c, lv_c, iv_c;
  bool bad = false;
  auto fetch = [&](int batch) {
    const int i = batch * 32 + lane;
    blk_e = -1;
    float ks = 0.f, vs = 1.f;
    if (i < mine) {
      const int slot = (c0 + warp + kWarps * i) * 16;
      const int blk = p.table[(size_t)b * p.max_blocks + (slot >> p.bs_shift)];
      if (blk < 0 || blk >= p.num_blocks) {
        bad = true;
      } else {
        blk_e = blk;
        ks = p.k_scale[(size_t)blk * p.Hkv + h];
        vs = p.v_scale[(size_t)blk * p.Hkv + h];
      }
    }
    ks_e = ks;
    iv_e = vs;  // turned into the reciprocal and logarithm when the boxes' turn comes (the load is in flight)
  };
  auto turn = [&]() {
    const float vs = kv8_clamp_scale(iv_e);
    ks_c = kv8_clamp_scale(ks_e);
    lv_c = __log2f(vs);
    iv_c = __fdividef(1.f, vs);
  };
  auto request = [&](int i) {  // box i of this warp -> stage i % kStagesR
    const int blk = __shfl_sync(0xffffffffu, blk_e, i & 31);
    if (lane == 0) {
      const int s = i % kStagesR;
      const int slot = (c0 + warp + kWarps * i) * 16;
      uint8_t* dst = ring + s * 2 * C::kBox;
      if (blk >= 0) {
        mbar_arrive_expect_tx(&s_full[warp][s], 2 * C::kBox);
        tma_load_3d(dst, &tmK, &s_full[warp][s], 0, slot & (p.bs - 1), blk * p.Hkv + h);
        tma_load_3d(dst + C::kBox, &tmV, &s_full[warp][s], 0, slot & (p.bs - 1), blk * p.Hkv + h);
      } else {
        mbar_arrive(&s_full[warp][s]);  // a bad table entry: the request's rows come out as 0
      }
    }
  };
  const int pre = min(mine, kStagesR);
  if (mine > 0) {
    fetch(0);
    __syncwarp();
    for (int i = 0; i < pre; ++i) request(i);
  }
  // a CTA that leaves early lets its copies land first
  auto drain = [&]() {
    if (lane == 0)
      for (int i = 0; i < pre; ++i) mbar_wait_bounded(&s_full[warp][i], 0, nullptr);
  };
  for (int i = tid; i < n; i += blockDim.x) {
    const int par = i == tid ? par0 : p.parent[(size_t)b * p.N + i];
    s_par[i] = par;
    if (i == 0 ? par != -1 : (par < 0 || par >= i)) err = SPEC_ERR_BAD_TREE;
  }
  if (__syncthreads_or(err == SPEC_ERR_BAD_TREE)) err = SPEC_ERR_BAD_TREE;
  // the final rows of a request that is refused, or of padded nodes; with several splits the merge does it
  auto refuse = [&]() {
    for (int c = tid; c < kRowsR * (D / 8); c += blockDim.x) {
      const int row = row0 + c / (D / 8), e = c % (D / 8);
      if (row >= rows) continue;
      const size_t o = orow_of(row);
      if (sp.n == 1) {
        *reinterpret_cast<uint4*>(p.out + o * D + e * 8) = make_uint4(0, 0, 0, 0);
        if (e == 0 && p.lse) p.lse[o] = 0.f;
      } else if (e == 0) {
        p.part_ml[sp.part + (row - row0)] = make_float2(0.f, -1.f);
      }
    }
  };
  if (err) {
    if (tid == 0 && rt == 0 && split == 0 && h == 0) set_status(p.dev_status, err);
    refuse();
    drain();
    return;
  }
  if (row0 >= n * p.G) {  // padded nodes only
    if (sp.n == 1) refuse();
    drain();
    return;
  }
  // ---- ancestors-or-self of the tile's rows ----
  if (tree) {
    if (tid < kRowsR) {
#pragma unroll
      for (int i = 0; i < kAncWords; ++i) s_anc[tid][i] = 0u;
      const int i = kv8_node(p, row0 + tid);
      if (row0 + tid < rows && i < n)
        for (int a = i; a >= 0; a = s_par[a]) s_anc[tid][a >> 5] |= 1u << (a & 31);
    }
    __syncthreads();
  }
  // queries as f16 times a power of two per row that brings the row's largest element to [16, 32); below 2^-18 of
  // it elements lose bits, 2^-29 of it at most
  uint32_t qb[RN][KS][2];
  float qf[RN][2];  // of rows 2t, 2t + 1: undoes that, with the softmax scale in log2 units
#pragma unroll
  for (int r = 0; r < RN; ++r) {
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < RUN / 8; ++i) {
      const uint32_t w[4] = {qv[r][i].x, qv[r][i].y, qv[r][i].z, qv[r][i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[j])), fabsf(bf16_hi(w[j]))));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // the factor 2^(4 - floor(log2 mx)) and its reciprocal are normal numbers up to the exponent 128 of an infinity; at
    // the lower end mx counts as 2^-100 at least
    const int e = max((int)(__float_as_uint(mx) >> 23) - 127, -100);
    const float up = __uint_as_float((uint32_t)(127 + 4 - e) << 23);
    const float down = __uint_as_float((uint32_t)(127 - 4 + e) << 23) * p.scale_log2;
    qf[r][0] = __shfl_sync(0xffffffffu, down, 8 * t);
    qf[r][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
    for (int i = 0; i < RUN / 8; ++i) {
      const uint32_t w[4] = {qv[r][i].x, qv[r][i].y, qv[r][i].z, qv[r][i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        qb[r][2 * i + (j >> 1)][j & 1] = pack_f16x2(bf16_lo(w[j]) * up, bf16_hi(w[j]) * up);
    }
  }
  float o[RN][NT][4];
#pragma unroll
  for (int r = 0; r < RN; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[r][j][i] = 0.f;
  RowState<RN> st;
#pragma unroll
  for (int r = 0; r < RN; ++r) {
    st.m[r][0] = st.m[r][1] = -INFINITY;
    st.l[r][0] = st.l[r][1] = 0.f;
  }

  // ---- the tree's keys, 16 at a time, in bf16 from global memory ----
  if (tree) {
    for (int j0 = (kWarps - 1 - warp) * 16; j0 < n; j0 += kWarps * 16) {
      float y[RN][4];
#pragma unroll
      for (int r = 0; r < RN; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[r][i] = 0.f;
      const bool in0 = j0 + g < n, in1 = j0 + g + 8 < n;
      const uint16_t* k0 = p.k_tree + (((size_t)b * p.N + (in0 ? j0 + g : 0)) * p.Hkv + h) * D + RUN * t;
      const uint16_t* k1 = p.k_tree + (((size_t)b * p.N + (in1 ? j0 + g + 8 : 0)) * p.Hkv + h) * D + RUN * t;
      const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < RUN / 8; ++i) {
        const uint4 x0 = in0 ? *reinterpret_cast<const uint4*>(k0 + 8 * i) : z;
        const uint4 x1 = in1 ? *reinterpret_cast<const uint4*>(k1 + 8 * i) : z;
#pragma unroll
        for (int r = 0; r < RN; ++r) {
          const int row = row0 + g + 8 * r;
          const uint4 q = row < rows ? *reinterpret_cast<const uint4*>(p.q + orow_of(row) * D + RUN * t + 8 * i) : z;
          mma_bf16(y[r], x0.x, x1.x, x0.y, x1.y, q.x, q.y);
          mma_bf16(y[r], x0.z, x1.z, x0.w, x1.w, q.z, q.w);
        }
      }
#pragma unroll
      for (int r = 0; r < RN; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = j0 + g + 8 * (i >> 1);
          const bool see = key < n && ((s_anc[8 * r + 2 * t + (i & 1)][key >> 5] >> (key & 31)) & 1u);
          y[r][i] = see ? y[r][i] * p.scale_log2 : -INFINITY;
        }
      softmax_step<RN, NT>(y, st, o, 1.f, false);
      // The weights as bf16, and what that rounding leaves: together to 2^-16 of them, as a short prefix leaves most to
      // the tree.
      uint32_t pb[RN][4];
#pragma unroll
      for (int r = 0; r < RN; ++r) {
        const uint32_t h0 = pack_bf16x2(y[r][0], y[r][1]), h1 = pack_bf16x2(y[r][2], y[r][3]);
        pb[r][0] = transpose8(h0);
        pb[r][1] = transpose8(h1);
        pb[r][2] = transpose8(pack_bf16x2(y[r][0] - bf16_lo(h0), y[r][1] - bf16_hi(h0)));
        pb[r][3] = transpose8(pack_bf16x2(y[r][2] - bf16_lo(h1), y[r][3] - bf16_hi(h1)));
      }
      // V rows 2t, 2t + 1, 2t + 8, 2t + 9 of the chunk, dimensions 2 NT g .. 2 NT g + 2 NT - 1, eight at a time; an
      // element that is no finite number enters as 0 and is added at the end, to the rows that see it only
#pragma unroll
      for (int i = 0; i < NT / 4; ++i) {
        uint32_t v[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = j0 + 2 * t + (k & 1) + (k >> 1) * 8;
          uint4 x = z;
          if (key < n)
            x = *reinterpret_cast<const uint4*>(p.v_tree + (((size_t)b * p.N + key) * p.Hkv + h) * D + 2 * NT * g + 8 * i);
          v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
          if (!(bf16_pair_finite(x.x) && bf16_pair_finite(x.y) && bf16_pair_finite(x.z) && bf16_pair_finite(x.w))) {
            atomicOr(&s_odd[key >> 5], 1u << (key & 31));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((v[k][e] & 0x7F80u) == 0x7F80u) v[k][e] &= 0xFFFF0000u;
              if ((v[k][e] & 0x7F800000u) == 0x7F800000u) v[k][e] &= 0xFFFFu;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a0 = __byte_perm(v[0][j], v[1][j], 0x5410), a1 = __byte_perm(v[0][j], v[1][j], 0x7632);
          const uint32_t a2 = __byte_perm(v[2][j], v[3][j], 0x5410), a3 = __byte_perm(v[2][j], v[3][j], 0x7632);
#pragma unroll
          for (int r = 0; r < RN; ++r) {
            mma_bf16(o[r][4 * i + j], a0, a1, a2, a3, pb[r][0], pb[r][1]);
            mma_bf16(o[r][4 * i + j], a0, a1, a2, a3, pb[r][2], pb[r][3]);
          }
        }
      }
    }
  }

  // ---- the prefix ----
  turn();
  bool ok = true;
  int i = 0;
  for (; i < mine; ++i) {
    const int s = i % kStagesR;
    if ((i & 31) == 0 && i > 0) turn();  // (the requests have moved on to this batch kStagesR boxes ago)
    const float ks = __shfl_sync(0xffffffffu, ks_c, i & 31);
    const float lv = __shfl_sync(0xffffffffu, lv_c, i & 31), inv_vs = __shfl_sync(0xffffffffu, iv_c, i & 31);
    // (the lanes leave together: what follows is the whole warp's)
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&s_full[warp][s], (i / kStagesR) & 1, &s_abort))) {
      ok = false;
      break;
    }
    const uint8_t* sk = ring + s * 2 * C::kBox;
    const uint8_t* sv = sk + C::kBox;
    const int left = (int)min(16ll, L - (c0 + warp + kWarps * i) * 16);  // keys of the box inside the prefix
    float y[RN][4];
#pragma unroll
    for (int r = 0; r < RN; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[r][e] = 0.f;
    uint32_t w[2][RUN / 4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int key = 8 * k + g;
      if constexpr (D == 128) {
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const uint4 x = *reinterpret_cast<const uint4*>(sk + key * 128 + (((2 * t + i2) ^ (key & 7)) << 4));
          w[k][4 * i2] = x.x; w[k][4 * i2 + 1] = x.y; w[k][4 * i2 + 2] = x.z; w[k][4 * i2 + 3] = x.w;
        }
      } else {
        const uint4 x = *reinterpret_cast<const uint4*>(sk + key * 64 + ((t ^ ((key >> 1) & 3)) << 4));
        w[k][0] = x.x; w[k][1] = x.y; w[k][2] = x.z; w[k][3] = x.w;
      }
    }
    uint32_t v[4][NT / 2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int key = 2 * t + (k & 1) + (k >> 1) * 8;
      const bool in = key < left;  // slots behind the prefix may hold anything
      if constexpr (D == 128) {
        uint4 x = *reinterpret_cast<const uint4*>(sv + key * 128 + ((g ^ (key & 7)) << 4));
        if (!in) x = make_uint4(0, 0, 0, 0);
        v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
      } else {
        uint2 x = *reinterpret_cast<const uint2*>(sv + key * 64 + (((g >> 1) ^ ((key >> 1) & 3)) << 4) + (g & 1) * 8);
        if (!in) x = make_uint2(0, 0);
        v[k][0] = x.x; v[k][1] = x.y;
      }
    }
    // the stage is read: request the box that takes it next
    __syncwarp();
    if (i + kStagesR < mine) {
      if (((i + kStagesR) & 31) == 0) fetch((i + kStagesR) >> 5);
      request(i + kStagesR);
    }
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const uint32_t a0 = codes_f16x2<0>(w[0][k]), a1 = codes_f16x2<0>(w[1][k]);
      const uint32_t a2 = codes_f16x2<1>(w[0][k]), a3 = codes_f16x2<1>(w[1][k]);
#pragma unroll
      for (int r = 0; r < RN; ++r) mma_f16(y[r], a0, a1, a2, a3, qb[r][k][0], qb[r][k][1]);
    }
#pragma unroll
    for (int r = 0; r < RN; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y[r][e] = g + 8 * (e >> 1) < left ? fmaf(y[r][e], qf[r][e & 1] * ks, lv) : -INFINITY;
    softmax_step<RN, NT>(y, st, o, inv_vs, tree && i == 0);
    uint32_t pb[RN][2];
#pragma unroll
    for (int r = 0; r < RN; ++r) {
      pb[r][0] = transpose8(pack_f16x2(y[r][0], y[r][1]));
      pb[r][1] = transpose8(pack_f16x2(y[r][2], y[r][3]));
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      // bytes 2j, 2j + 1 of the four rows: (row 2t, row 2t + 1) pairs for the two dimensions
      const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
      const uint32_t lo = __byte_perm(v[0][j >> 1], v[1][j >> 1], sel);
      const uint32_t hi = __byte_perm(v[2][j >> 1], v[3][j >> 1], sel);
      const uint32_t a0 = codes_f16x2<0>(lo), a1 = codes_f16x2<1>(lo), a2 = codes_f16x2<0>(hi), a3 = codes_f16x2<1>(hi);
#pragma unroll
      for (int r = 0; r < RN; ++r) mma_f16(o[r][j], a0, a1, a2, a3, pb[r][0], pb[r][1]);
    }
  }
  if (!ok && lane == 0) {
    set_status(p.dev_status, SPEC_ERR_TIMEOUT);
    s_abort = 1;
    // the boxes that have been asked for and not been seen land first (again with a limit)
    for (int j = i; j < min(mine, i + kStagesR); ++j)
      mbar_wait_bounded(&s_full[warp][j % kStagesR], (j / kStagesR) & 1, nullptr);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) {
    set_status(p.dev_status, SPEC_ERR_CAPACITY);
    s_bad = 1;
  }
  // ---- join the four warps' states ----
#pragma unroll
  for (int n8 = 0; n8 < RN; ++n8)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int s = 4; s < 32; s <<= 1) st.l[n8][r] += __shfl_xor_sync(0xffffffffu, st.l[n8][r], s);
      if (g == 0) {
        s_m[warp][8 * n8 + 2 * t + r] = st.m[n8][r];
        s_l[warp][8 * n8 + 2 * t + r] = st.l[n8][r];
      }
    }
  __syncthreads();  // every box has landed and been read: the ring's memory is free
  if (s_bad || s_abort) {
    refuse();
    return;
  }
  float* join = reinterpret_cast<float*>(base);
#pragma unroll
  for (int n8 = 0; n8 < RN; ++n8)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int rr = 8 * n8 + 2 * t + r;
      float M = s_m[0][rr];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) M = fmaxf(M, s_m[w][rr]);
      const float f = st.m[n8][r] == -INFINITY ? 0.f : ex2_approx(st.m[n8][r] - M);
      float* dst = join + (warp * kRowsR + rr) * (D + 4) + 2 * NT * g;  // dimensions 2 NT g ..
#pragma unroll
      for (int j = 0; j < NT; j += 2)
        *reinterpret_cast<float4*>(dst + 2 * j) =
            make_float4(o[n8][j][r] * f, o[n8][j][2 + r] * f, o[n8][j + 1][r] * f, o[n8][j + 1][2 + r] * f);
    }
  __syncthreads();
  for (int c = tid; c < kRowsR * (D / 4); c += blockDim.x) {
    const int rr = c / (D / 4), e = c % (D / 4), row = row0 + rr;
    if (row >= rows) break;
    const bool real = row < n * p.G;
    if (!real && sp.n > 1) continue;  // the merge zeroes padded nodes
    float M = s_m[0][rr];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, s_m[w][rr]);
    float l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      l += s_m[w][rr] == -INFINITY ? 0.f : s_l[w][rr] * ex2_approx(s_m[w][rr] - M);
      const float4 x = *reinterpret_cast<const float4*>(join + (w * kRowsR + rr) * (D + 4) + e * 4);
      a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
    }
    if (tree && real) {  // V elements of visible tree keys that are no finite numbers
      for (int w = 0; w < kAncWords; ++w)
        for (uint32_t m = s_odd[w] & s_anc[rr][w]; m; m &= m - 1) {
          const int key = w * 32 + __ffs(m) - 1;
          const uint2 x =
              *reinterpret_cast<const uint2*>(p.v_tree + (((size_t)b * p.N + key) * p.Hkv + h) * D + e * 4);
          const float f[4] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y)};
          if (!(fabsf(f[0]) < INFINITY)) a.x += f[0];
          if (!(fabsf(f[1]) < INFINITY)) a.y += f[1];
          if (!(fabsf(f[2]) < INFINITY)) a.z += f[2];
          if (!(fabsf(f[3]) < INFINITY)) a.w += f[3];
        }
    }
    const size_t orow = orow_of(row);
    if (sp.n > 1) {
      *reinterpret_cast<float4*>(p.part_o + (sp.part + rr) * D + e * 4) = a;
      if (e == 0) p.part_ml[sp.part + rr] = make_float2(M, l);
    } else {
      const float inv = real ? 1.f / l : 0.f;
      uint2 out = make_uint2(0, 0);
      if (real) out = make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
      *reinterpret_cast<uint2*>(p.out + orow * D + e * 4) = out;
      if (e == 0 && p.lse) p.lse[orow] = real ? (M + log2f(l)) * 0.69314718055994531f : 0.f;
    }
  }
}

// Joins the splits of a row: one warp per row of a request that was split, lanes over dimensions.
template <int D>
__global__ void __launch_bounds__(256) attn_kv8_merge_kernel(const Kv8AttnParams p) {
  constexpr int EPL = D / 32;
  const int lane = threadIdx.x & 31;
  pdl_wait();  // first of all: a launch that ended before the attention's would let its successor overtake it
  const int per_req = p.N * p.Hq;
  int item = blockIdx.x * 8 + (threadIdx.x >> 5);  // among the rows of the split requests that follow
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int2 cuts = b0 + lane < p.B ? __ldcg(p.used + b0 + lane) : make_int2(1, 0);
    const unsigned split = __ballot_sync(0xffffffffu, cuts.x > 1);
    const int items = __popc(split) * per_req;
    for (; item < items; item += gridDim.x * 8) {
      const int nth = item / per_req, in_req = item - nth * per_req;
      unsigned rest = split;
      for (int j = 0; j < nth; ++j) rest &= rest - 1;
      const int src = __ffs(rest) - 1, b = b0 + src;
      const int used = __shfl_sync(0xffffffffu, cuts.x, src), first = __shfl_sync(0xffffffffu, cuts.y, src);
      const int i = in_req / p.Hq, hq = in_req - i * p.Hq, h = hq / p.G;
      const size_t orow = (size_t)b * per_req + in_req;
      // the row's place in the partial results of split s
      const int row = i * p.G + hq - h * p.G, rt = row / p.rows_cta;
      auto part = [&](int s) { return kv8_part(p, b, h, rt, s, first) + (row - rt * p.rows_cta); };
      const int n = p.n_nodes[b];
      const float2 ml =
          lane < used && i < n ? __ldcg(p.part_ml + part(lane)) : make_float2(-INFINITY, i < n ? 0.f : -1.f);
      const bool bad = __any_sync(0xffffffffu, ml.y < 0.f);
      const float M = warp_max(ml.x);
      const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
      const float l = warp_sum(ml.y * f);
      uint16_t* out = p.out + orow * D + lane * EPL;
      float acc[EPL];
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
      for (int s0 = 0; s0 < used && !bad; s0 += 4) {  // four splits' loads at a time
        float x[4][EPL], w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[k] = __shfl_sync(0xffffffffu, f, (s0 + k) & 31);
          const float* src_o = p.part_o + part(s0 + k) * D + lane * EPL;
          if (s0 + k < used) {
            if constexpr (EPL == 4) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(src_o));
              x[k][0] = v.x; x[k][1] = v.y; x[k][2] = v.z; x[k][3] = v.w;
            } else {
              const float2 v = __ldcg(reinterpret_cast<const float2*>(src_o));
              x[k][0] = v.x; x[k][1] = v.y;
            }
          } else {
            w[k] = 0.f;
#pragma unroll
            for (int e = 0; e < EPL; ++e) x[k][e] = 0.f;
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int e = 0; e < EPL; ++e) acc[e] = fmaf(x[k][e], w[k], acc[e]);
      }
      const float inv = bad ? 0.f : 1.f / l;  // (a row that is refused: acc is 0)
#pragma unroll
      for (int e = 0; e < EPL; e += 2)
        *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
      if (p.lse && lane == 0) p.lse[orow] = bad ? 0.f : (M + log2f(l)) * 0.69314718055994531f;
    }
    item -= items;
  }
}

// ---- host side ------------------------------------------------------------------------------

Kv8AttnPlan plan_attention_kv8(int B, int N, int G, int Hkv, long long L_cap, int num_sms) {
  Kv8AttnPlan pl;
  const int rows = N * G;
  const long long heads = (long long)B * Hkv;
  // Sixteen rows or fewer: 32 requests of 16 rows at 4K take 87 us here (d 64: 58) and 130 (110) on the tensor-core
  // kernel; one at 2K 23.7 and 21.7.
  if (rows <= 16) {
    pl.groups = 0;
    pl.unit_shift = 6;
    pl.n_rt = 1;
    // four CTAs an SM, as 8 rows have them (with 16 two or three fit: the plan is then for more than run at once)
    pl.slots = num_sms * 4;
    pl.fixed_steps = 2;
  } else {
    // Two groups of 128 rows per CTA cost little more a key tile than one (each fills the other's waits), so one
    // is for few rows, and for calls that give every SM less than a few tiles.  One group against two: 63 nodes at 2K
    // 23.7 and 27.7 us, 8 of them at 1K 32.9 and 39.0, one of 255 at 4K 56.4 and 44.1, 32 of 63 at 4K 245 and 136.
    const long long tiles = (L_cap + 127) / 128;
    pl.groups = rows > 128 && heads * ((rows + 255) / 256) * tiles >= 4 * num_sms ? 2 : 1;
    pl.unit_shift = 7;
    pl.n_rt = (rows + 128 * pl.groups - 1) / (128 * pl.groups);
    pl.slots = num_sms;
    pl.fixed_steps = 7;
  }
  pl.rows_cta = pl.groups == 0 ? (rows + 7) / 8 * 8 : 128 * pl.groups;
  // units, with splits no shorter than 256 keys, kKv8Splits per request at most
  const long long per = (long long)Hkv * pl.n_rt, ctas = B * per, most = (L_cap + 255) / 256;
  const long long limit = most < 1 ? 1 : (most < kKv8Splits ? most : kKv8Splits);
  long long more;
  if (pl.groups == 0) {
    // one round of CTAs (four an SM) where splits are fine enough to fill it, else at least one and a half: just over
    // one leaves the second almost empty.  1.0 rounds and up against 1.5 and up: 32 requests of 2K to 6K 67 and 62 us, 48
    // of 4K 97 and 80, 20 of 8K 93 and 72, 4 of 32K (19 or 29 splits) 62 and 68.
    pl.base = (int)(pl.slots / ctas);
    if (pl.base < 4) pl.base = (int)((pl.slots * 3ll / 2 + ctas - 1) / ctas);
    if (pl.base > limit) pl.base = (int)limit;
    more = pl.slots * 2ll / 3 / per + 1;
  } else {
    // CTAs for every slot, and up to six where the requests fill the slots by themselves and that leaves a split 64
    // steps of the longest prefixes (those that are not used cost a microsecond or two a round)
    pl.base = (int)(pl.slots / ctas);
    pl.base = pl.base < 1 ? 1 : pl.base > limit ? (int)limit : pl.base;
    more = ctas * (L_cap >> pl.unit_shift) / 64;
    more = more > 6ll * pl.slots ? 6ll * pl.slots : more;
    if (more < pl.slots || pl.base > 1) more = pl.slots;
    more = (more + per - 1) / per - (long long)B * (pl.base - 1);
    if (more < 0) more = 0;
  }
  if (more > B * (limit - pl.base)) more = B * (limit - pl.base);
  pl.extra = (int)more;
  return pl;
}

template <int D, int RN>
static cudaError_t launch_rows(const CUtensorMap* tmK, const CUtensorMap* tmV, const Kv8AttnParams& p,
                               cudaStream_t stream) {
  using C = RowsCfg<D, RN>;
  cudaError_t err =
      cudaFuncSetAttribute(attn_kv8_rows_kernel<D, RN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (err != cudaSuccess) return err;
  const unsigned grid = (unsigned)(p.n_rt * p.Hkv * (p.B * p.base + p.extra));
  return launch_dependent(attn_kv8_rows_kernel<D, RN>, dim3(grid), dim3(kWarps * 32), C::kSmem, stream, *tmK, *tmV, p);
}

cudaError_t launch_attention_kv8_rows(const CUtensorMap* tmK, const CUtensorMap* tmV, const Kv8AttnParams& p,
                                      cudaStream_t stream) {
  const bool one = p.N * p.G <= 8;
  if (p.d == 128) return one ? launch_rows<128, 1>(tmK, tmV, p, stream) : launch_rows<128, 2>(tmK, tmV, p, stream);
  return one ? launch_rows<64, 1>(tmK, tmV, p, stream) : launch_rows<64, 2>(tmK, tmV, p, stream);
}

cudaError_t launch_attention_kv8_merge(const Kv8AttnParams& p, cudaStream_t stream) {
  // (which requests are split is known on the device only: as many CTAs as run at once, and their warps go on)
  const size_t want = ((size_t)p.B * p.N * p.Hq + 7) / 8;
  const unsigned blocks = (unsigned)(want < 152 * 4 ? want : 152 * 4);
  return p.d == 128 ? launch_dependent(attn_kv8_merge_kernel<128>, dim3(blocks), dim3(256), 0, stream, p)
                    : launch_dependent(attn_kv8_merge_kernel<64>, dim3(blocks), dim3(256), 0, stream, p);
}

}  // namespace spectree
