// K9: tree attention over the 8-bit paged cache, for few rows per KV head (single tokens, short drafts),
// and the merge of its key splits.
//
// Row (node i, query head j) against key s of block c: x = (q . k8) * kscale_c * scale (log2 units), weights
// 2^x, out = sum 2^x vscale_c v8 / sum 2^x.  The V scale is folded into the exponent: with
// y = x + log2(vscale_c) and a running reference m of y, P' = 2^(y - m) multiplies the codes themselves and
// the sum adds P' / vscale_c.  So no code is ever rescaled: e4m3 becomes f16 exactly, on the way from
// shared memory to the registers of m16n8k16 (16 rows of queries; keys, then dimensions, on N).
//
// With 16 rows or fewer a key's 2 d bytes carry 4 d * 16 products at most, far below what the tensor
// cores need to be busy: the kernel is bound by HBM.  What matters is bytes in flight, so every warp
// runs its own ring of TMA boxes of 16 keys and its own softmax state over every fourth box of the
// split, without any barrier between warps; the four states are joined at the end.
#include "common.cuh"
#include "kernels.cuh"
#include "kv8.cuh"
#include "pdl.cuh"

namespace spectree {

namespace {

constexpr int kWarps = 4;
constexpr int kStagesR = 4;      // boxes of 16 keys (K and V) in flight per warp
constexpr int kRowsR = 16;       // (node, head) rows per CTA
constexpr float kLazy = 8.f;     // the reference maximum may be 2^8 behind: P' <= 256, far inside f16

template <int D>
struct RowsCfg {
  static constexpr int kBox = 16 * D;                 // bytes of 16 keys of K (or V)
  static constexpr int kRing = kWarps * kStagesR * 2 * kBox;
  static constexpr int kJoin = kWarps * kRowsR * (D + 4) * 4;  // O of every warp, rows padded
  static constexpr int kSmem = 1024 + (kRing > kJoin ? kRing : kJoin);
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Softmax state of a thread's two rows (g and g + 8 of the tile); m is equal in the four lanes of a row, l
// covers this lane's keys only.
struct RowState {
  float m[2], l[2];
};

// y: this lane's four scores of each row (log2 units, V scale included).  Moves the references when a
// score has run ahead of one, then returns P' and adds it to the sums.  `rebase`, at the first prefix keys
// behind tree keys: references move down as well, as f16 weights need one near their own largest, however
// small the prefix's V scales are (the tree's bf16 weights bear any).
template <int NT>
__device__ __forceinline__ void softmax_step(float (&y)[2][4], RowState& st, float (&o)[NT][4], float inv_vs,
                                             bool rebase) {
  float mx[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) mx[r] = fmaxf(fmaxf(y[r][0], y[r][1]), fmaxf(y[r][2], y[r][3]));
  if (__any_sync(0xffffffffu, rebase || mx[0] > st.m[0] + kLazy || mx[1] > st.m[1] + kLazy)) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float v = mx[r];
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
      // each row by its own scores alone, so that no row's rounding depends on its neighbours
      const float mn = v > st.m[r] + kLazy || (rebase && v > -INFINITY) ? fmaxf(v, st.m[r] - 64.f) : st.m[r];
      const float f = mn == st.m[r] ? 1.f : ex2_approx(st.m[r] - mn);
      st.m[r] = mn;
      st.l[r] *= f;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        o[j][2 * r] *= f;
        o[j][2 * r + 1] *= f;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float mu = st.m[r] == -INFINITY ? 0.f : st.m[r];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[r][i] = ex2_approx(y[r][i] - mu);
    st.l[r] = fmaf((y[r][0] + y[r][1]) + (y[r][2] + y[r][3]), inv_vs, st.l[r]);
  }
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kWarps * 32)
    attn_kv8_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const Kv8AttnParams p) {
  using C = RowsCfg<D>;
  constexpr int RUN = D / 4;   // consecutive dimensions of a query or key row that a lane holds
  constexpr int KS = D / 16;   // k steps of Q K^T
  constexpr int NT = D / 8;    // n tiles of P V
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t s_full[kWarps][kStagesR];
  __shared__ int s_par[kMaxNodes];
  __shared__ uint32_t s_anc[kRowsR][kAncWords];
  __shared__ float s_m[kWarps][kRowsR], s_l[kWarps][kRowsR];
  __shared__ uint32_t s_odd[kAncWords];  // tree keys with an infinity or NaN in their V row
  __shared__ int s_bad;
  const int rt = blockIdx.x, split = blockIdx.y, bg = blockIdx.z;
  const int b = bg / p.Hkv, h = bg - b * p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  long long L;
  int n;
  int err = kv8_counts(p, b, &L, &n);
  const Kv8Split sp = kv8_split(L, p.n_split, p.unit_shift);
  if (split >= sp.n) return;
  const int row0 = rt * kRowsR, rows = p.N * p.G;
  if (tid == 0) {
    s_bad = 0;
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < kStagesR; ++s) mbar_init(&s_full[w][s], 1);
    fence_mbar_init();
  }
  if (tid < kAncWords) s_odd[tid] = 0u;
  for (int i = tid; i < n; i += blockDim.x) {
    const int par = p.parent[(size_t)b * p.N + i];
    s_par[i] = par;
    if (i == 0 ? par != -1 : (par < 0 || par >= i)) err = SPEC_ERR_BAD_TREE;
  }
  {
    const int any = __syncthreads_or(err == SPEC_ERR_BAD_TREE);
    if (any) err = SPEC_ERR_BAD_TREE;
  }
  // the final rows of a request that is refused, or of padded nodes; with several splits the merge does it
  auto orow_of = [&](int row) { return kv8_row(p, b, h, row); };
  auto refuse = [&]() {
    for (int c = tid; c < kRowsR * (D / 8); c += blockDim.x) {
      const int row = row0 + c / (D / 8), e = c % (D / 8);
      if (row >= rows) continue;
      const size_t o = orow_of(row);
      if (sp.n == 1) {
        *reinterpret_cast<uint4*>(p.out + o * D + e * 8) = make_uint4(0, 0, 0, 0);
        if (e == 0 && p.lse) p.lse[o] = 0.f;
      } else if (e == 0) {
        p.part_ml[o * p.n_split + split] = make_float2(0.f, -1.f);
      }
    }
  };
  if (err) {
    if (tid == 0 && rt == 0 && split == 0 && h == 0) set_status(p.dev_status, err);
    refuse();
    return;
  }
  if (row0 >= n * p.G) {  // padded nodes only
    if (sp.n == 1) refuse();
    return;
  }
  // ---- ancestors-or-self of the tile's rows (the last split takes the tree's keys) ----
  const bool tree = split == sp.n - 1;
  if (tree && tid < kRowsR) {
#pragma unroll
    for (int i = 0; i < kAncWords; ++i) s_anc[tid][i] = 0u;
    const int i = kv8_node(p, row0 + tid);
    if (row0 + tid < rows && i < n)
      for (int a = i; a >= 0; a = s_par[a]) s_anc[tid][a >> 5] |= 1u << (a & 31);
  }
  // ---- this warp's boxes: box c0 + warp + 4 i of 16 keys ----
  const int nbox = (int)((L + 15) >> 4);
  const int c0 = (split * sp.steps) << (p.unit_shift - 4);
  const int c1 = min(nbox, c0 + (sp.steps << (p.unit_shift - 4)));
  const int mine = c0 + warp < c1 ? (c1 - c0 - warp + kWarps - 1) / kWarps : 0;
  uint8_t* ring = base + warp * (kStagesR * 2 * C::kBox);
  // table entries and scales of 32 boxes at a time, one per lane: `e` for the boxes being requested, `c`
  // for those being worked on
  int blk_e = -1;
  float ksc_e = 0.f, vsc_e = 1.f, ksc_c = 0.f, vsc_c = 1.f;
  bool bad = false;
  auto fetch = [&](int batch) {
    const int i = batch * 32 + lane;
    blk_e = -1;
    ksc_e = 0.f;
    vsc_e = 1.f;
    if (i < mine) {
      const int slot = (c0 + warp + kWarps * i) * 16;
      const int blk = p.table[(size_t)b * p.max_blocks + (slot >> p.bs_shift)];
      if (blk < 0 || blk >= p.num_blocks) {
        bad = true;
      } else {
        blk_e = blk;
        ksc_e = p.k_scale[(size_t)blk * p.Hkv + h];
        vsc_e = p.v_scale[(size_t)blk * p.Hkv + h];
      }
    }
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
  if (mine > 0) {
    fetch(0);
    ksc_c = ksc_e;
    vsc_c = vsc_e;
    for (int i = 0; i < kStagesR && i < mine; ++i) request(i);
  }
  __syncthreads();  // s_anc

  // ---- queries: rows g and g + 8, dimensions [RUN t, RUN t + RUN), as f16 times a power of two per row
  // that brings the row's largest element to [16, 32); below 2^-18 of it elements lose bits, 2^-29 of it at
  // most
  uint32_t qa[KS][4];
  float qf[2];
  const uint16_t* qrow[2];
  bool has[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = row0 + g + 8 * r;
    has[r] = row < n * p.G;
    qrow[r] = p.q + orow_of(has[r] ? row : row0) * D + RUN * t;
    uint32_t w[RUN / 2];
#pragma unroll
    for (int i = 0; i < RUN / 8; ++i) {
      const uint4 v = has[r] ? *reinterpret_cast<const uint4*>(qrow[r] + 8 * i) : make_uint4(0, 0, 0, 0);
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < RUN / 2; ++i) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // exponent of 2^(4 - floor(log2 mx)), kept where the factor and its reciprocal are normal numbers
    const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 100);
    const float up = __uint_as_float((uint32_t)(127 + 4 - e) << 23);
    qf[r] = __uint_as_float((uint32_t)(127 - 4 + e) << 23) * p.scale_log2;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      qa[s][r] = pack_f16x2(bf16_lo(w[2 * s]) * up, bf16_hi(w[2 * s]) * up);
      qa[s][2 + r] = pack_f16x2(bf16_lo(w[2 * s + 1]) * up, bf16_hi(w[2 * s + 1]) * up);
    }
  }
  float o[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
  RowState st = {{-INFINITY, -INFINITY}, {0.f, 0.f}};

  // ---- the tree's keys, 16 at a time, in bf16 from global memory ----
  if (tree) {
    for (int j0 = (kWarps - 1 - warp) * 16; j0 < n; j0 += kWarps * 16) {
      float y[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int key = j0 + nt * 8 + g;
        const uint16_t* kr = p.k_tree + (((size_t)b * p.N + (key < n ? key : 0)) * p.Hkv + h) * D + RUN * t;
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < RUN / 8; ++i) {
          const uint4 kv = key < n ? *reinterpret_cast<const uint4*>(kr + 8 * i) : make_uint4(0, 0, 0, 0);
          const uint4 z = make_uint4(0, 0, 0, 0);
          const uint4 q0 = has[0] ? *reinterpret_cast<const uint4*>(qrow[0] + 8 * i) : z;
          const uint4 q1 = has[1] ? *reinterpret_cast<const uint4*>(qrow[1] + 8 * i) : z;
          const uint32_t a0[4] = {q0.x, q1.x, q0.y, q1.y}, a1[4] = {q0.z, q1.z, q0.w, q1.w};
          mma_bf16(c, a0, kv.x, kv.y);
          mma_bf16(c, a1, kv.z, kv.w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kk = j0 + nt * 8 + 2 * t + (i & 1), r = i >> 1;
          const bool see = kk < n && ((s_anc[g + 8 * r][kk >> 5] >> (kk & 31)) & 1u);
          y[r][nt * 2 + (i & 1)] = see ? c[i] * p.scale_log2 : -INFINITY;
        }
      }
      softmax_step<NT>(y, st, o, 1.f, false);
      const uint32_t pa[4] = {pack_bf16x2(y[0][0], y[0][1]), pack_bf16x2(y[1][0], y[1][1]),
                              pack_bf16x2(y[0][2], y[0][3]), pack_bf16x2(y[1][2], y[1][3])};
      // V rows 2t, 2t + 1, 2t + 8, 2t + 9 of the chunk, dimensions NT g .. NT g + NT - 1; a row with an
      // infinity or NaN enters as 0 and is added at the end, to the rows that see it only
      uint32_t v[4][NT / 2];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = j0 + 2 * t + (k & 1) + (k >> 1) * 8;
        bool fin = true;
#pragma unroll
        for (int i = 0; i < NT / 8; ++i) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (key < n)
            x = *reinterpret_cast<const uint4*>(p.v_tree + (((size_t)b * p.N + key) * p.Hkv + h) * D + NT * g + 8 * i);
          v[k][4 * i] = x.x; v[k][4 * i + 1] = x.y; v[k][4 * i + 2] = x.z; v[k][4 * i + 3] = x.w;
          fin = fin && bf16_pair_finite(x.x) && bf16_pair_finite(x.y) && bf16_pair_finite(x.z) && bf16_pair_finite(x.w);
        }
        if (!fin) {
          atomicOr(&s_odd[key >> 5], 1u << (key & 31));
#pragma unroll
          for (int i = 0; i < NT / 2; ++i) {
            if ((v[k][i] & 0x7F80u) == 0x7F80u) v[k][i] &= 0xFFFF0000u;
            if ((v[k][i] & 0x7F800000u) == 0x7F800000u) v[k][i] &= 0xFFFFu;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
        mma_bf16(o[j], pa, __byte_perm(v[0][j >> 1], v[1][j >> 1], sel), __byte_perm(v[2][j >> 1], v[3][j >> 1], sel));
      }
    }
  }

  // ---- the prefix ----
  bool ok = true;
  for (int i = 0; i < mine; ++i) {
    const int s = i % kStagesR;
    if ((i & 31) == 0 && i > 0) {  // (the requests have moved on to this batch kStagesR boxes ago)
      ksc_c = ksc_e;
      vsc_c = vsc_e;
    }
    const float ks = kv8_clamp_scale(__shfl_sync(0xffffffffu, ksc_c, i & 31));
    const float vs = kv8_clamp_scale(__shfl_sync(0xffffffffu, vsc_c, i & 31));
    const float lv = __log2f(vs), inv_vs = __fdividef(1.f, vs);
    if (!mbar_wait_bounded(&s_full[warp][s], (i / kStagesR) & 1, &s_bad)) {
      ok = false;
      break;
    }
    const uint8_t* sk = ring + s * 2 * C::kBox;
    const uint8_t* sv = sk + C::kBox;
    const int key0 = (c0 + warp + kWarps * i) * 16;
    const int left = (int)min(16ll, L - key0);  // keys of the box inside the prefix
    float y[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int key = nt * 8 + g;
      uint32_t w[RUN / 4];
      if constexpr (D == 128) {
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const uint4 x = *reinterpret_cast<const uint4*>(sk + key * 128 + (((2 * t + i2) ^ (key & 7)) << 4));
          w[4 * i2] = x.x; w[4 * i2 + 1] = x.y; w[4 * i2 + 2] = x.z; w[4 * i2 + 3] = x.w;
        }
      } else {
        const uint4 x = *reinterpret_cast<const uint4*>(sk + key * 64 + ((t ^ ((key >> 1) & 3)) << 4));
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
      }
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) mma_f16(c, qa[k], codes_f16x2<0>(w[k]), codes_f16x2<1>(w[k]));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int kk = nt * 8 + 2 * t + (e & 1), r = e >> 1;
        y[r][nt * 2 + (e & 1)] = kk < left ? fmaf(c[e], qf[r] * ks, lv) : -INFINITY;
      }
    }
    softmax_step<NT>(y, st, o, inv_vs, tree && i == 0);
    const uint32_t pa[4] = {pack_f16x2(y[0][0], y[0][1]), pack_f16x2(y[1][0], y[1][1]), pack_f16x2(y[0][2], y[0][3]),
                            pack_f16x2(y[1][2], y[1][3])};
    uint32_t v[4][NT / 4];
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
    for (int j = 0; j < NT; j += 2) {
      // bytes j, j + 1 of the four rows: (row 2t, row 2t + 1) pairs for dimensions j and j + 1
      const uint32_t sel = (j & 2) ? 0x7362u : 0x5140u;
      const uint32_t lo = __byte_perm(v[0][j >> 2], v[1][j >> 2], sel);
      const uint32_t hi = __byte_perm(v[2][j >> 2], v[3][j >> 2], sel);
      mma_f16(o[j], pa, codes_f16x2<0>(lo), codes_f16x2<0>(hi));
      mma_f16(o[j + 1], pa, codes_f16x2<1>(lo), codes_f16x2<1>(hi));
    }
  }
  if (!ok) {
    s_bad = 1;
    if (lane == 0) {
      set_status(p.dev_status, SPEC_ERR_TIMEOUT);
      // let the copies in flight land (again with a limit) before shared memory goes
      for (int s = 0; s < kStagesR && s < mine; ++s)
        for (int ph = 0; ph < 2; ++ph) mbar_wait_bounded(&s_full[warp][s], ph, nullptr);
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) {
    s_bad = 1;
    set_status(p.dev_status, SPEC_ERR_CAPACITY);
  }
  // ---- join the four warps' states ----
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 1);
    st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 2);
    if (t == 0) {
      s_m[warp][g + 8 * r] = st.m[r];
      s_l[warp][g + 8 * r] = st.l[r];
    }
  }
  __syncthreads();  // every box has landed and been read: the ring's memory is free
  if (s_bad) {
    refuse();
    return;
  }
  float* join = reinterpret_cast<float*>(base);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float M = s_m[0][g + 8 * r];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, s_m[w][g + 8 * r]);
    const float f = st.m[r] == -INFINITY ? 0.f : ex2_approx(st.m[r] - M);
    // row g + 8 r: dimensions NT (2t) + j and NT (2t + 1) + j
    float* dst = join + (warp * kRowsR + g + 8 * r) * (D + 4) + 2 * NT * t;
#pragma unroll
    for (int j = 0; j < NT; j += 4) {
      *reinterpret_cast<float4*>(dst + j) =
          make_float4(o[j][2 * r] * f, o[j + 1][2 * r] * f, o[j + 2][2 * r] * f, o[j + 3][2 * r] * f);
      *reinterpret_cast<float4*>(dst + NT + j) =
          make_float4(o[j][2 * r + 1] * f, o[j + 1][2 * r + 1] * f, o[j + 2][2 * r + 1] * f, o[j + 3][2 * r + 1] * f);
    }
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
      *reinterpret_cast<float4*>(p.part_o + (orow * p.n_split + split) * D + e * 4) = a;
      if (e == 0) p.part_ml[orow * p.n_split + split] = make_float2(M, l);
    } else {
      const float inv = real ? 1.f / l : 0.f;
      uint2 out = make_uint2(0, 0);
      if (real) out = make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
      *reinterpret_cast<uint2*>(p.out + orow * D + e * 4) = out;
      if (e == 0 && p.lse) p.lse[orow] = real ? (M + log2f(l)) * 0.69314718055994531f : 0.f;
    }
  }
}

// Joins the splits of a row: one warp per output row, lanes over dimensions.
template <int D>
__global__ void __launch_bounds__(256) attn_kv8_merge_kernel(const Kv8AttnParams p) {
  constexpr int EPL = D / 32;
  const int lane = threadIdx.x & 31;
  const size_t orow = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();  // first of all: a launch that ended before the attention's would let its successor overtake it
  if (orow >= (size_t)p.B * p.N * p.Hq) return;
  const int b = (int)(orow / ((size_t)p.N * p.Hq));
  const int i = (int)((orow / p.Hq) % p.N);
  long long L;
  int n;
  kv8_counts(p, b, &L, &n);
  const Kv8Split sp = kv8_split(L, p.n_split, p.unit_shift);
  if (sp.n == 1) return;  // written by the attention kernel itself
  float M = -INFINITY;
  bool bad = i >= n;
  for (int s = lane; s < sp.n; s += 32) {
    const float2 ml = bad ? make_float2(0.f, -1.f) : __ldcg(p.part_ml + orow * p.n_split + s);
    bad |= ml.y < 0.f;
    M = fmaxf(M, ml.x);
  }
  bad = __any_sync(0xffffffffu, bad);
  M = warp_max(M);
  uint16_t* out = p.out + orow * D + lane * EPL;
  if (bad) {
#pragma unroll
    for (int e = 0; e < EPL; ++e) out[e] = 0;
    if (p.lse && lane == 0) p.lse[orow] = 0.f;
    return;
  }
  float l = 0.f, acc[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
  for (int s = 0; s < sp.n; ++s) {
    const float2 ml = __ldcg(p.part_ml + orow * p.n_split + s);
    const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
    l = fmaf(ml.y, f, l);
    const float* src = p.part_o + (orow * p.n_split + s) * D + lane * EPL;
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = fmaf(__ldcg(src + e), f, acc[e]);
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int e = 0; e < EPL; e += 2)
    *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (p.lse && lane == 0) p.lse[orow] = (M + log2f(l)) * 0.69314718055994531f;
}

// ---- host side ------------------------------------------------------------------------------

Kv8AttnPlan plan_attention_kv8(int B, int N, int G, int Hkv, long long L_cap, int num_sms) {
  Kv8AttnPlan pl;
  const int rows = N * G;
  if (rows <= kRowsR) {
    pl.groups = 0;
    pl.unit_shift = 6;
    pl.n_rt = 1;
    // about four rounds of the three CTAs an SM holds, no split below 256 keys
    const long long base = (long long)B * Hkv;
    long long want = ((long long)num_sms * 12 + base - 1) / base;
    const long long most = (L_cap + 255) / 256;
    if (want > most) want = most;
    if (want > 64) want = 64;
    pl.n_split = want < 1 ? 1 : (int)want;
    return pl;
  }
  // two groups of 128 rows per CTA where that still gives every SM work before any splitting
  const long long units2 = (long long)B * Hkv * ((rows + 255) / 256);
  pl.groups = rows > 128 && units2 * 2 >= num_sms ? 2 : 1;
  pl.unit_shift = 7;
  pl.n_rt = (rows + 128 * pl.groups - 1) / (128 * pl.groups);
  // splits: the fewest rounds x (tiles + fixed work of a CTA, about kFixed tiles)
  const long long base = (long long)B * Hkv * pl.n_rt, tiles = (L_cap + 127) / 128;
  constexpr long long kFixed = 5;
  long long best = -1;
  pl.n_split = 1;
  for (int s = 1; s <= 32 && (s == 1 || (tiles + s - 1) / s >= 2); ++s) {
    const long long rounds = (base * s + num_sms - 1) / num_sms;
    const long long cost = rounds * ((tiles + s - 1) / s + kFixed) + (s > 1 ? 3 : 0);
    if (best < 0 || cost < best) {
      best = cost;
      pl.n_split = s;
    }
  }
  return pl;
}

template <int D>
static cudaError_t launch_rows(const CUtensorMap* tmK, const CUtensorMap* tmV, const Kv8AttnParams& p,
                               cudaStream_t stream) {
  using C = RowsCfg<D>;
  cudaError_t err =
      cudaFuncSetAttribute(attn_kv8_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (err != cudaSuccess) return err;
  attn_kv8_rows_kernel<D><<<dim3(p.n_rt, p.n_split, p.B * p.Hkv), kWarps * 32, C::kSmem, stream>>>(*tmK, *tmV, p);
  return cudaGetLastError();
}

cudaError_t launch_attention_kv8_rows(const CUtensorMap* tmK, const CUtensorMap* tmV, const Kv8AttnParams& p,
                                      cudaStream_t stream) {
  return p.d == 128 ? launch_rows<128>(tmK, tmV, p, stream) : launch_rows<64>(tmK, tmV, p, stream);
}

cudaError_t launch_attention_kv8_merge(const Kv8AttnParams& p, cudaStream_t stream) {
  const unsigned blocks = (unsigned)(((size_t)p.B * p.N * p.Hq + 7) / 8);
  return p.d == 128 ? launch_dependent(attn_kv8_merge_kernel<128>, dim3(blocks), dim3(256), 0, stream, p)
                    : launch_dependent(attn_kv8_merge_kernel<64>, dim3(blocks), dim3(256), 0, stream, p);
}

}  // namespace spectree
