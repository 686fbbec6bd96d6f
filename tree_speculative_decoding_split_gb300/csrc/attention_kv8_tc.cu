// K9t: tree attention over the 8-bit paged cache on tcgen05 tensor cores, for many rows per KV head.
//
// tcgen05 has no product of a 16-bit with an 8-bit operand.  So
//   S = Q K^T: the keys' codes feed the tensor cores as they lie, and Q enters as the sum of two e4m3 numbers
//   (scaled per row so that its largest element lies in [128, 256): hi its first four significant bits, lo the
//   rest, together q to 2^-17 of that largest): S = Qhi K^T + Qlo K^T at twice the 16-bit rate, the same tensor
//   time as 16-bit operands.
//   O += P V: splitting the weights the same way cost more instructions in the softmax (six per pair) than
//   anything else there, so here the codes of V become f16 instead (exactly, by two warps of their own, once
//   per tile for all rows), and P = 2^(y - m) is f16 (y: the score in log2 units with the V scale folded in, as
//   in the few-rows kernel).
// Accumulation is float32 (measured: 1e-7 relative for e4m3 products, as for bf16).  The tree's own keys (at
// most 255, bf16) come first, as bf16 tiles with bf16 Q and P as a pair of bf16 numbers (to 2^-16; single ones made
// the output of a row that the tree outweighs 0.0022 wrong instead of 0.0017, and are four tiles' work at most).
//
// One CTA owns (request, KV head, key split, NG x 128 rows).  Bound: per 128-key tile and 128 rows the
// tensor pipe takes 512 (S) + 512 (P V) cycles; the two groups fill each other's softmax.  TMEM: O 128
// columns and S 128 per group, 512 in all with two; P lies over the S it came from, so a group's S(t + 1) is
// issued when its P V(t) is done.  (With one group S has two buffers.)
//   warp 0     TMA producer: K and V rings of 128-key tiles (one box per block and tensor, issued by as many
//              lanes), the tile's scales; first of all it works out the CTA's share of the batch;
//   warp 1     MMA issuer;
//   warps 2, 3 V tiles to f16;
//   warps 4..  softmax, eight warps per group: two threads own a row (a TMEM lane), 64 keys of a tile each.
//              Both use the row's reference; whether one has to move is one barrier's OR per tile.  Moving it
//              and masking the tile that ends the prefix have loops of their own, which leaves the tiles' own short
//              (4 trees of 255 nodes 1880 -> 1861 us).
// Measured (graph replay): 4 trees of 255 nodes, 64 query heads on 8, lengths up to 128K, 1906 us = 1437 TFLOP/s,
// 0.74 of a large bf16 product's rate; a tile of both groups takes 3.3 K cycles for 2 K of tensor work.  32 trees of
// 63 nodes at 4K 140 us = 966 TFLOP/s: 256 CTAs on 152 SMs are 1.7 rounds, and about 30 K of a CTA's 140 K cycles go
// to its first two tiles and its last rows, which nothing overlaps.  8 trees of 127 nodes, d 64, 58 us.
// Tried and slower (63-node trees, batch 32 at 4K, when this stood at 160 us): P as e4m3 pairs with 128 keys a
// thread, four warps per group and a row maximum ahead of the weights, 238 us; with one S buffer shared by both groups
// and all descriptors in uniform registers, 203 us; with two threads per row, 211 us.  Four trees of 255 nodes, at
// 2112 us: two issuing warps with the V tiles converted by the softmax warps, 2567 us; waits with a suspend-time hint
// 2942 us, waits that only poll 3144 us.  The tree's tiles eight keys at a time in a rolled loop: 60 us for the 8
// trees of 127 nodes instead of 57.
#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"
#include "kv8.cuh"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace spectree {

namespace {

constexpr int kKT8 = 128;        // keys per prefix tile
constexpr int kTT = 64;          // keys per tree tile (bf16: the same bytes)
constexpr int kGR8 = 128;        // rows per group
constexpr int kKS = 3, kVS = 2;  // ring depths: K codes, V codes
constexpr int kV16 = 2;          // V tiles in f16
constexpr int kCS = 8;           // stages of the scales
// A row's reference m is an integer.  It moves when sixteen neighbouring weights sum to more than 2^15, well
// inside f16; a new one puts the row's largest weight into (1/2, 1].  So rows rarely move (every move costs a
// pass over O), and a weight is exact to 11 bits or to 2^-24 of the largest.
constexpr float kTop = 32768.f;

template <int D, int NG>
struct TcCfg {
  static constexpr int kThreads = 128 + 256 * NG;
  static constexpr int kQ = kGR8 * D * 2;      // Q bytes per group: bf16, or e4m3 hi then lo
  static constexpr int kSlot = kKT8 * D;       // ring slot
  static constexpr int kNB = NG == 2 ? 1 : 2;  // S (and P) buffers per group
  static constexpr int kColO = 0, kColS = NG * 128;
  static constexpr int kNanc = (kMaxNodes + 1) * kAncWords * 4;
  static constexpr int kTile16 = kKT8 * D * 2; // a V tile in f16
  static constexpr int kRing = NG * kQ + (kKS + kVS) * kSlot + kV16 * kTile16;
  static constexpr int kSmem = 1024 + kRing + kNanc + kCS * 8 * 16;
  static constexpr int kORow = D * 4 + 16;     // epilogue rows in shared memory, padded
  static_assert(kGR8 * NG * kORow <= kRing, "O staging does not fit");
};

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptors with type fields 0: D fp32, A and B e4m3 (kind::f8f6f4) or f16 (kind::f16).
__host__ __device__ constexpr uint32_t idesc_type0_f32(int M, int N, int b_mn_major) {
  return (1u << 4) | ((uint32_t)(b_mn_major ? 1 : 0) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Descriptor of an e4m3 tile of D-byte rows, swizzled over 128 (D = 128) or 64 bytes (D = 64); 8-row groups
// follow one another densely.
template <int D>
__device__ __forceinline__ uint64_t sdesc_kv8(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((8 * D) >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)(D == 128 ? 2 : 4) << 61;
  return d;
}
// Byte offset of 16-byte chunk ch of row r in such a tile.
template <int D>
__device__ __forceinline__ uint32_t kv8_off(int r, int ch) {
  return D == 128 ? (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
}
// ... and of chunk ch of row r in a 16-bit tile of `rows` rows: halves of 64 columns, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile16_off(int r, int ch, int rows) {
  return (uint32_t)((ch >> 3) * rows * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// The value's first four significant bits.
__device__ __forceinline__ float head4(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFF00000u); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two e4m3 codes (the low or high half of `w`) to f16, exactly.
template <int HALF>
__device__ __forceinline__ uint32_t kv8_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (HALF == 0)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
// Named barrier of `count` threads that returns the OR of their predicates.
__device__ __forceinline__ bool bar_or(int id, int count, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(id), "r"(count), "r"((uint32_t)pred)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ bool finite2(uint32_t w) {
  return (w & 0x7F80u) != 0x7F80u && (w & 0x7F800000u) != 0x7F800000u;
}

}  // namespace

template <int D, int NG>
__global__ void __launch_bounds__(TcCfg<D, NG>::kThreads, 1)
    attn_kv8_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CUtensorMap tmKt, const __grid_constant__ CUtensorMap tmVt,
                       const Kv8AttnParams p) {
  using C = TcCfg<D, NG>;
  constexpr int kRowsCta = kGR8 * NG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  uint8_t* sK = sQ + NG * C::kQ;
  uint8_t* sV = sK + kKS * C::kSlot;
  uint8_t* sV16 = sV + kVS * C::kSlot;
  uint32_t* s_nanc = reinterpret_cast<uint32_t*>(sV16 + kV16 * C::kTile16);  // [node][word] ancestors-or-self
  float4* s_cst = reinterpret_cast<float4*>(s_nanc + (kMaxNodes + 1) * kAncWords);  // [stage][16-key group]
  __shared__ uint64_t kfull[kKS], kempty[kKS], vfull[kVS], vempty[kVS], v16empty[kV16];
  // per group, and per buffer where there are two (one barrier could be two phases on)
  __shared__ uint64_t sfull[NG][C::kNB], pfull[NG][2], ofull[NG];
  __shared__ float s_qf[NG][kGR8];
  __shared__ float s_x[NG][2][kGR8];  // a row's threads tell each other their largest score; at the end, their sums
  __shared__ uint32_t s_w[NG][2][4];  // ... and which of the warp's rows move
  __shared__ uint64_t s_drained;
  __shared__ uint64_t s_pread[NG];  // P read by its product
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_bad, s_kissued, s_vissued;
  __shared__ int s_par[kMaxNodes];
  __shared__ uint32_t s_odd[kAncWords];
  __shared__ int s_any_odd;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ Kv8Work s_work;
  Kv8Work sp = kv8_own(p);
  if (warp == 1) {
    if (lane == 0) {
      for (int s = 0; s < kKS; ++s) {
        mbar_init(&kfull[s], 1);
        mbar_init(&kempty[s], 1);
      }
      for (int s = 0; s < kVS; ++s) {
        mbar_init(&vfull[s], 1);
        mbar_init(&vempty[s], 2);
      }
      for (int s = 0; s < kV16; ++s) mbar_init(&v16empty[s], 1);
      for (int g = 0; g < NG; ++g) {
        for (int i = 0; i < C::kNB; ++i) mbar_init(&sfull[g][i], 1);
        // a tile's weights are there; for group 0 also its V, and the keys of the scores that follow
        for (int i = 0; i < 2; ++i) mbar_init(&pfull[g][i], g == 0 ? 10 : 8);
        mbar_init(&ofull[g], 1);
        mbar_init(&s_pread[g], 1);
      }
      mbar_init(&s_drained, 1);
      s_abort = 0;
      s_bad = 0;
      s_any_odd = 0;
      s_kissued = 0;
      s_vissued = 0;
      fence_mbar_init();
    }
  }
  pdl_wait();  // what comes before in the stream may still be ending: nothing of it is read ahead of this
  pdl_launch_dependents();  // the merge may be launched
  // The queries, 16 bytes a lane, whole rows side by side, on their way while warp 0 works out the cut (where the
  // CTA's place in the grid says which).  As bf16 they lie where V tiles in f16 will: only the tree's scores read
  // them there, the prefix's take them as e4m3 hi and lo from sQ.
  constexpr int kQPer = kGR8 * (D / 8) / 256, kQStep = 256 / (D / 8);
  const int q_g = (warp - 4) >> 3, q_r0 = ((tid - 128) & 255) / (D / 8), q_ch = tid % (D / 8);
  uint8_t* q16 = sV16 + q_g * C::kQ;
  int par = -1;  // of node tid - 128
  auto fetch_q = [&]() {
    if (warp < 4) return;
    if (tid - 128 < p.N) par = p.parent[(size_t)sp.b * p.N + tid - 128];
#pragma unroll 2
    for (int k = 0; k < kQPer; ++k) {
      const int r = q_r0 + k * kQStep, row = sp.rt * kRowsCta + q_g * kGR8 + r;
      const bool in = row < p.N * p.G;  // (zeros otherwise)
      const uint16_t* from = p.q + kv8_row(p, sp.b, sp.h, in ? row : 0) * D + q_ch * 8;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(q16 + tile16_off(r, q_ch, kGR8))),
                   "l"(from), "r"(in ? 16 : 0)
                   : "memory");
    }
  };
  auto have_q = [&]() { asm volatile("cp.async.wait_all;" ::: "memory"); };
  const bool own = sp.b >= 0;
  if (own) fetch_q();
  if (warp == 0) {
    const Kv8Work w = kv8_begin(p, sp);
    if (lane == 0) s_work = w;
  }
  __syncthreads();
  sp = s_work;
  if (sp.b < 0) {  // a unit that its request does not use
    have_q();
    return;
  }
  if (!own) fetch_q();
  // ---- a CTA's tiles: the tree's (in the last split) and then keys [k0, k1) of the prefix ----
  struct Tiles {
    bool tree;
    int b, h;
    long long k0, k1;
    int Tt, T;
  };
  auto tiles_of = [&](const Kv8Work& w) {
    Tiles x;
    x.tree = w.split == w.n - 1;
    x.b = w.b;
    x.h = w.h;
    x.k0 = ((long long)w.split * w.steps) << p.unit_shift;
    x.k1 = min(w.L, x.k0 + ((long long)w.steps << p.unit_shift));
    x.Tt = x.tree ? (w.nodes + kTT - 1) / kTT : 0;
    x.T = x.Tt + (x.k1 > x.k0 ? (int)((x.k1 - x.k0 + kKT8 - 1) / kKT8) : 0);
    return x;
  };
  // ---- TMA: lane i < 128 / box of warp 0 takes box i of a tile; the first tiles are on their way while the tree is
  // checked ----
  const int box = min(p.bs, kKT8), nbox = kKT8 / box;
  const int out_z = p.num_blocks * p.Hkv;  // behind the map: reads as zeros
  // slot of this lane's box in prefix tile u, or -1 when it lies behind the split's keys
  auto slot_of = [&](const Tiles& w, int u) -> long long {
    const long long s = w.k0 + (long long)u * kKT8 + lane * box;
    return lane < nbox && s < w.k1 ? s : -1;
  };
  auto entry = [&](const Tiles& w, int u) -> int {
    const long long s = slot_of(w, u);
    return s >= 0 ? p.table[(size_t)w.b * p.max_blocks + (s >> p.bs_shift)] : -1;
  };
  // the block of tile u is loaded two tiles ahead and its scales one tile ahead of its requests
  int blk0 = -1, blk1 = -1;
  float ks0 = 0.f, vs0 = 0.f;
  auto scales = [&](const Tiles& w, int blk, float* ks, float* vs) {
    *ks = 0.f;
    *vs = 0.f;
    if (blk >= 0 && blk < p.num_blocks) {
      *ks = p.k_scale[(size_t)blk * p.Hkv + w.h];
      *vs = p.v_scale[(size_t)blk * p.Hkv + w.h];
    }
  };
  auto produce = [&](const Tiles& w, int t0, int t1) -> bool {
    for (int t = t0; t < t1; ++t) {
      const int ks = t % kKS, vs = t % kVS, u = t - w.Tt;
      int blk2 = -1;
      float ks1 = 0.f, vs1 = 0.f;
      if (u >= 0) {
        if (u == 0) scales(w, blk0, &ks0, &vs0);
        scales(w, blk1, &ks1, &vs1);
        blk2 = entry(w, u + 2);
      }
      const bool got = lane == 0 ? mbar_wait_bounded(&kempty[ks], ((t / kKS) & 1) ^ 1, &s_abort) : true;
      if (!__shfl_sync(0xffffffffu, got, 0)) return false;
      uint8_t* dk = sK + ks * C::kSlot;
      uint8_t* dv = sV + vs * C::kSlot;
      int y = 0, z = out_z;
      if (u >= 0) {
        const long long s = slot_of(w, u);
        if (s >= 0) {
          if (blk0 >= 0 && blk0 < p.num_blocks) {
            y = (int)(s & (p.bs - 1));
            z = blk0 * p.Hkv + w.h;
          } else {
            s_bad = 1;
          }
        }
      }
      // the copies first; the barrier's own arrival follows the scales, which the tile's readers need as well
      if (u < 0) {
        if (lane < D / 64) tma_load_4d(dk + lane * kTT * 128, &tmKt, &kfull[ks], lane * 64, w.h, t * kTT, w.b);
      } else if (lane < nbox) {
        tma_load_3d(dk + lane * box * D, &tmK, &kfull[ks], 0, y, z);
        // scales of the box's 16-key groups: K scale, log2 and reciprocal of the V scale
        const float sv = kv8_clamp_scale(vs0);
        const float4 c = make_float4(kv8_clamp_scale(ks0), __log2f(sv), __fdividef(1.f, sv), 0.f);
        for (int j = 0; j < box / 16; ++j) s_cst[(t % kCS) * 8 + lane * (box / 16) + j] = c;
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_expect_tx(&kfull[ks], C::kSlot);
        s_kissued = t + 1;
      }
      const bool gotv = lane == 0 ? mbar_wait_bounded(&vempty[vs], ((t / kVS) & 1) ^ 1, &s_abort) : true;
      if (!__shfl_sync(0xffffffffu, gotv, 0)) return false;
      if (lane == 0) {
        mbar_arrive_expect_tx(&vfull[vs], C::kSlot);
        s_vissued = t + 1;
      }
      __syncwarp();
      if (u < 0) {
        if (lane < D / 64) tma_load_4d(dv + lane * kTT * 128, &tmVt, &vfull[vs], lane * 64, w.h, t * kTT, w.b);
      } else {
        if (lane < nbox) tma_load_3d(dv + lane * box * D, &tmV, &vfull[vs], 0, y, z);
        blk0 = blk1;
        blk1 = blk2;
        ks0 = ks1;
        vs0 = vs1;
      }
    }
    return true;
  };
  int pre = 0;  // tiles asked for ahead of the barrier
  bool bad_tree = false;
  if (warp == 0) {
    const Tiles w = tiles_of(sp);
    blk0 = entry(w, 0);
    blk1 = entry(w, 1);
    if (!sp.err) pre = min(w.T, kVS);
    produce(w, 0, pre);
  } else if (warp == 1) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  } else if (warp == 2) {
    if (lane < kAncWords) s_odd[lane] = 0u;
  } else if (warp >= 4) {
    if (warp < 12) {
      const int i = tid - 128;  // (256 threads, at most 255 nodes)
      if (i < sp.nodes) {
        s_par[i] = par;
        bad_tree = i == 0 ? par != -1 : (par < 0 || par >= i);
      }
      if (!bar_or(10, 256, bad_tree) && i < sp.nodes) {  // ancestors-or-self
        uint32_t* w = s_nanc + i * kAncWords;
#pragma unroll
        for (int j = 0; j < kAncWords; ++j) w[j] = 0u;
        for (int a = i; a >= 0; a = s_par[a]) w[a >> 5] |= 1u << (a & 31);
      }
    }
    have_q();
    uint8_t* q8 = sQ + q_g * C::kQ;
#pragma unroll 2
    for (int k = 0; k < kQPer; ++k) {  // (this thread's own chunks)
      const int r = q_r0 + k * kQStep;
      const uint4 v = *reinterpret_cast<const uint4*>(q16 + tile16_off(r, q_ch, kGR8));
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
      float f[8], mx = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(x[j] << 16);
        f[2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
        mx = max3(mx, fabsf(f[2 * j]), fabsf(f[2 * j + 1]));
      }
#pragma unroll
      for (int o = 1; o < D / 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      // (both powers of two below are normal numbers up to the exponent 128 of an infinity; at the lower end a row's
      // largest element counts as 2^-100 at least)
      const int e = max((int)(__float_as_uint(mx) >> 23) - 127, -100);
      const float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);  // largest element into [128, 256)
      if (q_ch == 0) s_qf[q_g][r] = __uint_as_float((uint32_t)(127 - 7 + e) << 23) * p.scale_log2;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= up;
      uint8_t* to = q8 + kv8_off<D>(r, q_ch >> 1) + (q_ch & 1) * 8;
      *reinterpret_cast<uint2*>(to) = make_uint2(e4m3x4(head4(f[0]), head4(f[1]), head4(f[2]), head4(f[3])),
                                                 e4m3x4(head4(f[4]), head4(f[5]), head4(f[6]), head4(f[7])));
      *reinterpret_cast<uint2*>(to + kGR8 * D) =
          make_uint2(e4m3x4(f[0] - head4(f[0]), f[1] - head4(f[1]), f[2] - head4(f[2]), f[3] - head4(f[3])),
                     e4m3x4(f[4] - head4(f[4]), f[5] - head4(f[5]), f[6] - head4(f[6]), f[7] - head4(f[7])));
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  bad_tree = __syncthreads_or(bad_tree);
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const Kv8Work w = s_work;
  const int b = w.b, h = w.h, rt = w.rt, row0 = rt * kRowsCta, rows = p.N * p.G;
  auto orow_of = [&](int row) { return kv8_row(p, b, h, row); };
  // rows of a refused request or of padded nodes; with several splits the merge writes them
  auto refuse = [&]() {
    for (int c = tid; c < kRowsCta * (D / 8); c += C::kThreads) {
      const int row = row0 + c / (D / 8), e = c % (D / 8);
      if (row >= rows) continue;
      const size_t o = orow_of(row);
      if (w.n == 1) {
        *reinterpret_cast<uint4*>(p.out + o * D + e * 8) = make_uint4(0, 0, 0, 0);
        if (e == 0 && p.lse) p.lse[o] = 0.f;
      } else if (e == 0) {
        p.part_ml[w.part + (row - row0)] = make_float2(0.f, -1.f);
      }
    }
  };
  const Tiles own_tiles = tiles_of(w);
  const bool tree = own_tiles.tree;
  const long long k0 = own_tiles.k0, k1 = own_tiles.k1;
  const int n = w.nodes, Tt = own_tiles.Tt, T = own_tiles.T;
  const int err = bad_tree ? SPEC_ERR_BAD_TREE : w.err;
  if (err || row0 >= n * p.G) {  // refused, or padded nodes only (with several splits the merge zeroes those)
    if (err && tid == 0 && rt == 0 && w.split == 0 && h == 0) set_status(p.dev_status, err);
    if (err || w.n == 1) refuse();
    if (tid == 0)  // the copies land first
      for (int t = 0; t < pre; ++t) {
        mbar_wait_bounded(&kfull[t], 0, nullptr);
        mbar_wait_bounded(&vfull[t], 0, nullptr);
      }
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }
  // register shares of the warpgroups (two groups): 64 + 4 x 104 within the 5 x 96 the block was launched with
  if (warp < 4) {
    if constexpr (NG == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
    // ---- TMA producer, from where the first tiles ended ----
      if (!produce(own_tiles, pre, T) && lane == 0) {
        s_abort = 1;
        set_status(p.dev_status, SPEC_ERR_TIMEOUT);
      }
    } else if (warp == 1) {
    // ---- MMA issuer ----
    // The whole warp runs the loop, so that addresses and descriptors stay in uniform registers, and one
    // elected lane issues: beside two busy softmax warps on the same scheduler, a lane that computed its
    // descriptors in vector registers took 160 cycles for an MMA of 64.
    constexpr uint32_t idS8 = idesc_type0_f32(kGR8, kKT8, 0), idP16 = idesc_type0_f32(kGR8, D, 1);
    constexpr uint32_t idSt = idesc_bf16_f32(kGR8, kTT, 0), idPt = idesc_bf16_f32(kGR8, D, 1);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t sq0 = __shfl_sync(0xffffffffu, smem_u32(sQ), 0);
    const uint32_t sk0 = sq0 + NG * C::kQ, sv0 = sk0 + kKS * C::kSlot;
    const bool leader = elect_one();
    // Descriptors: the upper word is constant per layout, the lower one an address in 16-byte units, so that an
    // MMA's operands are a base and a constant.
    const uint32_t q16 = (sq0 & 0x3FFFFu) >> 4, k16 = (sk0 & 0x3FFFFu) >> 4, v16 = (sv0 & 0x3FFFFu) >> 4;
    const uint64_t hi8 = sdesc_kv8<D>(0), hi16 = sdesc_sw128(0, 0, 1024);
    const uint64_t hiVt = sdesc_sw128(0, kTT * 128, 1024), hiV = sdesc_sw128(0, kKT8 * 128, 1024);
    auto wait = [&](uint64_t* bar, uint32_t parity) {  // (one instruction for the warp: its lanes agree)
      return mbar_try_wait(bar, parity) || mbar_wait_bounded(bar, parity, &s_abort);
    };
    int kst = 0;  // ring stage of the next S tile
    auto issue_s = [&](auto tree_tile, int t, int g) {
      const uint32_t ts = tm + C::kColS + (NG == 2 ? g : t % C::kNB) * 128;
      const uint32_t qa = (tree_tile.value ? v16 + (kVS * C::kSlot >> 4) : q16) + g * (C::kQ >> 4);
      const uint32_t ka = k16 + kst * (C::kSlot >> 4);
      if (leader) {
        if constexpr (tree_tile.value) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16(ts, hi16 | (qa + (kk >> 2) * (kGR8 * 8) + (kk & 3) * 2),
                      hi16 | (ka + (kk >> 2) * (kTT * 8) + (kk & 3) * 2), idSt, kk > 0);
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {  // hi, then lo
            const int k = kk % (D / 32);
            umma_f8(ts, hi8 | (qa + (kk / (D / 32)) * (kGR8 * D / 16) + k * 2), hi8 | (ka + k * 2), idS8, kk > 0);
          }
        }
        umma_commit(&sfull[g][t % C::kNB]);
        if (g == NG - 1) umma_commit(&kempty[kst]);
      }
      if (g == NG - 1 && ++kst == kKS) kst = 0;
    };
    auto issue_pv = [&](auto tree_tile, int t, int g) {
      const uint32_t pt = tm + C::kColS + (NG == 2 ? g : t % C::kNB) * 128, ot = tm + C::kColO + g * 128;
      if (leader) {
        if constexpr (tree_tile.value) {
          const uint32_t va = v16 + (t % kVS) * (C::kSlot >> 4);
#pragma unroll
          for (int kk = 0; kk < kTT / 16; ++kk)
#pragma unroll
            for (int part = 0; part < 2; ++part)  // the weights' two parts
              umma_bf16_tmem_a(ot, pt + (kk >> 1) * 64 + part * 16 + (kk & 1) * 8, hiVt | (va + kk * 128), idPt,
                               t > 0 || kk > 0 || part > 0);
        } else {
          const uint32_t va = v16 + (kVS * C::kSlot >> 4) + (t % kV16) * (C::kTile16 >> 4);
#pragma unroll
          for (int kk = 0; kk < kKT8 / 16; ++kk)  // each half's weights lie over its own scores
            umma_bf16_tmem_a(ot, pt + (kk >> 2) * 64 + (kk & 3) * 8, hiV | (va + kk * 128), idP16, t > 0 || kk > 0);
        }
        // (with one S buffer the next scores' commit says so too)
        if (C::kNB > 1 || t == T - 1) umma_commit(&ofull[g]);
        if (g == NG - 1) {
          umma_commit(&v16empty[t % kV16]);
          if constexpr (tree_tile.value) {  // a tree tile's V was read where it landed
            umma_commit(&vempty[t % kVS]);
            umma_commit(&vempty[t % kVS]);
          }
        }
      }
    };
    // P V(t), and when that is done the buffer's next scores, which overwrite P: tensor instructions keep their order for
    // sure only where they have one accumulator and one shape (4 trees of 255 nodes 1862 us without the wait, 1906 with it; 32
    // of 63 nodes 136 and 140, 8 of 127 nodes with d 64 60.5 and 58.5)
    auto step = [&](auto pv_tree, auto s_tree, int t) -> bool {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (!wait(&pfull[g][t & 1], (t >> 1) & 1)) return false;
        tc_fence_after();
        issue_pv(pv_tree, t, g);
        if (t + C::kNB < T) {
          if (leader) umma_commit(&s_pread[g]);
          if (!wait(&s_pread[g], t & 1)) return false;
          issue_s(s_tree, t + C::kNB, g);
        }
      }
      return true;
    };
    using Yes = std::true_type;
    using No = std::false_type;
    auto run = [&]() -> bool {
      for (int t = 0; t < C::kNB && t < T; ++t) {
        if (!wait(&kfull[t % kKS], 0)) return false;
        for (int g = 0; g < NG; ++g) {
          tc_fence_after();
          if (t < Tt) issue_s(Yes(), t, g); else issue_s(No(), t, g);
        }
      }
      int t = 0;
      for (; t < Tt - C::kNB; ++t)
        if (!step(Yes(), Yes(), t)) return false;
      for (; t < Tt; ++t)
        if (!step(Yes(), No(), t)) return false;
      for (; t < T; ++t)
        if (!step(No(), No(), t)) return false;
      return true;
    };
    const bool ok = run();
    if (leader) {
      if (!ok) {
        s_abort = 1;
        set_status(p.dev_status, SPEC_ERR_TIMEOUT);
      }
      umma_commit(&s_drained);  // every MMA of this CTA
      mbar_wait_bounded(&s_drained, 0, nullptr);
    }
    } else {
      // ---- V tiles to f16 (warps 2, 3) ----
      bool ok = true;
      const int ct = tid - 64;
      for (int t = 0; t < T; ++t) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&vfull[t % kVS], (t / kVS) & 1, &s_abort) &&
                                         mbar_wait_bounded(&v16empty[t % kV16], ((t / kV16) & 1) ^ 1, &s_abort));
        if (!ok) break;
        // the tree's last scores are done with the bf16 queries (waited for ahead of the word that lets the next ones
        // begin, which would turn the barrier's phase over)
        if (t == Tt - 1) {
          for (int g = 0; g < NG && ok; ++g)
            ok = mbar_wait_bounded(&sfull[g][t % C::kNB], (t / C::kNB) & 1, &s_abort);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* src = sV + (t % kVS) * C::kSlot;
        if (t < Tt) {
          // a tree tile stays bf16; elements that are no finite numbers become 0 and their rows are noted.  Whether
          // this thread has any: the sum of all its elements times zero is NaN.
          constexpr int kChunks = kTT * (D / 8) / 64;
          __nv_bfloat162 odd = __floats2bfloat162_rn(0.f, 0.f);
          const __nv_bfloat162 zero = odd;
#pragma unroll 4
          for (int i = 0; i < kChunks; ++i) {
            const int c = ct + i * 64;
            const uint4 x = *reinterpret_cast<const uint4*>(src + tile16_off(c / (D / 8), c % (D / 8), kTT));
            odd = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.x), zero, odd);
            odd = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.y), zero, odd);
            odd = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.z), zero, odd);
            odd = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.w), zero, odd);
          }
          const bool any = !(__low2float(odd) == 0.f && __high2float(odd) == 0.f);
#pragma unroll 1
          for (int i = 0; i < kChunks && any; ++i) {
            const int c = ct + i * 64, r = c / (D / 8), key = t * kTT + r;
            uint4* at = reinterpret_cast<uint4*>(src + tile16_off(r, c % (D / 8), kTT));
            uint4 x = *at;
            if (finite2(x.x) && finite2(x.y) && finite2(x.z) && finite2(x.w)) continue;
            if (key < n) {
              atomicOr(&s_odd[key >> 5], 1u << (key & 31));
              s_any_odd = 1;
            }
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if ((w[j] & 0x7F80u) == 0x7F80u) w[j] &= 0xFFFF0000u;
              if ((w[j] & 0x7F800000u) == 0x7F800000u) w[j] &= 0xFFFFu;
            }
            *at = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          // 16 codes of a row -> two 16-byte chunks of the f16 tile (halves of 64 columns).  The lanes of the
          // second half take the row's neighbour, so that eight lanes meet eight bank groups in every access;
          // a thread's rows are whole swizzle periods apart, so all its addresses are one base plus a constant.
          constexpr int kSteps = kKT8 * (D / 16) / 64, kSrcStep = 1024, kDstStep = D == 128 ? 1024 : 2048;
          const int ch = ct % (D / 16), r0 = ct / (D / 16), r = D == 128 ? r0 ^ (ch >> 2) : r0;
          const uint8_t* from = src + kv8_off<D>(r, ch);
          uint8_t* to_a = sV16 + (t % kV16) * C::kTile16 + tile16_off(r, 2 * ch, kKT8);
          uint8_t* to_b = sV16 + (t % kV16) * C::kTile16 + tile16_off(r, 2 * ch + 1, kKT8);
          const int left = (int)min((long long)kKT8, k1 - (k0 + (long long)(t - Tt) * kKT8));
          auto convert = [&](int i, uint4 x) {
            *reinterpret_cast<uint4*>(to_a + i * kDstStep) =
                make_uint4(kv8_f16x2<0>(x.x), kv8_f16x2<1>(x.x), kv8_f16x2<0>(x.y), kv8_f16x2<1>(x.y));
            *reinterpret_cast<uint4*>(to_b + i * kDstStep) =
                make_uint4(kv8_f16x2<0>(x.z), kv8_f16x2<1>(x.z), kv8_f16x2<0>(x.w), kv8_f16x2<1>(x.w));
          };
          if (left == kKT8) {
#pragma unroll 4
            for (int i = 0; i < kSteps; ++i) convert(i, *reinterpret_cast<const uint4*>(from + i * kSrcStep));
          } else {  // slots behind the prefix may hold anything and become 0
#pragma unroll 1
            for (int i = 0; i < kSteps; ++i) {
              const uint4 x = *reinterpret_cast<const uint4*>(from + i * kSrcStep);
              convert(i, r + i * (64 / (D / 16)) < left ? x : make_uint4(0, 0, 0, 0));
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && t >= Tt) mbar_arrive(&vempty[t % kVS]);
        // with V goes the word that the keys of the next scores are there: the issuer has one wait per group
        const int tn = t + C::kNB;
        if (tn < T) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&kfull[tn % kKS], (tn / kKS) & 1, &s_abort));
          if (!ok) break;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[0][t & 1]);
      }
      if (!ok && lane == 0) {
        s_abort = 1;
        set_status(p.dev_status, SPEC_ERR_TIMEOUT);
      }
    }
  } else {
    if constexpr (NG == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ---- softmax ----
    const int g = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, q4 = warp & 3;
    const int rl = q4 * 32 + lane, rr = g * kGR8 + rl, row = row0 + rr;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tmem + C::kColS + (NG == 2 ? g : 0) * 128 + lane_off;
    const uint32_t tO = tmem + C::kColO + g * 128 + lane_off;
    const bool live = row < n * p.G;
    const float qf = s_qf[g][rl];  // undoes the row's scaling, with the softmax scale in log2 units
    // The pair's barriers below have no limit, and either warp's waits may give up.  So no warp leaves the tiles
    // early: it says that it gave up, and goes through the rest with its pair (no wait takes long then), for nothing.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, &s_abort))) s_abort = 1;
    };
    float m = -INFINITY, l = 0.f;  // the row's reference (P = 2^(y - m)), and the sum over this thread's keys
    const uint32_t* anc = s_nanc + (live ? kv8_node(p, row) : 0) * kAncWords;
    const int pair = 2 + g * 4 + q4;  // named barrier of the two warps that share rows
    // Moves the references of the rows that ask for it in either of their threads (`ask`, with the largest of
    // the thread's scores in `top`); O and the sums follow.  Also down, at the first tile behind the tree's
    // (`anew`): the tree's weights are bf16 and bear any reference, but the prefix's must start at the top of
    // f16's range, however small its V scales are.  Each row by its own scores alone.  Returns whether this row's
    // was asked for.
    auto move_references = [&](bool ask, bool anew, float top, int t) {
      s_x[g][half][rl] = top;
      const uint32_t mine = __ballot_sync(0xffffffffu, ask);
      if (lane == 0) s_w[g][half][q4] = mine;
      named_bar_sync(pair, 64);
      top = fmaxf(top, s_x[g][half ^ 1][rl]);
      const bool need = (((mine | s_w[g][half ^ 1][q4]) >> lane) & 1u) && top > -INFINITY;
      // (down by 64 at most, also where 64 is less than a step of m, and never down otherwise)
      const float mn = need ? fmaxf(ceilf(top), anew ? __fsub_ru(m, 64.f) : m) : m;
      const float f = mn == m ? 1.f : ex2_approx(m - mn);  // 0 when there was none
      named_bar_sync(pair, 64);                            // both have read before either writes again
      // (these scores came after P V(t - kNB); with one buffer there is nothing to wait for)
      if (t > 0 && __any_sync(0xffffffffu, mn != m)) {
        if (C::kNB > 1) wait(&ofull[g], (t - 1) & 1);
        tc_fence_after();
#pragma unroll 1
        for (int c = half * (D / 64); c < (half + 1) * (D / 64); ++c) {
          uint32_t o[32];
          tmem_ld_x32(tO + c * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
          tmem_st_x32(tO + c * 32, o);
        }
        tmem_st_wait();
      }
      l *= f;
      m = mn;
      return need;
    };
    for (int t = 0; t < T; ++t) {
      wait(&sfull[g][t % C::kNB], (t / C::kNB) & 1);
      tc_fence_after();
      const uint32_t ts = tS + (NG == 2 ? 0 : t % C::kNB) * 128;
      if (t < Tt) {
        // -- a tree tile: 64 keys, this thread's are nodes 64 t + 32 half + j --
        uint32_t x[32];
        tmem_ld_x32(ts + half * 32, x);
        tmem_ld_wait();
        const uint32_t bits = live ? anc[2 * t + half] : 0u;
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float y = (bits >> j) & 1u ? __uint_as_float(x[j]) * p.scale_log2 : -INFINITY;
          top = fmaxf(top, y);
          x[j] = __float_as_uint(y);
        }
        if (bar_or(pair, 64, top > m + 8.f)) move_references(top > m + 8.f, false, top, t);
        const float mu = m == -INFINITY ? 0.f : m;
        uint32_t pk[16];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float a = ex2_approx(__uint_as_float(x[j]) - mu), c = ex2_approx(__uint_as_float(x[j + 1]) - mu);
          sum += a + c;
          pk[j / 2] = pack_bf16x2(a, c);
          x[j] = __float_as_uint(a);
          x[j + 1] = __float_as_uint(c);
        }
        l += sum;
        tmem_st_x16(ts + half * 64, pk);
        // ... and what that rounding left: together the weights to 2^-16 of them, as a short prefix leaves most to the tree
#pragma unroll
        for (int j = 0; j < 32; j += 2)
          pk[j / 2] = pack_bf16x2(__uint_as_float(x[j]) - __uint_as_float(pk[j / 2] << 16),
                                  __uint_as_float(x[j + 1]) - __uint_as_float(pk[j / 2] & 0xFFFF0000u));
        tmem_st_x16(ts + half * 64 + 16, pk);
      } else {
        // -- a prefix tile: this thread's 64 keys are 4 groups of 16, each within one block --
        const float4* cst = s_cst + (t % kCS) * 8 + half * 4;
        // Weights of sixteen keys, 2^(f y + off); returns their sum.
        auto weigh = [&](const uint32_t* y, float f, float off, uint32_t* to) {
          const float2 f2 = make_float2(f, f), off2 = make_float2(off, off);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float2 w = __ffma2_rn(make_float2(__uint_as_float(y[j]), __uint_as_float(y[j + 1])), f2, off2);
            w = make_float2(ex2_approx(w.x), ex2_approx(w.y));
            sum[(j >> 1) & 1] = __fadd2_rn(sum[(j >> 1) & 1], w);
            const __half2 h2 = __floats2half2_rn(w.x, w.y);
            to[j / 2] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          const float2 s2 = __fadd2_rn(sum[0], sum[1]);
          return s2.x + s2.y;
        };
        const int keys = (int)min((long long)kKT8, k1 - (k0 + (long long)(t - Tt) * kKT8));
        float part = 0.f, most = 0.f;  // sum of the weights over the V scales; largest sum of sixteen
        if (keys < kKT8) {  // slots behind the prefix may hold anything: their scores become -inf where they lie
          const int left = keys - half * 64;
#pragma unroll 1
          for (int c = left < 32 ? 0 : 1; c < 2; ++c) {
            uint32_t x[32];
            tmem_ld_x32(ts + half * 64 + c * 32, x);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c * 32 + j >= left) x[j] = 0xFF800000u;
            tmem_st_x32(ts + half * 64 + c * 32, x);
          }
          tmem_st_wait();
        }
        // The factor of a score is never 0, as a row of zeros or a block of zeros would have it: -inf has to stay one (and
        // what is below 2^-126 moves no score).
        auto factor = [&](const float4& k) { return fmaxf(k.x * qf, FLT_MIN); };
        bool slow = t == Tt;
        if (!slow) {
          uint32_t pk[2][16];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
            tmem_ld_x32(ts + half * 64 + c * 32, x);
            tmem_ld_wait();
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
              const float4 k = cst[c * 2 + gr];
              const float s16 = weigh(x + gr * 16, factor(k), k.y - m, pk[c] + gr * 8);
              most = fmaxf(most, s16);
              part = fmaf(s16, k.z, part);
            }
          }
          slow = bar_or(pair, 64, most > kTop);
          if (!slow) {
            tmem_st_x16(ts + half * 64, pk[0]);  // over this thread's own scores
            tmem_st_x16(ts + half * 64 + 16, pk[1]);
          }
        }
        if (slow) {
          // the references move ahead of the weights: in the first tile, and where one has shown to lie too low
          float top = -INFINITY;  // the largest of this thread's scores
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
            tmem_ld_x32(ts + half * 64 + c * 32, x);
            tmem_ld_wait();
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
              float a = -INFINITY;
#pragma unroll
              for (int j = gr * 16; j < gr * 16 + 16; ++j) a = fmaxf(a, __uint_as_float(x[j]));
              const float4 k = cst[c * 2 + gr];
              top = fmaxf(top, __fmaf_rd(a, factor(k), k.y));
            }
          }
          const bool asked = move_references(t == Tt || most > kTop, t == Tt, top, t);
          // A row whose scores pass 2^23 asks for this wherever its largest comes up: m is y rounded down, so up to a step
          // of m below the product that the weights above take exactly.  Here its y is rounded as that of m was.
          const bool far = asked && fabsf(m) >= 0x1p23f, any_far = __any_sync(0xffffffffu, far);
          part = 0.f;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32], pk[16];
            tmem_ld_x32(ts + half * 64 + c * 32, x);
            tmem_ld_wait();
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
              const float4 k = cst[c * 2 + gr];
              float f = factor(k), off = k.y - m;
              if (any_far) {
#pragma unroll
                for (int j = gr * 16; j < gr * 16 + 16; ++j) {
                  const float y = __uint_as_float(x[j]);
                  x[j] = __float_as_uint(far ? __fadd_rn(__fmaf_rd(y, f, k.y), -m) : __fmaf_rn(y, f, off));
                }
                f = 1.f;
                off = 0.f;
              }
              part = fmaf(weigh(x + gr * 16, f, off, pk + gr * 8), k.z, part);
            }
            tmem_st_x16(ts + half * 64 + c * 16, pk);
          }
        }
        l += part;
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull[g][t & 1]);
    }
    // in turn: the scores of tile T - 1 follow P V(T - 1 - kNB) only, and a wait two phases ahead returns at once
    if (C::kNB > 1 && T >= 2) wait(&ofull[g], (T - 2) & 1);
    wait(&ofull[g], C::kNB == 1 ? 0 : (T - 1) & 1);
    const bool fin = __all_sync(0xffffffffu, *static_cast<volatile int*>(&s_abort) == 0);
    if (!fin && lane == 0) set_status(p.dev_status, SPEC_ERR_TIMEOUT);
    s_x[g][half][rl] = l;
    // every MMA of both groups has completed: Q and the rings are free for the O rows
    named_bar_sync(1, 256 * NG);
    l += s_x[g][half ^ 1][rl];
    const bool valid = row < rows && fin && !s_abort && !s_bad && (live || w.n == 1);
    uint8_t* srow = base + rr * C::kORow;
    const bool whole = w.n == 1;
    if (fin) {
      tc_fence_after();
      const float inv = whole ? (live ? 1.f / l : 0.f) : 1.f;
#pragma unroll 1
      for (int c = half * (D / 64); c < (half + 1) * (D / 64); ++c) {
        uint32_t o[32];
        tmem_ld_x32(tO + c * 32, o);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = live ? __float_as_uint(__uint_as_float(o[j]) * inv) : 0u;
        if (tree && live && s_any_odd) {  // V elements of visible tree keys that are no finite numbers
          for (int w = 0; w < kAncWords; ++w)
            for (uint32_t mask = s_odd[w] & anc[w]; mask; mask &= mask - 1) {
              const int key = w * 32 + __ffs(mask) - 1;
              const uint16_t* vt = p.v_tree + (((size_t)b * p.N + key) * p.Hkv + h) * D + c * 32;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float f = __uint_as_float((uint32_t)vt[j] << 16);
                if (!(fabsf(f) < INFINITY)) o[j] = __float_as_uint(__uint_as_float(o[j]) + f);
              }
            }
        }
        if (whole) {
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            *reinterpret_cast<uint4*>(srow + (c * 32 + j) * 2) =
                make_uint4(pack_bf16x2(__uint_as_float(o[j]), __uint_as_float(o[j + 1])),
                           pack_bf16x2(__uint_as_float(o[j + 2]), __uint_as_float(o[j + 3])),
                           pack_bf16x2(__uint_as_float(o[j + 4]), __uint_as_float(o[j + 5])),
                           pack_bf16x2(__uint_as_float(o[j + 6]), __uint_as_float(o[j + 7])));
        } else {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<uint4*>(srow + (c * 32 + j) * 4) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        }
      }
      if (valid && half == 0) {
        const size_t o = orow_of(row);
        if (!whole)
          p.part_ml[w.part + (row - row0)] = make_float2(m, l);
        else if (p.lse)
          p.lse[o] = live ? (m + log2f(l)) * 0.69314718055994531f : 0.f;
      }
    }
    // rows leave 16 bytes a lane, a row's lanes side by side
    named_bar_sync(1, 256 * NG);
    if (!s_abort && !s_bad) {
      const int vshift = whole ? (D == 128 ? 4 : 3) : (D == 128 ? 5 : 4), live_rows = whole ? rows : n * p.G;
#pragma unroll 4
      for (int c = tid - 128; c < kRowsCta << vshift; c += 256 * NG) {
        const int r = c >> vshift, e = c & ((1 << vshift) - 1);
        if (row0 + r >= live_rows) break;
        const size_t o = orow_of(row0 + r);
        const uint4 x = *reinterpret_cast<const uint4*>(base + r * C::kORow + e * 16);
        if (whole)
          *reinterpret_cast<uint4*>(p.out + o * D + e * 8) = x;
        else
          *reinterpret_cast<uint4*>(p.part_o + (w.part + r) * D + e * 4) = x;
      }
    }
  }

  __syncthreads();
  if (s_abort || s_bad) {
    if (tid == 0) {
      if (s_bad) set_status(p.dev_status, SPEC_ERR_CAPACITY);
      if (s_abort) {  // let the copies still in flight land before shared memory is released
        for (int u = max(0, s_kissued - kKS); u < s_kissued; ++u)
          mbar_wait_bounded(&kfull[u % kKS], (uint32_t)((u / kKS) & 1), nullptr);
        for (int u = max(0, s_vissued - kVS); u < s_vissued; ++u)
          mbar_wait_bounded(&vfull[u % kVS], (uint32_t)((u / kVS) & 1), nullptr);
      }
    }
    refuse();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D, int NG>
static cudaError_t launch_tc8(const CUtensorMap* tm, const Kv8AttnParams& p, cudaStream_t stream) {
  using C = TcCfg<D, NG>;
  cudaError_t err =
      cudaFuncSetAttribute(attn_kv8_tc_kernel<D, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (err != cudaSuccess) return err;
  return launch_dependent(attn_kv8_tc_kernel<D, NG>, dim3((unsigned)(p.n_rt * p.Hkv * (p.B * p.base + p.extra))),
                          dim3(C::kThreads), C::kSmem, stream, tm[0], tm[1], tm[2], tm[3], p);
}

cudaError_t launch_attention_kv8_tc(const CUtensorMap* tm, const Kv8AttnParams& p, int groups, cudaStream_t stream) {
  if (p.d == 128) return groups == 2 ? launch_tc8<128, 2>(tm, p, stream) : launch_tc8<128, 1>(tm, p, stream);
  return groups == 2 ? launch_tc8<64, 2>(tm, p, stream) : launch_tc8<64, 1>(tm, p, stream);
}

}  // namespace spectree
