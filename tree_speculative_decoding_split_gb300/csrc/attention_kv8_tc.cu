// K9t: tree attention over the 8-bit paged cache on tcgen05 tensor cores, for many rows per KV head.
//
// The codes feed the tensor cores as they lie in the cache.  tcgen05 has no product of a 16-bit with an
// 8-bit operand, so the 16-bit sides enter as sums of two e4m3 numbers: a number with 8 significant
// bits is hi + lo, hi its first 4 bits and lo the rest.
//   Q      scaled per row so that its largest element lies in [128, 256): hi + lo is q to 2^-17 of that;
//   P      2^(y - m) in [0, 448] (y = score in log2 units with the V scale folded in, as in the
//          few-rows kernel): hi by truncation, lo = P - hi, together as exact as bf16;
//   S = Qhi K^T + Qlo K^T and O += Phi V + Plo V, e4m3 x e4m3 at twice the 16-bit rate: the same tensor
//   time as 16-bit operands, half the bytes from HBM, through L2 and in shared memory, and no key or value
//   is ever converted.  Accumulation is float32 (measured: 1e-7 relative, as for bf16).
// The tree's own keys (at most 255, bf16) come first, as bf16 tiles with bf16 Q and P.
//
// One CTA owns (request, KV head, key split, NG x 128 rows).  Bound: per 128-key tile and 128 rows the
// tensor pipe takes 512 (S) + 512 (P V) cycles.  To keep it busy the issue order is fixed,
//   S_a(t)  P V_a(t - 1)  S_b(t)  P V_b(t - 1)  S_a(t + 1) ...
// so that a group's softmax has a whole round for tile t while both S read-outs hide behind a P V.
// TMEM (512 columns): O 2 x 128, one S of 128 columns shared by both groups, P 2 x 64 (hi and lo).  With one
// group: O 128, two S, P 64.
//   warp 0     TMA producer: K and V rings of 128-key tiles (one box per block and tensor, issued by as many
//              lanes), the tile's scales;
//   warp 1     MMA issuer; warps 2, 3 idle, so that register shares can move between warpgroups;
//   warps 4..  softmax, four warps per group, a thread owning a row (a TMEM lane): 128 scores in registers.
#include "common.cuh"
#include "kernels.cuh"
#include "kv8.cuh"
#include "tc_ptx.cuh"

namespace spectree {

namespace {

constexpr int kKT8 = 128;        // keys per prefix tile
constexpr int kTT = 64;          // keys per tree tile (bf16: the same bytes)
constexpr int kGR8 = 128;        // rows per group
constexpr int kKS = 4, kVS = 5;  // ring depths
constexpr int kCS = 8;           // stages of the scales
constexpr float kHead = 8.75f;   // P <= 2^8.75 < 448
constexpr float kFresh = 7.f;    // a new reference puts the row's largest P at 2^7

template <int D, int NG>
struct TcCfg {
  static constexpr int kThreads = 128 + 128 * NG;
  static constexpr int kQ = kGR8 * D * 2;      // Q bytes per group: bf16, or e4m3 hi then lo
  static constexpr int kSlot = kKT8 * D;       // ring slot
  static constexpr int kNB = NG == 2 ? 1 : 2;  // S buffers
  static constexpr int kColO = 0, kColS = NG * 128, kColP = NG * 128 + kNB * 128;
  static constexpr int kNanc = (kMaxNodes + 1) * kAncWords * 4;
  static constexpr int kRing = NG * kQ + (kKS + kVS) * kSlot;
  static constexpr int kSmem = 1024 + kRing + kNanc + kCS * 8 * 16;
  static constexpr int kORow = D * 4 + 16;     // epilogue rows in shared memory, padded
  static_assert(kGR8 * NG * kORow <= kRing, "O staging does not fit");
};

__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A (M x 32 per instruction) in tensor memory: row m in lane m, four consecutive K elements per column.
__device__ __forceinline__ void umma_e4m3_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4: D fp32, A and B e4m3.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, int b_mn_major) {
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
// ... and of chunk ch of row r in a bf16 tile of `rows` rows: halves of 64 columns, 128-byte swizzle.
__device__ __forceinline__ uint32_t bf16_off(int r, int ch, int rows) {
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

// The tile's constants and the exponentials are ordered (volatile): hoisted ahead of their use they cost more
// registers than a softmax thread has beside its 128 scores.
__device__ __forceinline__ float4 lds_f4(const float4* p) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(smem_u32(p)));
  return v;
}
__device__ __forceinline__ float ex2_ordered(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void store_row_bulk(void* gdst, const void* ssrc, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(gdst), "r"(smem_u32(ssrc)),
               "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void store_row_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

__device__ __forceinline__ bool finite2(uint32_t w) { return (w & 0x7F80u) != 0x7F80u && (w & 0x7F800000u) != 0x7F800000u; }

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
  uint32_t* s_nanc = reinterpret_cast<uint32_t*>(sV + kVS * C::kSlot);  // [node][word] ancestors-or-self
  float4* s_cst = reinterpret_cast<float4*>(s_nanc + (kMaxNodes + 1) * kAncWords);  // [stage][16-key group]
  __shared__ uint64_t kfull[kKS], kempty[kKS], vfull[kVS], vempty[kVS];
  // scores ready and read: per group, or with one group per S buffer (else a barrier could be two phases on)
  constexpr int kSB = NG * C::kNB;
  __shared__ uint64_t sfull[kSB], sfree[kSB], pfull[NG], ofull[NG], qready[NG];
  __shared__ uint64_t s_drained;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_bad, s_kissued, s_vissued;
  __shared__ int s_par[kMaxNodes];
  __shared__ uint32_t s_odd[kAncWords];
  const int rt = blockIdx.x, split = blockIdx.y, bg = blockIdx.z;
  const int b = bg / p.Hkv, h = bg - b * p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  long long L;
  int n;
  int err = kv8_counts(p, b, &L, &n);
  const Kv8Split sp = kv8_split(L, p.n_split, p.unit_shift);
  if (split >= sp.n) return;
  const int row0 = rt * kRowsCta, rows = p.N * p.G;
  auto orow_of = [&](int row) { return ((size_t)b * p.N + row / p.G) * p.Hq + h * p.G + row % p.G; };
  // rows of a refused request or of padded nodes; with several splits the merge writes them
  auto refuse = [&]() {
    for (int c = tid; c < kRowsCta * (D / 8); c += C::kThreads) {
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
  // barrier index and parity of step (tile t, group g)
  auto sbar = [](int t, int g) { return NG == 1 ? t % C::kNB : g; };
  auto spar = [](int t) { return (uint32_t)((NG == 1 ? t / C::kNB : t) & 1); };
  if (tid == 0) {
    for (int s = 0; s < kKS; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 1);
    }
    for (int s = 0; s < kVS; ++s) {
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 1);
    }
    for (int g = 0; g < kSB; ++g) {
      mbar_init(&sfull[g], 1);
      mbar_init(&sfree[g], 4);
    }
    for (int g = 0; g < NG; ++g) {
      mbar_init(&pfull[g], 4);
      mbar_init(&ofull[g], 1);
      mbar_init(&qready[g], 4);
    }
    mbar_init(&s_drained, 1);
    s_abort = 0;
    s_bad = 0;
    s_kissued = 0;
    s_vissued = 0;
    fence_mbar_init();
  }
  if (tid < kAncWords) s_odd[tid] = 0u;
  for (int i = tid; i < n; i += C::kThreads) {
    const int par = p.parent[(size_t)b * p.N + i];
    s_par[i] = par;
    if (i == 0 ? par != -1 : (par < 0 || par >= i)) err = SPEC_ERR_BAD_TREE;
  }
  if (__syncthreads_or(err == SPEC_ERR_BAD_TREE)) err = SPEC_ERR_BAD_TREE;
  if (err) {
    if (tid == 0 && rt == 0 && split == 0 && h == 0) set_status(p.dev_status, err);
    refuse();
    return;
  }
  if (row0 >= n * p.G) {
    if (sp.n == 1) refuse();
    return;
  }
  // ---- this CTA's tiles: the tree's (in the last split) and then keys [k0, k1) of the prefix ----
  const bool tree = split == sp.n - 1;
  const long long k0 = ((long long)split * sp.steps) << p.unit_shift;
  const long long k1 = min(L, k0 + ((long long)sp.steps << p.unit_shift));
  const int Tt = tree ? (n + kTT - 1) / kTT : 0;
  const int T = Tt + (k1 > k0 ? (int)((k1 - k0 + kKT8 - 1) / kKT8) : 0);
  if (tree)
    for (int i = tid; i < n; i += C::kThreads) {
      uint32_t* w = s_nanc + i * kAncWords;
#pragma unroll
      for (int j = 0; j < kAncWords; ++j) w[j] = 0u;
      for (int a = i; a >= 0; a = s_par[a]) w[a >> 5] |= 1u << (a & 31);
    }
  if (warp == 1) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // register shares of the warpgroups (two groups): 88 + 2 x 208 = the 3 x 168 that the block was launched with
  if (warp < 4) {
    if constexpr (NG == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
    // ---- TMA producer: lane i < 128 / box takes box i of a tile ----
    const int box = min(p.bs, kKT8), nbox = kKT8 / box;
    const int out_z = p.num_blocks * p.Hkv;  // behind the map: reads as zeros
    // slot of this lane's box in prefix tile u, or -1 when it lies behind the split's keys
    auto slot_of = [&](int u) -> long long {
      const long long s = k0 + (long long)u * kKT8 + lane * box;
      return lane < nbox && s < k1 ? s : -1;
    };
    auto entry = [&](int u) -> int {
      const long long s = slot_of(u);
      return s >= 0 ? p.table[(size_t)b * p.max_blocks + (s >> p.bs_shift)] : -1;
    };
    // the block of tile u is loaded two tiles ahead and its scales one tile ahead of its requests
    int blk0 = entry(0), blk1 = entry(1);
    float ks0 = 0.f, vs0 = 0.f;
    auto scales = [&](int blk, float* ks, float* vs) {
      *ks = 0.f;
      *vs = 0.f;
      if (blk >= 0 && blk < p.num_blocks) {
        *ks = p.k_scale[(size_t)blk * p.Hkv + h];
        *vs = p.v_scale[(size_t)blk * p.Hkv + h];
      }
    };
    scales(blk0, &ks0, &vs0);
    bool ok = true;
    for (int t = 0; t < T; ++t) {
      const int ks = t % kKS, vs = t % kVS, u = t - Tt;
      int blk2 = -1;
      float ks1 = 0.f, vs1 = 0.f;
      if (u >= 0) {
        scales(blk1, &ks1, &vs1);
        blk2 = entry(u + 2);
      }
      const bool got = lane == 0 ? mbar_wait_bounded(&kempty[ks], ((t / kKS) & 1) ^ 1, &s_abort) : true;
      if (!(ok = __shfl_sync(0xffffffffu, got, 0))) break;
      uint8_t* dk = sK + ks * C::kSlot;
      uint8_t* dv = sV + vs * C::kSlot;
      int y = 0, z = out_z;
      if (u >= 0) {
        const long long s = slot_of(u);
        if (s >= 0) {
          if (blk0 >= 0 && blk0 < p.num_blocks) {
            y = (int)(s & (p.bs - 1));
            z = blk0 * p.Hkv + h;
          } else {
            s_bad = 1;
          }
        }
        // scales of the box's 16-key groups: K scale, log2 and reciprocal of the V scale
        if (lane < nbox) {
          const float sv = kv8_clamp_scale(vs0);
          const float4 c = make_float4(kv8_clamp_scale(ks0), __log2f(sv), __fdividef(1.f, sv), 0.f);
          for (int j = 0; j < box / 16; ++j) s_cst[(t % kCS) * 8 + lane * (box / 16) + j] = c;
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_expect_tx(&kfull[ks], C::kSlot);
        s_kissued = t + 1;
      }
      __syncwarp();
      if (u < 0) {
        if (lane < D / 64) tma_load_4d(dk + lane * kTT * 128, &tmKt, &kfull[ks], lane * 64, h, t * kTT, b);
      } else if (lane < nbox) {
        tma_load_3d(dk + lane * box * D, &tmK, &kfull[ks], 0, y, z);
      }
      const bool gotv = lane == 0 ? mbar_wait_bounded(&vempty[vs], ((t / kVS) & 1) ^ 1, &s_abort) : true;
      if (!(ok = __shfl_sync(0xffffffffu, gotv, 0))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&vfull[vs], C::kSlot);
        s_vissued = t + 1;
      }
      __syncwarp();
      if (u < 0) {
        if (lane < D / 64) tma_load_4d(dv + lane * kTT * 128, &tmVt, &vfull[vs], lane * 64, h, t * kTT, b);
      } else {
        if (lane < nbox) tma_load_3d(dv + lane * box * D, &tmV, &vfull[vs], 0, y, z);
        blk0 = blk1;
        blk1 = blk2;
        ks0 = ks1;
        vs0 = vs1;
      }
    }
    if (!ok && lane == 0) {
      s_abort = 1;
      set_status(p.dev_status, SPEC_ERR_TIMEOUT);
    }
    } else if (warp == 1) {
    // ---- MMA issuer ----
    if (lane == 0) {
      constexpr uint32_t idS8 = idesc_e4m3_f32(kGR8, kKT8, 0), idP8 = idesc_e4m3_f32(kGR8, D, 1);
      constexpr uint32_t idSt = idesc_bf16_f32(kGR8, kTT, 0), idPt = idesc_bf16_f32(kGR8, D, 1);
      auto issue_s = [&](int t, int g) -> bool {
        const int u = t * NG + g;
        if (g == 0 && !mbar_wait_bounded(&kfull[t % kKS], (t / kKS) & 1, &s_abort)) return false;
        if (t == 0 && !mbar_wait_bounded(&qready[g], 0, &s_abort)) return false;
        if (t == Tt && Tt > 0 && !mbar_wait_bounded(&qready[g], 1, &s_abort)) return false;
        if (u >= C::kNB) {
          const int w = u - C::kNB;  // the step whose scores the buffer holds
          if (!mbar_wait_bounded(&sfree[sbar(w / NG, w % NG)], spar(w / NG), &s_abort)) return false;
        }
        tc_fence_after();
        const uint32_t ts = tmem + C::kColS + (u % C::kNB) * 128;
        const uint32_t qa = smem_u32(sQ + g * C::kQ), ka = smem_u32(sK + (t % kKS) * C::kSlot);
        if (t < Tt) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16(ts, sdesc_sw128(qa + (kk >> 2) * (kGR8 * 128) + (kk & 3) * 32, 0, 1024),
                      sdesc_sw128(ka + (kk >> 2) * (kTT * 128) + (kk & 3) * 32, 0, 1024), idSt, kk > 0);
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {  // hi, then lo
            const int k = kk % (D / 32);
            umma_e4m3(ts, sdesc_kv8<D>(qa + (kk / (D / 32)) * (kGR8 * D) + k * 32), sdesc_kv8<D>(ka + k * 32), idS8,
                      kk > 0);
          }
        }
        umma_commit(&sfull[sbar(t, g)]);
        if (g == NG - 1) umma_commit(&kempty[t % kKS]);
        return true;
      };
      auto issue_pv = [&](int t, int g) -> bool {
        if (g == 0 && !mbar_wait_bounded(&vfull[t % kVS], (t / kVS) & 1, &s_abort)) return false;
        if (!mbar_wait_bounded(&pfull[g], t & 1, &s_abort)) return false;
        tc_fence_after();
        const uint32_t pt = tmem + C::kColP + g * 64, ot = tmem + C::kColO + g * 128;
        const uint32_t va = smem_u32(sV + (t % kVS) * C::kSlot);
        if (t < Tt) {
#pragma unroll
          for (int kk = 0; kk < kTT / 16; ++kk)
            umma_bf16_tmem_a(ot, pt + kk * 8, sdesc_sw128(va + kk * 16 * 128, kTT * 128, 1024), idPt, t > 0 || kk > 0);
        } else {
#pragma unroll
          for (int kk = 0; kk < kKT8 / 16; ++kk) {  // hi, then lo
            const int k = kk % (kKT8 / 32);
            umma_e4m3_tmem_a(ot, pt + kk * 8, sdesc_kv8<D>(va + k * 32 * D), idP8, t > 0 || kk > 0);
          }
        }
        umma_commit(&ofull[g]);
        if (g == NG - 1) umma_commit(&vempty[t % kVS]);
        return true;
      };
      bool ok = true;
      for (int t = 0; t <= T && ok; ++t)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (ok && t < T) ok = issue_s(t, g);
          if (ok && t > 0) ok = issue_pv(t - 1, g);
        }
      if (!ok) {
        s_abort = 1;
        set_status(p.dev_status, SPEC_ERR_TIMEOUT);
      }
      umma_commit(&s_drained);  // every MMA of this CTA
      mbar_wait_bounded(&s_drained, 0, nullptr);
    }
    }
  } else {
    if constexpr (NG == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---- softmax ----
    const int g = (warp - 4) >> 2, q4 = warp & 3;
    const int rl = q4 * 32 + lane, rr = g * kGR8 + rl, row = row0 + rr;
    const int gtid = q4 * 32 + lane;  // thread of the group
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tmem + C::kColS + lane_off, tO = tmem + C::kColO + g * 128 + lane_off;
    const uint32_t tP = tmem + C::kColP + g * 64 + lane_off;
    const bool live = row < n * p.G;
    const uint16_t* q = p.q + orow_of(live ? row : row0) * D;
    uint8_t* myQ = sQ + g * C::kQ;
    float qf = 0.f;  // undoes the row's scaling, with the softmax scale in log2 units
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, &s_abort));
    };
    auto load_q = [&](int ch) { return live ? *reinterpret_cast<const uint4*>(q + ch * 8) : make_uint4(0, 0, 0, 0); };
    auto publish = [&](uint64_t* bar) {  // shared memory written here is for the tensor cores
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // this row as e4m3 hi and lo
    auto split_q = [&]() {
      // read twice (the second time from L1 or L2): a row of it beside the scores would not fit the registers
      float mx = 0.f;
#pragma unroll 8
      for (int i = 0; i < D / 8; ++i) {
        const uint4 w = load_q(i);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mx = max3(mx, fabsf(__uint_as_float(x[j] << 16)), fabsf(__uint_as_float(x[j] & 0xFFFF0000u)));
      }
      const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 100);
      const float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);  // largest element into [128, 256)
      qf = __uint_as_float((uint32_t)(127 - 7 + e) << 23) * p.scale_log2;
#pragma unroll 2
      for (int i = 0; i < D / 16; ++i) {
        uint32_t hi[4], lo[4];
        const uint4 w[2] = {load_q(2 * i), load_q(2 * i + 1)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 v = w[j >> 1];
          const uint32_t a = (j & 1) ? v.z : v.x, c = (j & 1) ? v.w : v.y;
          const float f[4] = {__uint_as_float(a << 16) * up, __uint_as_float(a & 0xFFFF0000u) * up,
                              __uint_as_float(c << 16) * up, __uint_as_float(c & 0xFFFF0000u) * up};
          hi[j] = e4m3x4(head4(f[0]), head4(f[1]), head4(f[2]), head4(f[3]));
          lo[j] = e4m3x4(f[0] - head4(f[0]), f[1] - head4(f[1]), f[2] - head4(f[2]), f[3] - head4(f[3]));
        }
        *reinterpret_cast<uint4*>(myQ + kv8_off<D>(rl, i)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(myQ + kGR8 * D + kv8_off<D>(rl, i)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    };
    if (Tt > 0) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) *reinterpret_cast<uint4*>(myQ + bf16_off(rl, i, kGR8)) = load_q(i);
    } else {
      split_q();
    }
    publish(&qready[g]);

    float m = -INFINITY, l = 0.f;  // reference (P = 2^(y - m)) and sum
    const uint32_t* anc = s_nanc + (live ? row / p.G : 0) * kAncWords;
    bool ok = true;
    // Moves the reference up when the tile's largest y has left the range of P; O follows.  At the first tile
    // behind the tree's (`rebase`) it moves down as well: the tree's weights are bf16 and bear any reference,
    // but the prefix's must start at the top of e4m3's range, however small its V scales are.
    auto advance = [&](float top, int t, bool rebase) {
      const bool need = top > m + kHead || (rebase && top > -INFINITY);
      if (__any_sync(0xffffffffu, need)) {
        const float mn = need ? fmaxf(top - kFresh, m - 64.f) : m;
        const float f = need ? ex2_approx(m - mn) : 1.f;  // 0 when there was none
        if (t > 0) {
          if (!wait(&ofull[g], (t - 1) & 1)) return false;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
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
      }
      return true;
    };
    for (int t = 0; t < T; ++t) {
      if (!wait(&sfull[sbar(t, g)], spar(t))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t ts = tS + ((t * NG + g) % C::kNB) * 128;
      if (t < Tt) {
        // -- a tree tile: 64 keys, node t * 64 + j --
        uint32_t s0[32], s1[32];
        tmem_ld_x32(ts, s0);
        tmem_ld_x32(ts + 32, s1);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfree[sbar(t, g)]);
        if (t == Tt - 1 && T > Tt) {  // the last product with the bf16 queries is done: make room for hi and lo
          split_q();
          publish(&qready[g]);
        }
        const uint32_t w0 = live ? anc[2 * t] : 0u, w1 = live ? anc[2 * t + 1] : 0u;
        float v[64], top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          v[j] = (w0 >> j) & 1u ? __uint_as_float(s0[j]) * p.scale_log2 : -INFINITY;
          v[32 + j] = (w1 >> j) & 1u ? __uint_as_float(s1[j]) * p.scale_log2 : -INFINITY;
          top = max3(top, v[j], v[32 + j]);
        }
        if (!advance(top, t, false)) {
          ok = false;
          break;
        }
        const float mu = m == -INFINITY ? 0.f : m;
        uint32_t pk[32];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 64; j += 2) {
          const float a = ex2_approx(v[j] - mu), c = ex2_approx(v[j + 1] - mu);
          sum += a + c;
          pk[j / 2] = pack_bf16x2(a, c);
        }
        l += sum;
        // V elements that are no finite numbers enter as 0 and are noted; both groups do the whole tile, as
        // each one's product may run before the other has looked
        if (!wait(&vfull[t % kVS], (t / kVS) & 1)) {
          ok = false;
          break;
        }
        uint8_t* tv = sV + (t % kVS) * C::kSlot;
#pragma unroll 1
        for (int c = gtid; c < kTT * (D / 8); c += kGR8) {
          const int r = c / (D / 8), key = t * kTT + r;
          uint4* at = reinterpret_cast<uint4*>(tv + bf16_off(r, c % (D / 8), kTT));
          uint4 x = *at;
          if (finite2(x.x) && finite2(x.y) && finite2(x.z) && finite2(x.w)) continue;
          if (key < n) atomicOr(&s_odd[key >> 5], 1u << (key & 31));
          uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if ((w[j] & 0x7F80u) == 0x7F80u) w[j] &= 0xFFFF0000u;
            if ((w[j] & 0x7F800000u) == 0x7F800000u) w[j] &= 0xFFFFu;
          }
          *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        if (t > 0 && !wait(&ofull[g], (t - 1) & 1)) {
          ok = false;
          break;
        }
        tmem_st_x32(tP, pk);
      } else {
        // -- a prefix tile: 128 keys in 8 groups of 16, each within one block --
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_x32(ts + c * 32, s[c]);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfree[sbar(t, g)]);
        const int left = (int)min((long long)kKT8, k1 - (k0 + (long long)(t - Tt) * kKT8));
        if (left < kKT8) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c * 32 + j >= left) s[c][j] = 0xFF800000u;
          // slots behind the prefix may hold anything: their V rows become 0 (by both groups, as above)
          if (!wait(&vfull[t % kVS], (t / kVS) & 1)) {
            ok = false;
            break;
          }
          uint8_t* tv = sV + (t % kVS) * C::kSlot;
          for (int c = left * (D / 16) + gtid; c < kKT8 * (D / 16); c += kGR8)
            *reinterpret_cast<uint4*>(tv + c * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        const float4* cst = s_cst + (t % kCS) * 8;
        float top = -INFINITY;
#pragma unroll
        for (int gr = 0; gr < 8; ++gr) {
          const uint32_t* x = &s[gr >> 1][(gr & 1) * 16];
          float a = __uint_as_float(x[0]);
#pragma unroll
          for (int j = 1; j < 15; j += 2) a = max3(a, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
          a = fmaxf(a, __uint_as_float(x[15]));
          const float4 c = lds_f4(cst + gr);
          top = fmaxf(top, fmaf(a, c.x * qf, c.y));
        }
        if (!advance(top, t, t == Tt && t > 0)) {
          ok = false;
          break;
        }
        const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // 64 keys at a time
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int gr = 0; gr < 4; ++gr) {
            const uint32_t* x = &s[half * 2 + (gr >> 1)][(gr & 1) * 16];
            const float4 c = lds_f4(cst + half * 4 + gr);
            const float f = c.x * qf, off = c.y - mu;
            const float2 f2 = make_float2(f, f), off2 = make_float2(off, off);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              float2 a = __ffma2_rn(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), f2, off2);
              float2 e = __ffma2_rn(make_float2(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])), f2, off2);
              a = make_float2(ex2_ordered(a.x), ex2_ordered(a.y));
              e = make_float2(ex2_ordered(e.x), ex2_ordered(e.y));
              sum = __fadd2_rn(sum, __fadd2_rn(a, e));
              const float2 ah = make_float2(head4(a.x), head4(a.y)), eh = make_float2(head4(e.x), head4(e.y));
              const float2 al = __fadd2_rn(a, make_float2(-ah.x, -ah.y)), el = __fadd2_rn(e, make_float2(-eh.x, -eh.y));
              hi[gr * 4 + j / 4] = e4m3x4(ah.x, ah.y, eh.x, eh.y);
              lo[gr * 4 + j / 4] = e4m3x4(al.x, al.y, el.x, el.y);
            }
            l = fmaf(sum.x + sum.y, c.z, l);
          }
          // P V(t - 1) has read P
          if (half == 0 && t > 0 && !wait(&ofull[g], (t - 1) & 1)) ok = false;
          tmem_st_x16(tP + half * 16, hi);
          tmem_st_x16(tP + 32 + half * 16, lo);
        }
        if (!ok) break;
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull[g]);
    }
    const bool fin = ok && wait(&ofull[g], (T - 1) & 1);
    if (!fin && lane == 0) {
      s_abort = 1;
      set_status(p.dev_status, SPEC_ERR_TIMEOUT);
    }
    // every MMA of both groups has completed: Q and the rings are free for the O rows
    named_bar_sync(1, 128 * NG);
    const bool valid = row < rows && fin && !s_abort && !s_bad && (live || sp.n == 1);
    if (fin) {
      tc_fence_after();
      uint8_t* srow = base + rr * C::kORow;
      const bool whole = sp.n == 1;
      const float inv = whole ? (live ? 1.f / l : 0.f) : 1.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld_x32(tO + c * 32, o);
        tmem_ld_wait();
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = live ? __uint_as_float(o[j]) * inv : 0.f;
        if (tree && live) {  // V elements of visible tree keys that are no finite numbers
          for (int w = 0; w < kAncWords; ++w)
            for (uint32_t mask = s_odd[w] & anc[w]; mask; mask &= mask - 1) {
              const int key = w * 32 + __ffs(mask) - 1;
              const uint16_t* vt = p.v_tree + (((size_t)b * p.N + key) * p.Hkv + h) * D + c * 32;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float f = __uint_as_float((uint32_t)vt[j] << 16);
                if (!(fabsf(f) < INFINITY)) x[j] += f;
              }
            }
        }
        if (whole) {
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            *reinterpret_cast<uint4*>(srow + (c * 32 + j) * 2) =
                make_uint4(pack_bf16x2(x[j], x[j + 1]), pack_bf16x2(x[j + 2], x[j + 3]), pack_bf16x2(x[j + 4], x[j + 5]),
                           pack_bf16x2(x[j + 6], x[j + 7]));
        } else {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(srow + (c * 32 + j) * 4) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
        }
      }
      if (valid) {
        const size_t o = orow_of(row);
        if (whole) {
          if (p.lse) p.lse[o] = live ? (m + log2f(l)) * 0.69314718055994531f : 0.f;
        } else {
          p.part_ml[o * p.n_split + split] = make_float2(m, l);
        }
        fence_proxy_async_smem();
        if (whole)
          store_row_bulk(p.out + o * D, srow, D * 2);
        else
          store_row_bulk(p.part_o + (o * p.n_split + split) * D, srow, D * 4);
        store_row_wait();
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
  attn_kv8_tc_kernel<D, NG>
      <<<dim3(p.n_rt, p.n_split, p.B * p.Hkv), C::kThreads, C::kSmem, stream>>>(tm[0], tm[1], tm[2], tm[3], p);
  return cudaGetLastError();
}

cudaError_t launch_attention_kv8_tc(const CUtensorMap* tm, const Kv8AttnParams& p, int groups, cudaStream_t stream) {
  if (p.d == 128) return groups == 2 ? launch_tc8<128, 2>(tm, p, stream) : launch_tc8<128, 1>(tm, p, stream);
  return groups == 2 ? launch_tc8<64, 2>(tm, p, stream) : launch_tc8<64, 1>(tm, p, stream);
}

}  // namespace spectree
