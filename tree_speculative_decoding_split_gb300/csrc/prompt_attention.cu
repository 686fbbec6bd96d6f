// K11: causal attention over packed prompts on tcgen05 tensor cores.
//
// (The pages start from a cached prefix -- qiita "EAGLE-3とMedusaで実装するSpeculative Decoding実践ガイド", section
// "並列検証"; this is the attention that a prompt goes through on its way there.)
//
//   out[i] = sum_{j <= i} 2^(y_ij - m_i) v_j / sum_{j <= i} 2^(y_ij - m_i),   y_ij = log2(e) scale q_i . k_j
// in one pass over the keys with a running maximum m and sum.  4 d operations per visible pair against 2 d bytes per
// row: bound by the tensor cores from a few hundred rows on.
//
// An item is 2 x tg rows of one request with the G query heads of one KV head: a 128-row group (the M of one MMA)
// holds tg = 128 / G rows times G heads, so that each K/V tile is read once for all of them and the causal edge of
// a group is tg rows long, not 128.  Persistent CTAs take items in the plan's order, longest first, in
// turns that run back and forth (the CTA that took the longest of one turn takes the shortest of the next).
//
// Roles (12 warps):
//   warp 0      TMA: Q of each group, then K and V tiles of 128 keys through one ring of 32 KB stages
//   warp 1      MMA issuer of both groups.  Per tile and group: O += P V, then S of the next tile, one behind
//               the other: tensor instructions of one thread run in order, so the next S may overwrite the
//               scores that P lies on, and a commit behind S also tells that P V is done.
//   warps 2, 3  guard: in tiles that hold keys some row does not see (the causal edge, the end of a request) V's
//               infinities and NaN are set to 0, since 0 * inf would reach rows that do not see them; the rows that do
//               see them get them back at the end.  Scores of unseen keys are replaced, so K needs no guard.
//   warps 4-11  softmax, four warps per group, one row per thread: scores from tensor memory, running
//               maximum, P as bf16 over the scores' own columns.  O is rescaled only when a maximum has grown by more
//               than 2^8 (P and the sum use the same stale one); its row leaves through the same thread at the end.
// Tensor memory: 2 x (S 128 + O d) columns.

#include "pdl.cuh"
#include "prompt.cuh"
#include "tc_ptx.cuh"

namespace spectree {

namespace {

constexpr int kKeys = 128;        // keys per tile
constexpr int kRows = 128;        // rows per group
constexpr int kThreads = 384;
constexpr float kRescale = 8.f;   // log2
constexpr float kExact = 262144.f;  // 2^18: maxima from here on, in log2 units, take differences ahead of the scale

template <int D>
struct PromptCfg {
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kTile = kKeys * D * 2;   // K or V tile bytes
  static constexpr int kQ = kRows * D * 2;      // a group's Q
  static constexpr int kSmem = 1024 + 2 * kQ + kStages * kTile;
  static constexpr int kColS = 0, kColO = 256;
};

// The registers of a launch, 384 x 168, shared out anew: the softmax threads hold a row of 128 scores each.
// 128 x 88 + 256 x 208 = 384 x 168.
constexpr int kRegsLaunch = 168, kRegsIssue = 88, kRegsSoftmax = 208;
static_assert(128 * kRegsIssue + 256 * kRegsSoftmax <= kThreads * kRegsLaunch, "more registers than the launch has");

template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Does a word hold a bf16 infinity or NaN, in its lower or upper half?
__device__ __forceinline__ bool special_lo(uint32_t w) { return (w & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ bool special_hi(uint32_t w) { return (w & 0x7f800000u) == 0x7f800000u; }

// An item as every role sees it.
struct Work {
  int r0, n, tok, g;
  int tiles[2];  // key tiles of each group, 0 for a group without rows
  int all;       // tiles of the item
  int edge;      // its first tile with a key that some row does not see
};

__device__ __forceinline__ Work work_of(const PromptAttnParams& p, const PromptItem& it, int g) {
  Work w;
  w.r0 = it.r0;
  w.n = it.n;
  w.tok = it.tok;
  w.g = g;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const int left = it.n - it.tok - a * p.tg;  // rows from this group's first one on
    const int rows = left < p.tg ? left : p.tg;
    w.tiles[a] = rows > 0 ? (it.tok + a * p.tg + rows - 1) / kKeys + 1 : 0;
  }
  w.all = w.tiles[1] ? w.tiles[1] : w.tiles[0];
  w.edge = (w.tok + 1) / kKeys;  // the first t with 128 t + 127 > tok
  return w;
}

// The u-th item of this CTA, or -1: turns of gridDim.x items, every other one taken from behind.
__device__ __forceinline__ int item_index(int u, int total) {
  const long long at = (long long)u * gridDim.x + ((u & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  return at < total ? (int)at : -1;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const PromptAttnParams p) {
  using C = PromptCfg<D>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;                  // [group][d / 64][128 rows][128 B]
  uint8_t* sKV = base + 2 * C::kQ;     // [stage][d / 64][128 keys][128 B]
  // A tile lands on `full`, one for the guard on `held` instead: each has phases of its own, so that whoever waits
  // on one of them takes part in every phase of it (a waiter that sat out a phase could not tell its parity).
  __shared__ uint64_t full[kStages], held[kStages];
  __shared__ uint64_t guarded[kStages];  // V tile looked over by the guard
  __shared__ uint64_t empty[kStages];    // tile read by every MMA
  __shared__ uint64_t qfull[2], qempty[2];
  __shared__ uint64_t sfull[2];        // S computed (and everything issued before it)
  __shared__ uint64_t pfull[2];        // P written
  __shared__ uint64_t ofull[2];        // O complete
  __shared__ uint64_t ofree[2];        // O read
  __shared__ uint64_t drained;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_special;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&held[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&guarded[s], 2);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&qfull[a], 1);
      mbar_init(&qempty[a], 1);
      mbar_init(&sfull[a], 1);
      mbar_init(&pfull[a], 4);
      mbar_init(&ofull[a], 1);
      mbar_init(&ofree[a], 4);
    }
    mbar_init(&drained, 1);
    s_abort = 0;
    s_special = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();  // the plan
  const int total = p.count[0] * p.Hkv;
  auto work_at = [&](int at) { return work_of(p, p.items[at / p.Hkv], at % p.Hkv); };

  if (warp < 4) {
    regs_dec<kRegsIssue>();
    if (warp == 0) {
      // ---- TMA producer ----
      if (lane == 0) {
        int at_stage = 0;
        uint32_t round = 0;
        // per stage: have full and held been used, and the parity of their next phase
        uint32_t f_sent = 0, f_phase = 0, h_sent = 0, h_phase = 0;
        uint32_t qround[2] = {0, 0};
        bool ok = true;
        auto tile = [&](const CUtensorMap* tm, const Work& w, int t, bool guard) -> bool {
          if (!mbar_wait_bounded(&empty[at_stage], (round & 1) ^ 1, &s_abort)) return false;
          uint64_t* bar = guard ? &held[at_stage] : &full[at_stage];
          mbar_arrive_expect_tx(bar, C::kTile);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sKV + at_stage * C::kTile + c * kKeys * 128, tm, bar, c * 64, w.g, w.r0 + t * kKeys);
          const uint32_t bit = 1u << at_stage;
          if (guard) {
            h_sent |= bit;
            h_phase ^= bit;
          } else {
            f_sent |= bit;
            f_phase ^= bit;
          }
          if (++at_stage == kStages) {
            at_stage = 0;
            ++round;
          }
          return true;
        };
        auto queries = [&](const Work& w, int a) -> bool {
          if (w.tiles[a] == 0) return true;
          if (!mbar_wait_bounded(&qempty[a], (qround[a] & 1) ^ 1, &s_abort)) return false;
          mbar_arrive_expect_tx(&qfull[a], (D / 64) * p.tg * p.G * 128);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sQ + a * C::kQ + c * kRows * 128, &tmQ, &qfull[a], c * 64, w.g * p.G, w.r0 + w.tok + a * p.tg);
          ++qround[a];
          return true;
        };
        for (int u = 0, at; ok && (at = item_index(u, total)) >= 0; ++u) {
          const Work w = work_at(at);
          ok = queries(w, 0) && tile(&tmK, w, 0, false) && queries(w, 1);
          for (int t = 0; ok && t < w.all; ++t) {
            ok = tile(&tmV, w, t, t >= w.edge);
            if (ok && t + 1 < w.all) ok = tile(&tmK, w, t + 1, false);
          }
        }
        if (!ok) {
          s_abort = 1;
          set_status(p.dev_status, SPEC_ERR_TIMEOUT);
          // what is under way lands before shared memory is given up: the last load of every barrier
          for (int s = 0; s < kStages; ++s) {
            if ((f_sent >> s) & 1) mbar_wait_bounded(&full[s], ((f_phase >> s) & 1) ^ 1, nullptr);
            if ((h_sent >> s) & 1) mbar_wait_bounded(&held[s], ((h_phase >> s) & 1) ^ 1, nullptr);
          }
          for (int a = 0; a < 2; ++a)
            if (qround[a]) mbar_wait_bounded(&qfull[a], (qround[a] - 1) & 1, nullptr);
        }
      }
    } else if (warp == 1) {
      // ---- MMA issuer ----
      if (lane == 0) {
        constexpr uint32_t idS = idesc_bf16_f32(kRows, kKeys, 0);
        constexpr uint32_t idP = idesc_bf16_f32(kRows, D, 1);
        uint32_t at_load = 0;          // loads before the item's first tile; K(t) is load 2 t, V(t) 2 t + 1 of an item
        uint32_t f_phase = 0, g_phase = 0;  // per stage: parity of the next phase of full and guarded
        uint32_t q_n[2] = {0, 0}, p_n[2] = {0, 0}, o_n[2] = {0, 0};
        bool ok = true;
        auto landed = [&](uint32_t load, bool guard) {
          const int st = load % kStages;
          const uint32_t parity = ((guard ? g_phase : f_phase) >> st) & 1;
          if (guard)
            g_phase ^= 1u << st;
          else
            f_phase ^= 1u << st;
          return mbar_wait_bounded(guard ? &guarded[st] : &full[st], parity, &s_abort);
        };
        auto scores = [&](uint32_t load, int a) {
          tc_fence_after();
          const uint32_t qa = smem_u32(sQ + a * C::kQ), ka = smem_u32(sKV + (load % kStages) * C::kTile);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16(tmem + C::kColS + a * kKeys, sdesc_sw128(qa + (kk >> 2) * (kRows * 128) + (kk & 3) * 32, 0, 1024),
                      sdesc_sw128(ka + (kk >> 2) * (kKeys * 128) + (kk & 3) * 32, 0, 1024), idS, kk > 0);
          umma_commit(&sfull[a]);
        };
        for (int u = 0, at; ok && (at = item_index(u, total)) >= 0; ++u) {
          const Work w = work_at(at);
          ok = landed(at_load, false);
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            if (!ok || w.tiles[a] == 0) continue;
            ok = mbar_wait_bounded(&qfull[a], q_n[a]++ & 1, &s_abort);
            if (!ok) continue;
            scores(at_load, a);
            if (w.tiles[a] == 1) umma_commit(&qempty[a]);
          }
          if (ok) umma_commit(&empty[at_load % kStages]);
          for (int t = 0; ok && t < w.all; ++t) {
            const uint32_t lv = at_load + 2 * t + 1, lk = lv + 1;
            const int sv = lv % kStages;
            ok = landed(lv, t >= w.edge);
            bool next = false;             // K(t + 1) has been waited for
            const uint32_t va = smem_u32(sKV + sv * C::kTile);
#pragma unroll
            for (int a = 0; a < 2; ++a) {
              if (!ok || t >= w.tiles[a]) continue;
              if (t == 0) ok = mbar_wait_bounded(&ofree[a], (o_n[a]++ & 1) ^ 1, &s_abort);
              ok = ok && mbar_wait_bounded(&pfull[a], p_n[a]++ & 1, &s_abort);
              if (!ok) continue;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                umma_bf16_tmem_a(tmem + C::kColO + a * D, tmem + C::kColS + a * kKeys + kk * 8,
                                 sdesc_sw128(va + kk * 2048, kKeys * 128, 1024), idP, (t > 0 || kk > 0) ? 1u : 0u);
              if (t + 1 < w.tiles[a]) {
                ok = next || landed(lk, false);
                next = true;
                if (!ok) continue;
                scores(lk, a);
                if (t + 2 == w.tiles[a]) umma_commit(&qempty[a]);
              } else {
                umma_commit(&ofull[a]);
              }
            }
            if (ok) {
              umma_commit(&empty[sv]);
              if (t + 1 < w.all) umma_commit(&empty[lk % kStages]);
            }
          }
          at_load += 2 * w.all;
        }
        if (!ok) {
          s_abort = 1;
          set_status(p.dev_status, SPEC_ERR_TIMEOUT);
        }
        umma_commit(&drained);
        mbar_wait_bounded(&drained, 0, nullptr);
      }
    } else {
      // ---- guard ----
      uint32_t at_load = 0, phase = 0;
      bool ok = true;
      for (int u = 0, at; ok && (at = item_index(u, total)) >= 0; ++u) {
        const Work w = work_at(at);
        for (int t = w.edge; t < w.all; ++t) {
          const int st = (at_load + 2 * t + 1) % kStages;
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&held[st], (phase >> st) & 1, &s_abort));
          if (!ok) break;
          phase ^= 1u << st;
          uint4* v = reinterpret_cast<uint4*>(sKV + st * C::kTile);
          bool found = false;
#pragma unroll 4
          for (int i = (warp - 2) * 32 + lane; i < C::kTile / 16; i += 64) {
            uint4 x = v[i];
            const bool bad = special_lo(x.x) || special_hi(x.x) || special_lo(x.y) || special_hi(x.y) || special_lo(x.z) ||
                             special_hi(x.z) || special_lo(x.w) || special_hi(x.w);
            if (bad) {
              found = true;
              auto clean = [](uint32_t y) {
                if (special_lo(y)) y &= 0xffff0000u;
                if (special_hi(y)) y &= 0x0000ffffu;
                return y;
              };
              v[i] = make_uint4(clean(x.x), clean(x.y), clean(x.z), clean(x.w));
            }
          }
          if (found) *static_cast<volatile int*>(&s_special) = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&guarded[st]);
        }
        at_load += 2 * w.all;
      }
      if (!ok && lane == 0) {
        s_abort = 1;
        set_status(p.dev_status, SPEC_ERR_TIMEOUT);
      }
    }
  } else {
    // ---- softmax: group a, one row per thread ----
    regs_inc<kRegsSoftmax>();
    const int a = (warp - 4) >> 2, q4 = warp & 3;
    const int rl = q4 * 32 + lane;
    const int my_tok = rl / p.G, my_head = rl - my_tok * p.G;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tmem + C::kColS + a * kKeys + lane_off;
    const uint32_t tO = tmem + C::kColO + a * D + lane_off;
    const float grow = kRescale / p.scale_log2;
    uint32_t s_n = 0, o_n = 0;
    bool ok = true;
    for (int u = 0, at; ok && (at = item_index(u, total)) >= 0; ++u) {
      const Work w = work_at(at);
      if (w.tiles[a] == 0) continue;
      const int first = w.tok + a * p.tg;   // the group's first row
      const int row = first + my_tok;
      float m_run = -INFINITY, l_run = 0.f;  // the maximum in the scores' own units
      for (int t = 0; t < w.tiles[a]; ++t) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sfull[a], s_n++ & 1, &s_abort));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_x32(tS + c * 32, s[c]);
        tmem_ld_wait();
        if (t * kKeys + kKeys - 1 > first) {  // keys behind a row's own: out
          const int lim = row - t * kKeys;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c * 32 + j > lim) s[c][j] = 0xff800000u;
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = __uint_as_float(s[c][0]);
#pragma unroll
          for (int j = 1; j < 32; ++j) mx[c] = fmaxf(mx[c], __uint_as_float(s[c][j]));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const bool need = top > m_run + grow;  // the first finite maximum among them
        if (__any_sync(0xffffffffu, need)) {
          const float f = need ? exp2f((m_run - top) * p.scale_log2) : 1.f;
          if (t > 0) {  // O is complete up to the tile before: the commit behind these scores says so
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld_x32(tO + c * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st_x32(tO + c * 32, o);
            }
          }
          if (need) {
            l_run *= f;
            m_run = top;
          }
        }
        const float ref = m_run == -INFINITY ? 0.f : m_run;
        const float2 sc = make_float2(p.scale_log2, p.scale_log2);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        float shift = ref * p.scale_log2;
        if (__any_sync(0xffffffffu, fabsf(shift) >= kExact)) {
          // the rounding of this product would reach into the exponents: such rows take differences ahead of the scale
          const bool far = fabsf(shift) >= kExact;
          const float r = far ? ref : 0.f;
          shift = far ? 0.f : shift;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j) s[c][j] = __float_as_uint(__uint_as_float(s[c][j]) - r);
        }
        const float2 off = make_float2(-shift, -shift);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[c][j]), __uint_as_float(s[c][j + 1])), sc, off);
            const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
            sum[(j >> 1) & 1] = __fadd2_rn(sum[(j >> 1) & 1], make_float2(p0, p1));
            pk[j / 2] = pack_bf16x2(p0, p1);
          }
          tmem_st_x16(tS + c * 16, pk);
        }
        l_run += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[a]);
      }
      ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(&ofull[a], o_n++ & 1, &s_abort));
      if (!ok) break;
      tc_fence_after();
      const bool valid = rl < p.tg * p.G && row < w.n;
      const size_t orow = valid ? (size_t)(w.r0 + row) * p.Hq + w.g * p.G + my_head : 0;
      const float inv = l_run > 0.f ? 1.f / l_run : (l_run == 0.f ? 0.f : l_run);  // (a NaN sum stays NaN)
      uint32_t o[D / 32][32];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) tmem_ld_x32(tO + c * 32, o[c]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ofree[a]);
      if (valid) {
        uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D);
        const bool special = *static_cast<volatile int*>(&s_special) != 0;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[c][j] = __float_as_uint(__uint_as_float(o[c][j]) * inv);
          if (special) {
            // V's infinities and NaN that the guard has taken out, of the keys this row sees
            for (int key = w.edge * kKeys; key <= row; ++key) {
              const uint16_t* v = p.v + (size_t)(w.r0 + key) * p.v_stride + (size_t)w.g * D + c * 32;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const uint32_t x = (uint32_t)v[j] << 16;
                if (special_hi(x)) o[c][j] = __float_as_uint(__uint_as_float(o[c][j]) + __uint_as_float(x));
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            dst[c * 4 + j / 8] = make_uint4(pack_bf16x2(__uint_as_float(o[c][j]), __uint_as_float(o[c][j + 1])),
                                            pack_bf16x2(__uint_as_float(o[c][j + 2]), __uint_as_float(o[c][j + 3])),
                                            pack_bf16x2(__uint_as_float(o[c][j + 4]), __uint_as_float(o[c][j + 5])),
                                            pack_bf16x2(__uint_as_float(o[c][j + 6]), __uint_as_float(o[c][j + 7])));
        }
        if (p.lse) p.lse[orow] = m_run * p.scale + logf(l_run);
      }
    }
    if (!ok && lane == 0) {
      s_abort = 1;
      set_status(p.dev_status, SPEC_ERR_TIMEOUT);
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D>
static cudaError_t launch_as(const CUtensorMap* tmQ, const CUtensorMap* tmK, const CUtensorMap* tmV,
                             const PromptAttnParams& p, int grid, cudaStream_t stream) {
  cudaFuncAttributes at;
  cudaError_t err = cudaFuncGetAttributes(&at, prompt_attn_kernel<D>);
  if (err != cudaSuccess) return err;
  if (at.numRegs != kRegsLaunch) return cudaErrorInvalidKernelImage;  // the shares above are of this many
  err = cudaFuncSetAttribute(prompt_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptCfg<D>::kSmem);
  if (err != cudaSuccess) return err;
  return launch_dependent(prompt_attn_kernel<D>, dim3(grid), dim3(kThreads), PromptCfg<D>::kSmem, stream, *tmQ, *tmK, *tmV, p);
}

cudaError_t launch_prompt_attention(int d, const CUtensorMap* tmQ, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                    const PromptAttnParams& p, int grid, cudaStream_t stream) {
  return d == 128 ? launch_as<128>(tmQ, tmK, tmV, p, grid, stream) : launch_as<64>(tmQ, tmK, tmV, p, grid, stream);
}

}  // namespace spectree
