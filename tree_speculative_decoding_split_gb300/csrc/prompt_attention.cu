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
//   warp 0      TMA: Q of each group, then K and V tiles of 128 keys through one ring (5 stages of 32 KB, at d 64 8 of 16 KB)
//   warps 1, 2  MMA issuers, one for each group, in turns.  A turn is O += P V of a tile and S of the next one; the
//               commit behind S also tells that P V is done.  Tensor instructions keep their order for sure only where
//               they have one accumulator and one shape, so S may not overwrite a P that P V has yet to read: at d 64
//               P has columns of its own, at d 128, where tensor memory is full and P lies over its own scores, S is
//               issued when P V is done (2770 us without that wait, 2830 with it, at the 16384 rows below).  The tensor cores
//               queue little, so whatever else an issuer waits for, it waits for during the other's turn.
//   warp 3      guard: in tiles that hold keys some row does not see (the causal edge, the end of a request) V's
//               infinities and NaN are set to 0, since 0 * inf would reach rows that do not see them; the rows that do
//               see them get them back at the end.  Scores of unseen keys are replaced, so K needs no guard.
//   warps 4-11  softmax, four warps per group, one row per thread: scores from tensor memory, P as bf16 back
//               to it.  O is rescaled only where a row's weights of a tile sum up to more than 2^8 (until then P and
//               the sum use an older maximum); its row leaves through the same thread at the end.
// P's completion and the turns go through named barriers, which wait without a limit: the tensor cores' reading slows
// every access to shared memory, mbarriers included, to some 180 cycles (when they came in, 3250 cycles a tile of both
// groups became 2900).  So a warp whose other waits gave up does no more work but meets these barriers up to its last item.
// Tensor memory: 2 x (S 128 + O d) columns, and 2 x 64 for P at d 64.
//
// What bounds it: a tile of both groups is 2048 cycles of MMA at d 128 and takes 2920; the rest is the way from S to P and
// back (1000 cycles of softmax, 600 of hand-offs, 150 of the wait for P V), which two groups do not hide in full and for more
// tensor memory is too small.  16384 rows of 64 heads on 8: 2840 us, 1549 TFLOP/s, at the power limit.  At d 64 the MMAs of S
// halve in number, those of P V (64 columns of output) take as long as with 128, and that way does not change: 2650 cycles a
// tile, and 3600 to go from one item to the next, which weighs where prompts are short.  48 prompts of up to 1800 rows, 16
// heads on 8: 185 us.  (Graph replays; a Python call takes 2880 and 186.)
// Weights go into P as bf16, off by 2^-8 of each at most, so that out is 0.0020 to 0.0022 from 64 bits where its own rounding
// alone leaves 0.0016.  As a pair of bf16 numbers they leave no more than that, at half as many MMAs again and more to store:
// 4450 us at the rows above (2770 then), 307 for the 48 prompts (184), 18.3 for one of 500 rows (12.4).  The sum, the maximum
// and O stay in fp32, and the sum adds the weights before that rounding.

#include "pdl.cuh"
#include "prompt.cuh"
#include "tc_ptx.cuh"

namespace spectree {

namespace {

constexpr int kKeys = 128;        // keys per tile
constexpr int kRows = 128;        // rows per group
constexpr int kThreads = 384;
constexpr int kBarTurn = 1, kBarP = 3;  // named barriers: an issuer's turn, a group's P written
constexpr float kGrown = 256.f;   // a row's sum over a tile from which on it takes the tile's maximum as its reference
constexpr float kExact = 262144.f;  // 2^18: maxima from here on, in log2 units, take differences ahead of the scale

template <int D>
struct PromptCfg {
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kTile = kKeys * D * 2;   // K or V tile bytes
  static constexpr int kQ = kRows * D * 2;      // a group's Q
  static constexpr int kSmem = 1024 + 2 * kQ + kStages * kTile;
  static constexpr int kColS = 0, kColO = 256;
  static constexpr bool kOver = D == 128;       // P lies over its own scores
  static constexpr int kColP = kOver ? kColS : 384, kWideP = kOver ? kKeys : kKeys / 2;
};

// mbar_wait_bounded with all but the first try out of line: a wait that is over costs the issuing threads a few instructions.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, int* abort) { return mbar_wait_bounded(bar, parity, abort); }
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* abort) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void named_arrive(int id, int count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// tmem_ld_wait, with the registers that it is for: nothing is taken from them ahead of it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&a)[4][32]) {
  tmem_ld_wait();
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int j = 0; j < 32; j += 16)
      asm volatile("" : "+r"(a[c][j]), "+r"(a[c][j + 1]), "+r"(a[c][j + 2]), "+r"(a[c][j + 3]), "+r"(a[c][j + 4]),
                   "+r"(a[c][j + 5]), "+r"(a[c][j + 6]), "+r"(a[c][j + 7]), "+r"(a[c][j + 8]), "+r"(a[c][j + 9]),
                   "+r"(a[c][j + 10]), "+r"(a[c][j + 11]), "+r"(a[c][j + 12]), "+r"(a[c][j + 13]), "+r"(a[c][j + 14]),
                   "+r"(a[c][j + 15]));
}

// A tile's weights in two passes over its scores, of which a row sees those up to key `lim`: the maximum, with what is
// there brought to it where it has grown (with_o: O holds something; the commit behind the scores says
// that it is complete), then P over the scores that have been read.  Where the reference is so large that its product
// with the scale would be rounded by whole units, differences are taken ahead of the scale.  The whole warp comes here
// where one of its rows has to (`mine`); the others take the steps, and the order of additions, of the ordinary way, so that
// a row's bits do not tell what lies beside it.  Returns the row's reference (in the scores' units) and sum.  Out of line
// and in loops: it runs once or twice an item, and cold code costs more than its instructions.
template <int D>
__device__ __noinline__ float2 tile_again(uint32_t tS, uint32_t tP, uint32_t tO, int lim, bool mine, bool with_o, float2 ml,
                                          float head, float scale_log2) {
  float top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t s[32];
    tmem_ld_x32(tS + c * 32, s);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (c * 32 + j <= lim) top = fmaxf(top, __uint_as_float(s[j]));
  }
  top += head;
  const bool need = mine && top > ml.x;  // (the first finite maximum among them)
  if (__any_sync(0xffffffffu, need)) {
    const float f = need ? exp2f((ml.x - top) * scale_log2) : 1.f;
    if (with_o) {
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld_x32(tO + c * 32, o);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
        tmem_st_x32(tO + c * 32, o);
      }
    }
    if (need) ml = make_float2(top, ml.y * f);
  }
  const float ref = ml.x == -INFINITY ? 0.f : ml.x;
  const bool far = fabsf(ref * scale_log2) >= kExact;
  const float shift = far ? 0.f : ref * scale_log2, before = far ? ref : 0.f;
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t s[32], pk[16];
    tmem_ld_x32(tS + c * 32, s);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      float w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        w[e] = ex2_approx(fmaf(__uint_as_float(s[j + e]) - before, scale_log2, -shift));
        if (c * 32 + j + e > lim) w[e] = 0.f;
      }
      sum[(j >> 1) & 1] = __fadd2_rn(sum[(j >> 1) & 1], make_float2(w[0], w[1]));
      pk[j / 2] = pack_bf16x2(w[0], w[1]);
    }
    tmem_st_x16(tP + c * 16, pk);
  }
  ml.y += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
  tmem_st_wait();
  return ml;
}

// The upper bits of a word's halves that are a bf16 infinity or NaN (exponent all ones); the word without these.
__device__ __forceinline__ uint32_t specials(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ uint32_t clean(uint32_t w) {
  const uint32_t bad = specials(w);
  return w & ~((bad & 0x80000000u ? 0xffff0000u : 0u) | (bad & 0x8000u ? 0xffffu : 0u));
}

// 64 bytes of a row: in whole 32-byte sectors where the rows begin on one.
__device__ __forceinline__ void store_64(uint16_t* dst, const uint32_t (&y)[16], bool sectors) {
  if (sectors) {
#pragma unroll
    for (int j = 0; j < 16; j += 8)
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 2 * j), "r"(y[j]), "r"(y[j + 1]),
                   "r"(y[j + 2]), "r"(y[j + 3]), "r"(y[j + 4]), "r"(y[j + 5]), "r"(y[j + 6]), "r"(y[j + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int j = 0; j < 16; j += 4) *reinterpret_cast<uint4*>(dst + 2 * j) = make_uint4(y[j], y[j + 1], y[j + 2], y[j + 3]);
  }
}

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
  __shared__ uint64_t pread[2];        // P read (where the next scores go over it)
  __shared__ uint64_t ofull[2];        // O complete
  __shared__ uint64_t ofree[2];        // O read
  __shared__ uint64_t drained[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_special;
  __shared__ PlanShared s_plan;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&held[s], 1);
      mbar_init(&empty[s], 2);
      mbar_init(&guarded[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&qfull[a], 1);
      mbar_init(&qempty[a], 1);
      mbar_init(&sfull[a], 1);
      mbar_init(&pread[a], 1);
      mbar_init(&ofull[a], 1);
      mbar_init(&drained[a], 1);
      mbar_init(&ofree[a], 4);
    }
    s_abort = 0;
    s_special = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  // Rows behind the last head, where G does not divide 128, are never loaded: zeros, not what shared memory holds, whose
  // scores could outgrow their reference time and again.
  const int behind = (kRows - p.tg * p.G) * 8;  // 16-byte pieces in each of the 2 D / 64 slabs
  for (int i = tid; i < 2 * (D / 64) * behind; i += kThreads) {
    const int slab = i / behind, at = i - slab * behind;
    *reinterpret_cast<uint4*>(sQ + slab * kRows * 128 + p.tg * p.G * 128 + at * 16) = make_uint4(0, 0, 0, 0);
  }
  if (behind) fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();  // the plan
  const PlanReader<false> plan(p.plan, s_plan, p.dev_status);
  const int total = plan.count * p.Hkv;
  // This CTA's items one by one, the next one's entry fetched while the current one is under way.
  int u = 0, at = item_index(0, total);
  PromptItem entry = at >= 0 ? plan.item(at / p.Hkv) : PromptItem{};
  auto take = [&](Work& w) -> bool {
    if (at < 0) return false;
    w = work_of(p, entry, at % p.Hkv);
    at = item_index(++u, total);
    if (at >= 0) entry = plan.item(at / p.Hkv);
    return true;
  };

  if (warp < 4) {
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
        for (Work w; ok && take(w);) {
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
    } else if (warp < 3) {
      // ---- MMA issuer of group a: the whole warp waits, one lane issues ----
      const int a = warp - 1;
      constexpr uint32_t idS = idesc_bf16_f32(kRows, kKeys, 0);
      constexpr uint32_t idP = idesc_bf16_f32(kRows, D, 1);
      const uint32_t q_lo = (smem_u32(sQ + a * C::kQ) >> 4), kv_lo = (smem_u32(sKV) >> 4);
      const uint32_t v_mn = ((kKeys * 128) >> 4) << 16;  // V (MN-major): the distance of its two halves of d
      const uint32_t tS = tmem + C::kColS + a * kKeys, tO = tmem + C::kColO + a * D, tP = tmem + C::kColP + a * C::kWideP;
      int st = 0;                          // stage of the next load
      uint32_t f_phase = 0, g_phase = 0;   // per stage: parity of the next phase of full and guarded
      uint32_t q_n = 0, p_n = 0;
      bool ok = true;
      // The next load has landed (and been looked over); its stage.
      auto landed = [&](bool guard) -> int {
        uint32_t& phase = guard ? g_phase : f_phase;
        const int at = st;
        ok = ok && wait(guard ? &guarded[at] : &full[at], (phase >> at) & 1, &s_abort);
        phase ^= 1u << at;
        st = at + 1 == kStages ? 0 : at + 1;
        return at;
      };
      auto arrive = [&](uint64_t* bar) {
        if (lane == 0) mbar_arrive(bar);
      };
      auto scores = [&](int k) {
        const uint32_t k_lo = kv_lo + k * (C::kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * ((kKeys * 128) >> 4) + (kk & 3) * 2;
          umma_bf16(tS, desc_sw128(q_lo + off), desc_sw128(k_lo + off), idS, kk > 0);
        }
      };
      if (a == 1) named_arrive(kBarTurn, 64);  // group 0 begins
      // An issuer whose wait gave up issues nothing more, but takes and hands on its turns to the last item's end.
      for (Work w; take(w);) {
        const int tiles = a ? w.tiles[1] : w.tiles[0];
        int k = landed(false);
        if (tiles > 0) {
          ok = ok && wait(&qfull[a], q_n & 1, &s_abort);
          if (C::kOver && q_n > 0) ok = ok && wait(&ofull[a], (q_n - 1) & 1, &s_abort);  // the last item's P read
        }
        ok = __all_sync(0xffffffffu, ok);
        named_bar_sync(kBarTurn + a, 64);
        tc_fence_after();
        if (ok && tiles > 0 && lane == 0) {
          scores(k);
          umma_commit(&sfull[a]);
          if (tiles == 1) umma_commit(&qempty[a]);
        }
        __syncwarp();
        named_arrive(kBarTurn + (a ^ 1), 64);
        if (ok && tiles == 0) arrive(&empty[k]);
        for (int t = 0; t < w.all; ++t) {
          const int v = landed(t >= w.edge);
          const bool more = t + 1 < w.all;
          if (more) k = landed(false);
          if (t == 0 && tiles > 0) ok = ok && wait(&ofree[a], (q_n & 1) ^ 1, &s_abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) s_abort = 1;
          if (t < tiles) named_bar_sync(kBarP + a, 160);
          named_bar_sync(kBarTurn + a, 64);
          tc_fence_after();
          if (ok && t < tiles && lane == 0) {
            const uint32_t v_lo = (kv_lo + v * (C::kTile >> 4)) | v_mn;
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              umma_bf16_tmem_a(tO, tP + kk * 8, desc_sw128(v_lo + kk * (2048 >> 4)), idP, (t > 0 || kk > 0) ? 1u : 0u);
            if (t + 1 < tiles) {
              if (C::kOver) {
                umma_commit(&pread[a]);
                ok = wait(&pread[a], p_n++ & 1, &s_abort);
              }
              if (ok) {
                scores(k);
                umma_commit(&sfull[a]);
                if (t + 2 == tiles) umma_commit(&qempty[a]);
              }
            } else {
              umma_commit(&ofull[a]);
            }
          }
          __syncwarp();
          named_arrive(kBarTurn + (a ^ 1), 64);
          if (ok && t >= tiles) arrive(&empty[v]);
          if (ok && more && t + 1 >= tiles) arrive(&empty[k]);
        }
        if (tiles > 0) ++q_n;
      }
      if (a == 0) named_bar_sync(kBarTurn, 64);  // (the turn that group 1 hands on at the end)
      if (lane == 0) {
        if (!ok) {
          s_abort = 1;
          set_status(p.dev_status, SPEC_ERR_TIMEOUT);
        }
        umma_commit(&drained[a]);
        mbar_wait_bounded(&drained[a], 0, nullptr);
      }
    } else {
      // ---- guard ----
      uint32_t at_load = 0, phase = 0;
      bool ok = true;
      for (Work w; ok && take(w);) {
        for (int t = w.edge; t < w.all; ++t) {
          const int st = (at_load + 2 * t + 1) % kStages;
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&held[st], (phase >> st) & 1, &s_abort));
          if (!ok) break;
          phase ^= 1u << st;
          uint4* v = reinterpret_cast<uint4*>(sKV + st * C::kTile);
          bool found = false;
#pragma unroll 1
          for (int i = lane; i < C::kTile / 16; i += 32 * 8) {
            uint4 x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = v[i + 32 * j];
            uint32_t bad = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) bad |= specials(x[j].x) | specials(x[j].y) | specials(x[j].z) | specials(x[j].w);
            if (bad) {
              found = true;
#pragma unroll
              for (int j = 0; j < 8; ++j) v[i + 32 * j] = make_uint4(clean(x[j].x), clean(x[j].y), clean(x[j].z), clean(x[j].w));
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
    const int a = (warp - 4) >> 2, q4 = warp & 3;
    const int rl = q4 * 32 + lane;
    const int my_tok = rl / p.G, my_head = rl - my_tok * p.G;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tmem + C::kColS + a * kKeys + lane_off;
    const uint32_t tO = tmem + C::kColO + a * D + lane_off;
    const uint32_t tP = tmem + C::kColP + a * C::kWideP + lane_off;
    uint32_t s_n = 0, o_n = 0;
    int st = 0;  // stage of the item's next load to release
    bool ok = true;
    Work w, next;
    for (bool have = take(next); have;) {
      w = next;
      // Scores, or O, tell that the group's MMAs before them are done: the stages they read are released for it.
      auto released = [&]() {
        if (ok && lane == 0 && q4 == 0) mbar_arrive(&empty[st]);
        st = st + 1 == kStages ? 0 : st + 1;
      };
      if (w.tiles[a] == 0) {
        st = (st + 2 * w.all) % kStages;
        have = take(next);
        continue;
      }
      const int first = w.tok + a * p.tg;   // the group's first row
      const int row = first + my_tok;
      const bool valid = rl < p.tg * p.G && row < w.n;  // (rows behind the last head, or of the next request, count for nothing)
      float m_run = -INFINITY, l_run = 0.f;  // the reference, in the scores' own units, and the weights' sum
      for (int t = 0; t < w.tiles[a]; ++t) {
        // (a warp whose wait gave up goes on to its last tile: the issuer waits for it without a limit)
        ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded(&sfull[a], s_n++ & 1, &s_abort));
        if (!ok) s_abort = 1;
        if (t > 0) released();  // V(t - 1)
        released();             // K(t)
        tc_fence_after();
        const bool edge = t * kKeys + kKeys - 1 > first;  // some row does not see all of the tile's keys
        // Weights are taken by the reference there is, the first tile's maximum at first.  Their sum tells where scores have
        // outgrown it (no weight is larger than the sum, so V of up to 2^-8 of float32's range stays within it; what overflows
        // shows as well): tile_again then does the tile once more, by its maximum.  (So does a row that has seen nothing but
        // -inf, whose reference is none yet.)  No other tile needs one, which is a pass less on the way from S to P.  The
        // reference lies kPromptHead above that maximum, so that a tile's scores have to grow by e^9 before it moves (on the
        // maximum itself by 2, and then some row of a warp goes through its tile again nearly every time: prompts whose scores
        // rise by e^10 from their first row to their last take 58 us so, 33 as it is; 2048 rows, 32 heads on 8).
        bool mine = false, again = false;
        if (ok) {
          uint32_t s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_x32(tS + c * 32, s[c]);
          tmem_ld_wait_for(s);
          if (edge) {
            const int lim = row - t * kKeys;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (__any_sync(0xffffffffu, lim < c * 32 + 31)) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (c * 32 + j > lim) s[c][j] = 0xff800000u;
              }
          }
          if (t == 0) {
            float first_mx[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              first_mx[c] = -INFINITY;
#pragma unroll
              for (int j = 0; j < 32; j += 2)
                first_mx[c] = max3(first_mx[c], __uint_as_float(s[c][j]), __uint_as_float(s[c][j + 1]));
            }
            // (128 is no multiple of every G: rows behind the last head have a reference all the same)
            m_run = rl < p.tg * p.G ? max3(fmaxf(first_mx[0], first_mx[1]), first_mx[2], first_mx[3]) + p.head : 0.f;
          }
          // (without a reference: weights that do not count, and tile_again)
          const float shift = (m_run == -INFINITY ? INFINITY : m_run) * p.scale_log2;
          const float2 sc = make_float2(p.scale_log2, p.scale_log2), off = make_float2(-shift, -shift);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          uint32_t pk[2][32];
#pragma unroll
          for (int j = 0; j < kKeys; j += 2) {
            const float s0 = __uint_as_float(s[j / 32][j % 32]), s1 = __uint_as_float(s[j / 32][j % 32 + 1]);
            const float2 x = __ffma2_rn(make_float2(s0, s1), sc, off);
            const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
            sum[(j >> 1) & 1] = __fadd2_rn(sum[(j >> 1) & 1], make_float2(p0, p1));
            pk[j / 64][j % 64 / 2] = pack_bf16x2(p0, p1);
          }
          const float part = (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
          mine = valid && (part > kGrown || fabsf(shift) >= kExact);
          again = __any_sync(0xffffffffu, mine);
          if (!again) {
            l_run += part;
            tmem_st_x32(tP, pk[0]);
            tmem_st_x32(tP + 32, pk[1]);
            tmem_st_wait();
          }
        }
        if (ok && again) {
          const float2 ml = tile_again<D>(tS, tP, tO, edge ? row - t * kKeys : kKeys, mine, t > 0, make_float2(m_run, l_run),
                                          p.head, p.scale_log2);
          m_run = ml.x;
          l_run = ml.y;
        }
        tc_fence_before();
        __syncwarp();
        // (not an arrival alone: a warp whose next wait gives up must not come to the next tile's before the issuer has left
        // this one's)
        named_bar_sync(kBarP + a, 160);
      }
      have = take(next);
      ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded(&ofull[a], o_n++ & 1, &s_abort));
      if (!ok) s_abort = 1;
      released();
      st = (st + 2 * (w.all - w.tiles[a])) % kStages;  // (a group with fewer tiles than the item)
      if (!ok) continue;
      tc_fence_after();
      const size_t orow = valid ? (size_t)(w.r0 + row) * p.Hq + w.g * p.G + my_head : 0;
      // (from the rounded product that the weights were taken by, and near the maximum, so that what the head adds is not rounded)
      const float lse =
          fmaf(__fmul_rn(m_run, p.scale_log2) - kPromptHead, 0.69314718f, logf(l_run * (float)(1 << (int)kPromptHead)));
      const float inv = l_run > 0.f ? 1.f / l_run : (l_run == 0.f ? 0.f : l_run);  // (a NaN sum stays NaN)
      const bool special = *static_cast<volatile int*>(&s_special) != 0;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld_x32(tO + c * 32, o);
        tmem_ld_wait();
        if (c == D / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ofree[a]);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * inv);
        if (special && valid) {
          // V's infinities and NaN that the guard has taken out, of the keys this row sees
          for (int key = w.edge * kKeys; key <= row; ++key) {
            const uint16_t* v = p.v + (size_t)(w.r0 + key) * p.v_stride + (size_t)w.g * D + c * 32;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const uint32_t x = (uint32_t)v[j] << 16;
              if (specials(x)) o[j] = __float_as_uint(__uint_as_float(o[j]) + __uint_as_float(x));
            }
          }
        }
        if (valid) {
          uint32_t y[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = pack_bf16x2(__uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1]));
          store_64(p.out + orow * D + c * 32, y, p.out32);
        }
      }
      if (valid && p.lse) p.lse[orow] = lse;
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
  cudaError_t err = cudaFuncSetAttribute(prompt_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptCfg<D>::kSmem);
  if (err != cudaSuccess) return err;
  return launch_dependent(prompt_attn_kernel<D>, dim3(grid), dim3(kThreads), PromptCfg<D>::kSmem, stream, *tmQ, *tmK, *tmV, p);
}

cudaError_t launch_prompt_attention(int d, const CUtensorMap* tmQ, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                    const PromptAttnParams& p, int grid, cudaStream_t stream) {
  return d == 128 ? launch_as<128>(tmQ, tmK, tmV, p, grid, stream) : launch_as<64>(tmQ, tmK, tmV, p, grid, stream);
}

}  // namespace spectree
