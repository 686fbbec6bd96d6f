// K12: the attention weight that each key gets from a prompt's last rows.
//
//   weight[g][j] = sum_{i >= j, window} sum_{h in g} 2^(log2(e) (scale q_ih . k_j - lse_ih))
// The second look over a prompt that says which of its keys the answer will read (what a budget keeps is chosen by
// it).  With the log-sum-exp at hand no maximum is needed, and with keys on the M side of the product a key's sum
// over the queries is one thread's walk along its own row of tensor memory: no reduction between threads, no
// atomics, one order of terms.
//
// Keys come in tiles of 128 (the M of an MMA); every CTA has an even share of all tiles, in stretches of one request and KV
// head.  The window's rows times the G heads are the columns (N), in chunks of tc = 128 / G rows, up to three of which
// stay in shared memory with their lse while the stretch's keys stream past.  Longer windows take several such passes over a
// stretch (its keys come from L2 then), the later ones adding to what the earlier ones wrote.  K is read once, 2 d
// bytes for 2 d operations a column: a window of 64 rows with 4 heads a group is where HBM, MMA and exponentials
// (512 cycles for 128 x 128 of each) take equally long.
//
// Roles (12 warps): warp 0 TMA (a ring of key tiles, three slots of query chunks), warp 3 the chunks' lse, warps 4-11 sums:
// two groups of four warps take every other key tile, each with two score buffers of 128 columns, so that products run
// while sums are taken; warps 1 and 2 issue their MMAs.
//
// What bounds it: 8 prompts of 512 to 32768 rows, 64 heads on 8, window 37: 89.1 us where the bytes take 41.5; loads and
// hand-offs alone 59, with the MMAs 77, and exponentials fill in only as far as two groups overlap (three groups 148 us, four
// with one buffer each 122: less room for keys and queries).  One prompt of 16384 rows, window 64: 13.2 us with 32 heads on 8
// (of which a launch, a start and seven tiles one behind the other), 20.6 with 40 on 8, where no chunk is a whole one; 9.3 with
// 32 on 8 and window 16.

#include "pdl.cuh"
#include "prompt.cuh"
#include "tc_ptx.cuh"

namespace spectree {

namespace {

constexpr int kKeys = 128;   // keys per tile
constexpr int kCols = 128;   // columns per chunk at most
constexpr int kThreads = 384;
constexpr int kKSlots = 4, kQSlots = 3;

template <int D>
struct WeightCfg {
  static constexpr int kK = kKeys * D * 2;
  static constexpr int kQ = kCols * D * 2;
  static constexpr int kSmem = 1024 + kKSlots * kK + kQSlots * kQ;
};

// (in the order it is written)
__device__ __forceinline__ float4 lds_f4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}
struct Work {
  int r0, n, key, g;   // first key
  int tiles;
  int q0, chunks;      // the window's first row and its chunks
  int passes, per;     // passes over the keys, chunks of a pass
};

// The CTA's tiles are an even share [at, end) of all: the plan's pieces of 128 keys, head after head.  A stretch is what
// one request and head have of it.
template <bool FEW>
__device__ __forceinline__ Work work_of(const KeyWeightsParams& p, const PlanReader<FEW>& plan, int at, int end) {
  Work w;
  w.g = at / plan.count;
  const PromptItem it = plan.item(at - w.g * plan.count);
  w.r0 = it.r0;
  w.n = it.n;
  w.key = it.tok;
  const int tiles = (it.n - it.tok + kKeys - 1) / kKeys;
  w.tiles = tiles < end - at ? tiles : end - at;
  w.q0 = it.n > p.window ? it.n - p.window : 0;
  w.chunks = (it.n - w.q0 + p.tc - 1) / p.tc;
  w.passes = (w.chunks + kQSlots - 1) / kQSlots;
  w.per = (w.chunks + w.passes - 1) / w.passes;
  return w;
}
// The pass's chunks that some key of tile `i` is visible to: [first, end).  Later tiles need fewer of them.
struct Chunks {
  int first, end;
};
__device__ __forceinline__ Chunks chunks_of(const KeyWeightsParams& p, const Work& w, int pass, int i) {
  const int key = w.key + i * kKeys;
  const int first = key > w.q0 ? (key - w.q0) / p.tc : 0;  // the chunk of the first row that sees the tile's first key
  Chunks c;
  c.first = first > pass * w.per ? first : pass * w.per;
  c.end = (pass + 1) * w.per < w.chunks ? (pass + 1) * w.per : w.chunks;
  return c;
}
// The chunk that comes as the u-th for tile `i`.  Every other tile of a request takes them backwards, and so one of the two
// groups does: a short last chunk of one beside a whole one of the other, as two groups in step would want the exponentials'
// unit at the same time (8 prompts 90.9 us in step, 89.1 so).  By the request's own tiles, not by the group, which depends
// on the batch: a key's terms are added in one order whatever comes with it.
__device__ __forceinline__ int turned(const Work& w, const Chunks& c, int u, int i) {
  return (w.key / kKeys + i) & 1 ? c.first + c.end - 1 - u : u;
}
// Rows of chunk c in the window.
__device__ __forceinline__ int chunk_rows(const KeyWeightsParams& p, const Work& w, int c) {
  const int left = w.n - w.q0 - c * p.tc;
  return left < p.tc ? left : p.tc;
}

}  // namespace

template <int D, bool FEW>
__global__ void __launch_bounds__(kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const KeyWeightsParams p) {
  using C = WeightCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = base;                      // [slot][d / 64][128 keys][128 B]
  uint8_t* sQ = base + kKSlots * C::kK;    // [slot][d / 64][128 rows][128 B]
  __shared__ uint64_t kfull[kKSlots], kempty[kKSlots], qfull[kQSlots], qempty[kQSlots];
  __shared__ uint64_t sfull[4], sfree[4];  // [group][buffer]
  __shared__ uint64_t lfull, lfree;        // the pass's lse written, read
  __shared__ uint64_t drained[2];
  __shared__ __align__(16) float s_lse[kQSlots][kCols];  // log2(e) lse, +inf behind the window
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ PlanShared s_plan;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kKSlots; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 1);
    }
    for (int s = 0; s < kQSlots; ++s) {
      mbar_init(&qfull[s], 1);
      mbar_init(&qempty[s], 2);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sfree[s], 4);
    }
    mbar_init(&lfull, 1);
    mbar_init(&lfree, 8);
    mbar_init(&drained[0], 1);
    mbar_init(&drained[1], 1);
    s_abort = 0;
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
  const PlanReader<FEW> plan(p.plan, s_plan, p.dev_status);
  int begin, end;
  if (p.per_head) {  // neighbouring CTAs take the same keys of neighbouring heads, which lie together in memory
    const int head = blockIdx.x % p.Hkv;
    const long long i = blockIdx.x / p.Hkv;
    // (one tile more than there are: the batch's last one, at its window's edge, counts twice.  One prompt of 16K 14.6 us
    // without, 13.2 so)
    begin = (int)((plan.count + 1) * i / p.per_head);
    end = (int)((plan.count + 1) * (i + 1) / p.per_head);
    begin = head * plan.count + (begin < plan.count ? begin : plan.count);
    end = head * plan.count + (end < plan.count ? end : plan.count);
  } else {
    const long long total = (long long)plan.count * p.Hkv;
    begin = (int)(total * blockIdx.x / gridDim.x);
    end = (int)(total * (blockIdx.x + 1) / gridDim.x);
  }
  bool ok = true;

  if (warp == 0) {
    // ---- TMA producer ----
    if (lane == 0) {
      uint32_t k_n = 0, q_n[kQSlots] = {0, 0, 0};
      Work w;
      for (int at = begin; ok && at < end; at += w.tiles) {
        w = work_of(p, plan, at, end);
        for (int pass = 0; ok && pass < w.passes; ++pass) {
          for (int i = 0; ok && i < w.tiles; ++i) {
            const Chunks c = chunks_of(p, w, pass, i);
            if (c.first >= c.end) break;  // (so do all later tiles)
            const int ks = k_n % kKSlots;
            ok = mbar_wait_bounded(&kempty[ks], ((k_n / kKSlots) & 1) ^ 1, &s_abort);
            if (!ok) break;
            mbar_arrive_expect_tx(&kfull[ks], C::kK);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(sK + ks * C::kK + h * kKeys * 128, &tmK, &kfull[ks], h * 64, w.g, w.r0 + w.key + i * kKeys);
            ++k_n;
            if (i > 0) continue;
#pragma unroll
            for (int s = 0; s < kQSlots; ++s) {  // the first tile needs every chunk that any tile needs
              const int ch = pass * w.per + s;
              if (!ok || ch < c.first || ch >= c.end) continue;
              ok = mbar_wait_bounded(&qempty[s], (q_n[s] & 1) ^ 1, &s_abort);
              if (!ok) continue;
              mbar_arrive_expect_tx(&qfull[s], (D / 64) * p.tc * p.G * 128);
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_load_3d(sQ + s * C::kQ + h * kCols * 128, &tmQ, &qfull[s], h * 64, w.g * p.G, w.r0 + w.q0 + ch * p.tc);
              ++q_n[s];
            }
          }
        }
      }
      if (!ok) {
        s_abort = 1;
        set_status(p.dev_status, SPEC_ERR_TIMEOUT);
        for (uint32_t s = 0; s < kKSlots; ++s) {  // what is under way lands first: the last load of every slot
          const uint32_t n = (k_n + kKSlots - 1 - s) / kKSlots;
          if (n) mbar_wait_bounded(&kfull[s], (n - 1) & 1, nullptr);
        }
#pragma unroll
        for (int s = 0; s < kQSlots; ++s)
          if (q_n[s]) mbar_wait_bounded(&qfull[s], (q_n[s] - 1) & 1, nullptr);
      }
    }
  } else if (warp < 3) {
    // ---- MMA issuer of group a (one for both would wait for one group's buffers while the other runs dry) ----
    if (lane == 0) {
      const int a = warp - 1;
      const uint32_t k_lo0 = smem_u32(sK) >> 4, q_lo0 = smem_u32(sQ) >> 4;
      uint32_t k_n = 0, q_n[kQSlots] = {0, 0, 0}, s_n = 0;
      Work w;
      for (int at = begin; ok && at < end; at += w.tiles) {
        w = work_of(p, plan, at, end);
        for (int pass = 0; ok && pass < w.passes; ++pass) {
          const Chunks all = chunks_of(p, w, pass, 0);
          if (all.first >= all.end) continue;
#pragma unroll
          for (int s = 0; s < kQSlots; ++s) {
            const int ch = pass * w.per + s;
            if (ch >= all.first && ch < all.end) ok = ok && mbar_wait_bounded(&qfull[s], q_n[s]++ & 1, &s_abort);
          }
          for (int i = 0; ok && i < w.tiles; ++i) {
            const Chunks c = chunks_of(p, w, pass, i);
            if (c.first >= c.end) break;
            const int ks = k_n % kKSlots;
            const uint32_t k_phase = (k_n / kKSlots) & 1;
            if ((int)(k_n++ & 1) != a) continue;   // (slots alternate as groups do: each sees every phase of its own)
            ok = mbar_wait_bounded(&kfull[ks], k_phase, &s_abort);
            const uint32_t k_lo = k_lo0 + ks * (C::kK >> 4);
            for (int u = c.first; u < c.end; ++u) {
              const int ch = turned(w, c, u, i);
              const int buf = a * 2 + (s_n & 1);
              ok = ok && mbar_wait_bounded(&sfree[buf], ((s_n >> 1) & 1) ^ 1, &s_abort);
              if (!ok) break;
              ++s_n;
              tc_fence_after();
              // as many columns as the chunk has, in steps of 16
              const uint32_t idS = idesc_bf16_f32(kKeys, (chunk_rows(p, w, ch) * p.G + 15) & ~15, 0);
              const uint32_t q_lo = q_lo0 + (ch - pass * w.per) * (C::kQ >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * ((kKeys * 128) >> 4) + (kk & 3) * 2;
                umma_bf16(tmem + buf * kCols, desc_sw128(k_lo + off), desc_sw128(q_lo + off), idS, kk > 0);
              }
              umma_commit(&sfull[buf]);
            }
            if (ok) umma_commit(&kempty[ks]);
          }
#pragma unroll
          for (int s = 0; s < kQSlots; ++s) {
            const int ch = pass * w.per + s;
            if (ok && ch >= all.first && ch < all.end) umma_commit(&qempty[s]);
          }
        }
      }
      if (!ok) {
        s_abort = 1;
        set_status(p.dev_status, SPEC_ERR_TIMEOUT);
      }
      umma_commit(&drained[a]);
      mbar_wait_bounded(&drained[a], 0, nullptr);
    }
  } else if (warp == 3) {
    // ---- the chunks' lse: four columns per thread and chunk, fetched while the pass before is under way ----
    uint32_t l_n = 0;
    Work w;
    for (int at = begin; ok && at < end; at += w.tiles) {
      w = work_of(p, plan, at, end);
      for (int pass = 0; ok && pass < w.passes; ++pass) {
        float x[kQSlots][4];
#pragma unroll
        for (int s = 0; s < kQSlots; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int ch = pass * w.per + s, col = lane + 32 * e, tok = col / p.G;
            const bool there = s < w.per && ch < w.chunks && tok < chunk_rows(p, w, ch);
            x[s][e] = there ? p.lse[(size_t)(w.r0 + w.q0 + ch * p.tc + tok) * p.Hq + w.g * p.G + col - tok * p.G] *
                                  1.4426950408889634f
                            : INFINITY;
          }
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&lfree, (l_n & 1) ^ 1, &s_abort));
        if (!ok) break;
#pragma unroll
        for (int s = 0; s < kQSlots; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) s_lse[s][lane + 32 * e] = x[s][e];
        __syncwarp();
        if (lane == 0) mbar_arrive(&lfull);
        ++l_n;
      }
    }
    if (!ok && lane == 0) {
      s_abort = 1;
      set_status(p.dev_status, SPEC_ERR_TIMEOUT);
    }
  } else {
    // ---- sums: group a, one key per thread ----
    const int a = (warp - 4) >> 2, q4 = warp & 3;
    const int kl = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const float2 sc = make_float2(p.scale_log2, p.scale_log2);
    uint32_t k_n = 0, s_n = 0, l_n = 0;
    Work w;
    for (int at = begin; ok && at < end; at += w.tiles) {
      w = work_of(p, plan, at, end);
      float* weight = p.weight + (size_t)w.g * p.n_rows + w.r0;
      for (int pass = 0; ok && pass < w.passes; ++pass) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&lfull, l_n++ & 1, &s_abort));
        for (int i = 0; ok && i < w.tiles; ++i) {
          const Chunks c = chunks_of(p, w, pass, i);
          const int key0 = w.key + i * kKeys, key = key0 + kl;
          if (c.first >= c.end) {  // nothing of this pass: group 0 writes what pass 0 has to
            if (pass == 0 && a == 0 && key < w.n) weight[key] = 0.f;
            continue;
          }
          if ((int)(k_n++ & 1) != a) continue;
          float sum_w = pass > 0 && key < w.n ? weight[key] : 0.f;
          for (int u = c.first; u < c.end; ++u) {
            const int ch = turned(w, c, u, i);
            const int buf = a * 2 + (s_n & 1);
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sfull[buf], (s_n >> 1) & 1, &s_abort));
            if (!ok) break;
            ++s_n;
            const float* lse = s_lse[ch - pass * w.per];
            const int row0 = w.q0 + ch * p.tc;
            // columns [lo, cols) count: rows from this key on, inside the window
            const int cols = chunk_rows(p, w, ch) * p.G;
            const int lo = key > row0 ? (key - row0) * p.G : 0;
            const bool edge = row0 < key0 + kKeys - 1;
            tc_fence_after();
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const uint32_t tS = tmem + buf * kCols + lane_off;
            if (cols == kCols && !edge) {
              // a whole chunk: its 128 columns in one go, their lse eight reads ahead (in blocks of 64 columns, as below,
              // 8 prompts take 108 us instead of 89; reads that the compiler may move came first, all of them, and
              // registers ran out, in an earlier form of this loop)
              uint32_t s[4][32];
#pragma unroll
              for (int b = 0; b < 4; ++b) tmem_ld_x32(tS + b * 32, s[b]);
              const uint32_t at_lse = smem_u32(lse);
              float4 ahead[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) ahead[j] = lds_f4(at_lse + j * 16);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < kCols; j += 4) {
                const float4 l4 = ahead[j / 4 % 8];
                if (j + 32 < kCols) ahead[j / 4 % 8] = lds_f4(at_lse + (j + 32) * 4);
                const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[j / 32][j % 32]), __uint_as_float(s[j / 32][j % 32 + 1])),
                                            sc, make_float2(-l4.x, -l4.y));
                const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[j / 32][j % 32 + 2]), __uint_as_float(s[j / 32][j % 32 + 3])),
                                            sc, make_float2(-l4.z, -l4.w));
                sum[0] = __fadd2_rn(sum[0], make_float2(ex2_approx(x.x), ex2_approx(x.y)));
                sum[1] = __fadd2_rn(sum[1], make_float2(ex2_approx(y.x), ex2_approx(y.y)));
              }
            } else {
#pragma unroll 1
            for (int q = 0; q < cols; q += 64) {
              uint32_t s[2][32];
              tmem_ld_x32(tS + q, s[0]);
              if (q + 32 < cols) tmem_ld_x32(tS + q + 32, s[1]);
              tmem_ld_wait();
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const int q1 = q + b * 32;
                if (q1 >= cols) break;
                if (edge) {  // (masked behind the lse, which may be infinite or NaN where a row does not count)
#pragma unroll
                  for (int j = 0; j < 32; ++j) {
                    const float x = fmaf(__uint_as_float(s[b][j]), p.scale_log2, -lse[q1 + j]);
                    s[b][j] = __float_as_uint(q1 + j < lo || q1 + j >= cols ? -INFINITY : x);
                  }
#pragma unroll
                  for (int j = 0; j < 32; j += 4) {
                    const float x0 = __uint_as_float(s[b][j]), x1 = __uint_as_float(s[b][j + 1]);
                    const float x2 = __uint_as_float(s[b][j + 2]), x3 = __uint_as_float(s[b][j + 3]);
                    sum[0] = __fadd2_rn(sum[0], make_float2(ex2_approx(x0), ex2_approx(x1)));
                    sum[1] = __fadd2_rn(sum[1], make_float2(ex2_approx(x2), ex2_approx(x3)));
                  }
                  continue;
                }
                if (q1 + 32 > cols) {
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if (q1 + j >= cols) s[b][j] = 0xff800000u;  // (whose lse is +inf)
                }
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                  const float4 l4 = *reinterpret_cast<const float4*>(lse + q1 + j);
                  const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[b][j]), __uint_as_float(s[b][j + 1])), sc,
                                              make_float2(-l4.x, -l4.y));
                  const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[b][j + 2]), __uint_as_float(s[b][j + 3])), sc,
                                              make_float2(-l4.z, -l4.w));
                  sum[0] = __fadd2_rn(sum[0], make_float2(ex2_approx(x.x), ex2_approx(x.y)));
                  sum[1] = __fadd2_rn(sum[1], make_float2(ex2_approx(y.x), ex2_approx(y.y)));
                }
              }
            }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sfree[buf]);
            sum_w += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
          }
          if (ok && key < w.n) weight[key] = sum_w;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&lfree);
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

template <int D, bool FEW>
static cudaError_t launch_as(const CUtensorMap* tmQ, const CUtensorMap* tmK, const KeyWeightsParams& p, int grid,
                             cudaStream_t stream) {
  const cudaError_t err =
      cudaFuncSetAttribute(key_weights_kernel<D, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize, WeightCfg<D>::kSmem);
  if (err != cudaSuccess) return err;
  return launch_dependent(key_weights_kernel<D, FEW>, dim3(grid), dim3(kThreads), WeightCfg<D>::kSmem, stream, *tmQ, *tmK, p);
}

cudaError_t launch_key_weights(int d, const CUtensorMap* tmQ, const CUtensorMap* tmK, const KeyWeightsParams& p, int grid,
                               cudaStream_t stream) {
  if (!p.plan.items && p.plan.B > 1)
    return d == 128 ? launch_as<128, true>(tmQ, tmK, p, grid, stream) : launch_as<64, true>(tmQ, tmK, p, grid, stream);
  return d == 128 ? launch_as<128, false>(tmQ, tmK, p, grid, stream) : launch_as<64, false>(tmQ, tmK, p, grid, stream);
}

}  // namespace spectree
