// K12: the attention weight that each key gets from a prompt's last rows.
//
//   weight[g][j] = sum_{i >= j, window} sum_{h in g} 2^(log2(e) (scale q_ih . k_j - lse_ih))
// The second look over a prompt that says which of its keys the answer will read (what a budget keeps is chosen by
// it).  With the log-sum-exp at hand no maximum is needed, and with keys on the M side of the product a key's sum
// over the queries is one thread's walk along its own row of tensor memory: no reduction between threads, no
// atomics, one order of terms.
//
// An item is 256 keys of one request and KV head, as two groups of 128 (the M of an MMA); the window's rows times
// the G heads come past them in chunks of tc = 128 / G rows (N).  K is read once; Q chunks come from L2.  2 d
// operations per pair against 2 d bytes per key: a window of 64 rows with 4 heads a group is where HBM and the
// exponentials take equally long.
//
// Roles (10 warps): warp 0 TMA (two slots of 256 keys, three of a Q chunk), warp 1 MMA issuer, warps 2-9 sums, four per
// group, each group with two score buffers of 128 columns, so that the products run while sums are taken.

#include "pdl.cuh"
#include "prompt.cuh"
#include "tc_ptx.cuh"

namespace spectree {

namespace {

constexpr int kKeys = 128;   // keys per group
constexpr int kCols = 128;   // query rows per chunk
constexpr int kThreads = 320;
constexpr int kKSlots = 2, kQSlots = 3;

template <int D>
struct WeightCfg {
  static constexpr int kK = kKeys * D * 2;   // a group's keys
  static constexpr int kQ = kCols * D * 2;
  static constexpr int kSmem = 1024 + kKSlots * 2 * kK + kQSlots * kQ;
};

struct Work {
  int r0, n, key, g;  // first key of the item
  int q0, chunks;     // the window's first row and its chunks
  int groups;
};

__device__ __forceinline__ Work work_of(const KeyWeightsParams& p, const PlanReader& plan, int at) {
  const PromptItem it = plan.item(at / p.Hkv);
  Work w;
  w.r0 = it.r0;
  w.n = it.n;
  w.key = it.tok;
  w.g = at % p.Hkv;
  w.q0 = it.n > p.window ? it.n - p.window : 0;
  w.chunks = (it.n - w.q0 + p.tc - 1) / p.tc;
  w.groups = it.n - it.tok > kKeys ? 2 : 1;
  return w;
}
// Chunks are taken from the window's end; those that no key of a group is visible to are left out, which are the last.
__device__ __forceinline__ int chunk_row(const KeyWeightsParams& p, const Work& w, int c) {
  return w.q0 + (w.chunks - 1 - c) * p.tc;
}
__device__ __forceinline__ int chunks_of(const KeyWeightsParams& p, const Work& w, int a) {
  if (a >= w.groups) return 0;
  const int first = w.key + a * kKeys;             // the group's first key: rows before it see none of them
  const int skip = first > w.q0 ? (first - w.q0) / p.tc : 0;
  return w.chunks - skip;                          // (first < n, so one chunk at least is left)
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const KeyWeightsParams p) {
  using C = WeightCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = base;                          // [slot][group][d / 64][128 keys][128 B]
  uint8_t* sQ = base + kKSlots * 2 * C::kK;    // [slot][d / 64][128 rows][128 B]
  __shared__ uint64_t kfull[kKSlots], kempty[kKSlots], qfull[kQSlots], qempty[kQSlots];
  __shared__ uint64_t sfull[4], sfree[4];      // [group][buffer]
  __shared__ uint64_t drained;
  __shared__ __align__(16) float s_lse[2][kCols];  // [group]: log2(e) lse of the chunk's columns, +inf behind the window
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kKSlots; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 1);
    }
    for (int s = 0; s < kQSlots; ++s) {
      mbar_init(&qfull[s], 1);
      mbar_init(&qempty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sfree[s], 4);
    }
    mbar_init(&drained, 1);
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
  const PlanReader plan(p.plan, p.dev_status);
  const int total = plan.count * p.Hkv;

  if (warp == 0) {
    // ---- TMA producer ----
    if (lane == 0) {
      uint32_t k_n = 0, q_n = 0;
      bool ok = true;
      for (int at = blockIdx.x; ok && at < total; at += gridDim.x) {
        const Work w = work_of(p, plan, at);
        const int ks = k_n % kKSlots;
        ok = mbar_wait_bounded(&kempty[ks], ((k_n / kKSlots) & 1) ^ 1, &s_abort);
        if (!ok) break;
        mbar_arrive_expect_tx(&kfull[ks], w.groups * C::kK);
        for (int a = 0; a < w.groups; ++a)
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sK + (ks * 2 + a) * C::kK + c * kKeys * 128, &tmK, &kfull[ks], c * 64, w.g, w.r0 + w.key + a * kKeys);
        ++k_n;
        const int chunks = chunks_of(p, w, 0);  // group 0 has the earlier keys, so no fewer than group 1
        for (int c = 0; ok && c < chunks; ++c) {
          const int qs = q_n % kQSlots;
          ok = mbar_wait_bounded(&qempty[qs], ((q_n / kQSlots) & 1) ^ 1, &s_abort);
          if (!ok) break;
          mbar_arrive_expect_tx(&qfull[qs], (D / 64) * p.tc * p.G * 128);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(sQ + qs * C::kQ + h * kCols * 128, &tmQ, &qfull[qs], h * 64, w.g * p.G, w.r0 + chunk_row(p, w, c));
          ++q_n;
        }
      }
      if (!ok) {
        s_abort = 1;
        set_status(p.dev_status, SPEC_ERR_TIMEOUT);
        for (uint32_t s = 0; s < kKSlots; ++s) {  // what is under way lands first: the last load of every slot
          const uint32_t n = (k_n + kKSlots - 1 - s) / kKSlots;
          if (n) mbar_wait_bounded(&kfull[s], (n - 1) & 1, nullptr);
        }
        for (uint32_t s = 0; s < kQSlots; ++s) {
          const uint32_t n = (q_n + kQSlots - 1 - s) / kQSlots;
          if (n) mbar_wait_bounded(&qfull[s], (n - 1) & 1, nullptr);
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer ----
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16_f32(kKeys, kCols, 0);
      uint32_t k_n = 0, q_n = 0, s_n[2] = {0, 0};
      bool ok = true;
      for (int at = blockIdx.x; ok && at < total; at += gridDim.x) {
        const Work w = work_of(p, plan, at);
        const int ks = k_n % kKSlots;
        ok = mbar_wait_bounded(&kfull[ks], (k_n / kKSlots) & 1, &s_abort);
        const int chunks[2] = {chunks_of(p, w, 0), chunks_of(p, w, 1)};
        for (int c = 0; ok && c < chunks[0]; ++c) {
          const int qs = q_n % kQSlots;
          ok = mbar_wait_bounded(&qfull[qs], (q_n / kQSlots) & 1, &s_abort);
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            if (!ok || c >= chunks[a]) continue;
            const int buf = a * 2 + (s_n[a] & 1);
            ok = mbar_wait_bounded(&sfree[buf], ((s_n[a] >> 1) & 1) ^ 1, &s_abort);
            if (!ok) continue;
            ++s_n[a];
            tc_fence_after();
            const uint32_t ka = smem_u32(sK + (ks * 2 + a) * C::kK), qa = smem_u32(sQ + qs * C::kQ);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_bf16(tmem + buf * kCols, sdesc_sw128(ka + (kk >> 2) * (kKeys * 128) + (kk & 3) * 32, 0, 1024),
                        sdesc_sw128(qa + (kk >> 2) * (kCols * 128) + (kk & 3) * 32, 0, 1024), idS, kk > 0);
            umma_commit(&sfull[buf]);
          }
          if (!ok) break;
          umma_commit(&qempty[qs]);
          ++q_n;
        }
        if (ok) umma_commit(&kempty[ks]);
        ++k_n;
      }
      if (!ok) {
        s_abort = 1;
        set_status(p.dev_status, SPEC_ERR_TIMEOUT);
      }
      umma_commit(&drained);
      mbar_wait_bounded(&drained, 0, nullptr);
    }
  } else {
    // ---- sums: group a, one key per thread ----
    const int a = (warp - 2) >> 2, q4 = warp & 3;
    const int kl = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const int col_tok = kl / p.G, col_head = kl - col_tok * p.G;  // the column whose lse this thread fetches
    uint32_t s_n = 0;
    bool ok = true;
    // A warp whose wait gave up goes on with its group's barriers to the last item: no wait takes long any more.
    for (int at = blockIdx.x; at < total; at += gridDim.x) {
      const Work w = work_of(p, plan, at);
      const int chunks = chunks_of(p, w, a);
      if (chunks == 0) continue;
      const int key = w.key + a * kKeys + kl, last_key = w.key + a * kKeys + kKeys - 1;
      float total_w = 0.f;
      auto fetch = [&](int c) {  // log2(e) lse of this thread's column
        const int row = chunk_row(p, w, c) + col_tok;
        return col_tok < p.tc && row < w.n ? p.lse[(size_t)(w.r0 + row) * p.Hq + w.g * p.G + col_head] * 1.4426950408889634f
                                           : INFINITY;
      };
      float next = fetch(0);
      for (int c = 0; c < chunks; ++c) {
        const float* lse = s_lse[a];
        named_bar_sync(1 + a, 128);  // the chunk before has been read
        s_lse[a][kl] = next;
        named_bar_sync(1 + a, 128);
        if (c + 1 < chunks) next = fetch(c + 1);
        const int buf = a * 2 + (s_n & 1);
        ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded(&sfull[buf], (s_n >> 1) & 1, &s_abort));
        if (!ok) s_abort = 1;
        const int row0 = chunk_row(p, w, c);
        // columns [lo, hi) count: rows from this key on, inside the window
        const bool edge = row0 < last_key || row0 + p.tc > w.n || p.tc * p.G < kCols;
        const int lo = key > row0 ? (key - row0) * p.G : 0;
        const int hi = (w.n - row0 < p.tc ? w.n - row0 : p.tc) * p.G;
        tc_fence_after();
        const float2 sc = make_float2(p.scale_log2, p.scale_log2);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 2
        for (int q = 0; q < kCols; q += 32) {
          uint32_t s[32];
          if (ok) {
            tmem_ld_x32(tmem + buf * kCols + q + lane_off, s);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] = 0u;
          }
          if (edge) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (q + j < lo || q + j >= hi) s[j] = 0xff800000u;
          }
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(lse + q + j);
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), sc, make_float2(-l4.x, -l4.y));
            const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[j + 2]), __uint_as_float(s[j + 3])), sc, make_float2(-l4.z, -l4.w));
            sum[0] = __fadd2_rn(sum[0], make_float2(ex2_approx(x.x), ex2_approx(x.y)));
            sum[1] = __fadd2_rn(sum[1], make_float2(ex2_approx(y.x), ex2_approx(y.y)));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfree[buf]);
        ++s_n;
        total_w += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
      }
      if (!ok) {
        if (lane == 0) {
          s_abort = 1;
          set_status(p.dev_status, SPEC_ERR_TIMEOUT);
        }
      } else if (key < w.n) {
        p.weight[(size_t)w.g * p.n_rows + w.r0 + key] = total_w;
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D>
static cudaError_t launch_as(const CUtensorMap* tmQ, const CUtensorMap* tmK, const KeyWeightsParams& p, int grid,
                             cudaStream_t stream) {
  const cudaError_t err =
      cudaFuncSetAttribute(key_weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, WeightCfg<D>::kSmem);
  if (err != cudaSuccess) return err;
  return launch_dependent(key_weights_kernel<D>, dim3(grid), dim3(kThreads), WeightCfg<D>::kSmem, stream, *tmQ, *tmK, p);
}

cudaError_t launch_key_weights(int d, const CUtensorMap* tmQ, const CUtensorMap* tmK, const KeyWeightsParams& p, int grid,
                               cudaStream_t stream) {
  return d == 128 ? launch_as<128>(tmQ, tmK, p, grid, stream) : launch_as<64>(tmQ, tmK, p, grid, stream);
}

}  // namespace spectree
