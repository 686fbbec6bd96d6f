// Parameters, device helpers and launches of the kernels that take prompts to the cache: positions and their
// rotation, causal attention over packed prompts, key weights and the rows kept for a budget.
#pragma once

#include "common.cuh"

namespace spectree {

// ---- K10: positions, rotation -----------------------------------------------------------------
struct PositionsParams {
  int B, N;
  long long n_rows;
  const int32_t* pos0;       // [B]
  const int32_t* row_start;  // [B + 1] (packed rows) or nullptr
  const int32_t* parent;     // [B][N] (trees) or nullptr
  const int32_t* n_nodes;
  int32_t* positions;        // [n_rows] or [B][N]
  int fill;                  // packed rows: -1 for rows of no request
  int32_t* dev_status;
};
cudaError_t launch_rope_positions(const PositionsParams& p, cudaStream_t stream);

struct RopeParams {
  int is_bf16, interleaved, Hq, Hk, d, rot;
  long long n_rows;
  long long q_stride, k_stride, q_out_stride, k_out_stride;
  float amplitude;
  const void* q;
  const void* k;
  const int32_t* positions;
  const int64_t* turns;
  void* q_out;
  void* k_out;
};
cudaError_t launch_rope(const RopeParams& p, int num_sms, cudaStream_t stream);

// ---- the plan of a call over packed rows -------------------------------------------------------
// A work item: `tokens` rows of one request from row `tok` on; the kernels take every KV head of it.
struct PromptItem {
  int r0;   // the request's first row
  int n;    // its rows
  int tok;  // the item's first row, counted in the request
  int pad;
};
// Cuts [from(n), n) of every request into pieces of `step` rows and lists them; count[0] = items, 0 for a bad
// row_start (SPEC_ERR_CAPACITY).  by_work: the items with the most keys behind them first.
struct PlanParams {
  int B, step, by_work;
  long long n_rows;
  const int32_t* row_start;
  PromptItem* items;
  int32_t* count;
  int32_t* dev_status;
};
// Items that a plan can hold at most.
inline long long plan_items(long long n_rows, int B, int step) { return n_rows / step + (B < n_rows ? B : n_rows); }
cudaError_t launch_prompt_plan(const PlanParams& p, cudaStream_t stream);

// What a kernel reads of its plan.  Without a list (items == nullptr) it finds the pieces in row_start itself, which saves
// the 3 to 4 us of another kernel ahead: those of a single request in order or (by_work) the last first and, in a kernel of the
// key weights' own (FEW), those of up to kPlanInKernel requests in order (8 prompts 93.2 to 89.1 us; code that does both
// took 0.4 us longer for a single one, and 1.1 us in the attention).
constexpr int kPlanInKernel = 32;
struct PlanView {
  const PromptItem* items;
  const int32_t* count;
  const int32_t* row_start;
  long long n_rows;
  int B, step, by_work;
};
struct PlanShared {
  int first[kPlanInKernel + 1];  // pieces before each request
  int start[kPlanInKernel + 1];  // its row_start
};
template <bool FEW>
struct PlanReader {
  const PlanView& v;
  const PlanShared& s;
  int count, r0, n;
  // By all threads of the block.
  __device__ __forceinline__ PlanReader(const PlanView& view, PlanShared& shared, int32_t* dev_status) : v(view), s(shared) {
    r0 = n = 0;
    bool ok = true;
    if (!FEW && v.items) {
      count = v.count[0];
    } else if (!FEW) {
      r0 = v.row_start[0];
      n = v.row_start[1] - r0;
      ok = r0 >= 0 && v.row_start[1] >= r0 && v.row_start[1] <= v.n_rows;
      count = ok ? (int)(((long long)n + v.step - 1) / v.step) : 0;
    } else {
      if (threadIdx.x < 32) {
        const int b = threadIdx.x;
        const int lo = b < v.B ? v.row_start[b] : 0, hi = b < v.B ? v.row_start[b + 1] : 0;
        ok = !__any_sync(0xffffffffu, lo < 0 || hi < lo || hi > v.n_rows);
        int sum = ok ? (int)(((long long)hi - lo + v.step - 1) / v.step) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, sum, o);
          if (b >= o) sum += y;
        }
        if (b < v.B) shared.start[b] = lo, shared.start[b + 1] = hi;  // (neighbours write the same)
        shared.first[b + 1] = sum;
        if (b == 0) shared.first[0] = 0;
      }
      __syncthreads();
      count = s.first[v.B];
    }
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) set_status(dev_status, SPEC_ERR_CAPACITY);
  }
  __device__ __forceinline__ PromptItem item(int i) const {
    if (!FEW && v.items) return v.items[i];
    PromptItem it;
    it.pad = 0;
    if (!FEW) {
      it.r0 = r0;
      it.n = n;
      it.tok = (v.by_work ? count - 1 - i : i) * v.step;
      return it;
    }
    int b = 0;  // the last request with first <= i (those without pieces share their follower's)
#pragma unroll 1
    for (int half = kPlanInKernel / 2; half > 0; half >>= 1)
      if (b + half < v.B && s.first[b + half] <= i) b += half;
    it.r0 = s.start[b];
    it.n = s.start[b + 1] - it.r0;
    it.tok = (i - s.first[b]) * v.step;
    return it;
  }
};

// ---- K11: causal attention over packed prompts --------------------------------------------------
// log2: the largest weight when a row's reference is taken is 2^-12.  Larger, and what V's smallest numbers leave in O would
// leave float32 (at 2^-16, rows of V near 2^-126 come out with 30 % more error; at 2^-12 as without).
constexpr float kPromptHead = 12.f;
struct PromptAttnParams {
  int Hq, Hkv, G, tg;       // tg: rows of a request per 128-row group (128 / G)
  float scale_log2;
  float head;               // how far a row's reference lies above its maximum, in the scores' units (kPromptHead)
  PlanView plan;
  const uint16_t* v;        // for keys with infinities
  long long v_stride;
  uint16_t* out;            // [n_rows][Hq][d]
  bool out32;               // rows of out begin on 32 bytes
  float* lse;               // [n_rows][Hq] or nullptr
  int32_t* dev_status;
};
cudaError_t launch_prompt_attention(int d, const CUtensorMap* tmQ, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                    const PromptAttnParams& p, int grid, cudaStream_t stream);

// ---- K12: key weights -----------------------------------------------------------------------------
constexpr int kWeightKeys = 128;  // keys per tile
struct KeyWeightsParams {
  int Hq, Hkv, G, tc;       // tc: rows of the window per chunk (128 / G)
  int window;
  int per_head;             // CTAs of each head, 0 where shares run over heads
  float scale_log2;
  long long n_rows;
  PlanView plan;
  const float* lse;         // [n_rows][Hq]
  float* weight;            // [Hkv][n_rows]
  int32_t* dev_status;
};
cudaError_t launch_key_weights(int d, const CUtensorMap* tmQ, const CUtensorMap* tmK, const KeyWeightsParams& p, int grid,
                               cudaStream_t stream);

// ---- K13: rows kept for a budget -------------------------------------------------------------------
struct KeepParams {
  int B, Hkv, row_bytes;    // row_bytes: of one head's row
  int budget, first, last;
  long long n_rows, rows_out;
  long long k_stride, v_stride;  // bytes between rows
  const uint8_t* k;
  const uint8_t* v;
  const float* weight;
  const int32_t* row_start;
  uint8_t* k_out;
  uint8_t* v_out;
  int32_t* index;
  int32_t* keep_start;
  int32_t* n_keep;
  int32_t* dev_status;
};
// source: [rows_out][Hkv] numbers of the chosen rows, handed from the choice to the copy.
cudaError_t launch_kv_keep(const KeepParams& p, int32_t* source, int num_sms, cudaStream_t stream);

// Is row_start an ascending walk within [0, n_rows]?  All threads of the block call it; the verdict is the same in all.
__device__ __forceinline__ bool row_start_ok(const int32_t* row_start, int B, long long n_rows) {
  int bad = 0;
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    const int lo = row_start[b], hi = row_start[b + 1];
    bad |= lo < 0 || hi < lo || hi > n_rows;
  }
  return !__syncthreads_or(bad);
}

// The request that row `r` belongs to: the last b in [lo, hi) with row_start[b] <= r.
__device__ __forceinline__ int request_of(const int32_t* row_start, int lo, int hi, long long r) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (row_start[mid] <= r)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

}  // namespace spectree
