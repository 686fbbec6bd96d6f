// The plan of a call over packed prompt rows: every request cut into pieces, listed for the persistent CTAs of
// the kernel behind.
//
// Lengths are on the device only, so the list is made there, by one CTA: row_start is checked, the pieces of each
// request are counted and summed, and each piece finds its request by a search over the sums.  For causal
// attention pieces are listed by falling work (a counting sort over the number of key tiles before a piece's
// end): CTAs take them from the front, so the longest never start last.  (Which of two pieces of equal work
// comes first is left to the atomics; no result depends on it.)  It takes 3 to 4 us, most of it a launch and three
// reads of row_start behind one another; calls of a single request, and key weights of few, do without (PlanReader).

#include "pdl.cuh"
#include "prompt.cuh"

namespace spectree {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 2048;
constexpr int kPlanMaxBatch = SPEC_MAX_RESERVE_BATCH;

// Exclusive prefix sum over the block's threads; *total gets the sum.
__device__ __forceinline__ long long block_scan(long long x, long long* s_warp, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  const long long before = (warp ? s_warp[warp - 1] : 0) + v - x;
  *total = s_warp[31];
  __syncthreads();
  return before;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  __shared__ int s_first[kPlanMaxBatch];  // items before each request (their sum stays below 2^31)
  __shared__ int s_bin[kPlanBins];
  __shared__ long long s_warp[32];
  __shared__ int s_most;
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0) s_most = 0;
  if (!row_start_ok(p.row_start, p.B, p.n_rows)) {
    if (tid == 0) {
      set_status(p.dev_status, SPEC_ERR_CAPACITY);
      p.count[0] = 0;
    }
    return;
  }
  // thread t takes requests [t * per, (t + 1) * per)
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = tid * per, b1 = b0 + per < p.B ? b0 + per : p.B;
  long long mine = 0;
  int most = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = p.row_start[b + 1] - p.row_start[b];
    mine += (n + p.step - 1) / p.step;
    most = n > most ? n : most;
  }
  long long total;
  long long at = block_scan(mine, s_warp, &total);
  for (int b = b0; b < b1; ++b) {
    s_first[b] = (int)at;
    at += (p.row_start[b + 1] - p.row_start[b] + p.step - 1) / p.step;
  }
  if (p.by_work) {
    atomicMax(&s_most, (most + 127) >> 7);
    for (int i = tid; i < kPlanBins; i += kPlanThreads) s_bin[i] = 0;
  }
  __syncthreads();
  int shift = 0;
  while ((s_most >> shift) >= kPlanBins) ++shift;
  const int items = (int)total;
  auto item = [&](int i) {
    int lo = 0, hi = p.B;  // the last request with s_first <= i (those without items share their follower's)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_first[mid] <= i)
        lo = mid;
      else
        hi = mid;
    }
    PromptItem it;
    it.r0 = p.row_start[lo];
    it.n = p.row_start[lo + 1] - it.r0;
    it.tok = (i - s_first[lo]) * p.step;
    it.pad = 0;
    return it;
  };
  auto bin_of = [&](const PromptItem& it) {  // falling with the key tiles before the item's end
    const long long end = (long long)it.tok + p.step < it.n ? it.tok + p.step : it.n;
    return kPlanBins - 1 - (int)(((end + 127) >> 7) >> shift);
  };
  if (!p.by_work) {
    for (int i = tid; i < items; i += kPlanThreads) p.items[i] = item(i);
  } else {
    for (int i = tid; i < items; i += kPlanThreads) atomicAdd(&s_bin[bin_of(item(i))], 1);
    __syncthreads();
    const int x0 = s_bin[2 * tid], x1 = s_bin[2 * tid + 1];
    long long sum;
    const int before = (int)block_scan((long long)x0 + x1, s_warp, &sum);
    s_bin[2 * tid] = before;
    s_bin[2 * tid + 1] = before + x0;
    __syncthreads();
    for (int i = tid; i < items; i += kPlanThreads) {
      const PromptItem it = item(i);
      p.items[atomicAdd(&s_bin[bin_of(it)], 1)] = it;
    }
  }
  if (tid == 0) p.count[0] = items;
}
static_assert(kPlanBins == 2 * kPlanThreads, "two bins per thread");

}  // namespace

cudaError_t launch_prompt_plan(const PlanParams& p, cudaStream_t stream) {
  return launch_dependent(plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
}

}  // namespace spectree
