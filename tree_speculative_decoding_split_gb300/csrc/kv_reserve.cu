// K7: block tables and slot maps from request lengths, on the device (spec_kv_reserve).
//
// want_b = ceil((len_b + new_b) / bs).  With exclusive prefix sums over the requests of what each gives
// back (held - want), takes (want - held) and adds (new), every released entry, taken block and new row
// has its place by arithmetic alone, so the order is fixed and nothing is counted by atomics:
//   r-th given back  -> list[f + R - 1 - r];   a-th taken <- list[f + R - 1 - a]   (f = free, R given back)
// A taken block may be one given back by another request in the same call, so the two steps are
// separated by a barrier.
//
// Bound: latency.  The tables' changes are a few KB; what takes time is the chain of counts, scan, list, tables and
// slots.  So small calls are one CTA that writes the slot map as well, and the sums of all three kinds are scanned
// together (apart, the two calls below took 12.8, 16.9 and 31.2 us).  Measured with a cold cache, a call with its slot map
// and one without: 10.7 us for one request, 14.8 for 32, 26.4 for 512 prompts with 1 M slots.
#include "common.cuh"
#include "kernels.cuh"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace spectree {

namespace {

constexpr int kRowsPerThread = 8;  // slot-map entries one thread of the map kernel writes: a 64-byte run

// The last b with start[b] <= x (start is non-decreasing, start[0] <= x < start[n]).
__device__ __forceinline__ int owner_of(const int* start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// What a thread's requests give back, take and add.
struct Sums {
  int rel, need;
  long long rows;
};
// Inclusive scan of one record per thread over the block; `total` gets the sum.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* s_warp, Sums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int r = __shfl_up_sync(0xffffffffu, v.rel, o), t = __shfl_up_sync(0xffffffffu, v.need, o);
    const long long a = __shfl_up_sync(0xffffffffu, v.rows, o);
    if (lane >= o) {
      v.rel += r;
      v.need += t;
      v.rows += a;
    }
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  // every warp scans the warps' sums (32 at most)
  Sums w = lane < nw ? s_warp[lane] : Sums{0, 0, 0};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int r = __shfl_up_sync(0xffffffffu, w.rel, o), t = __shfl_up_sync(0xffffffffu, w.need, o);
    const long long a = __shfl_up_sync(0xffffffffu, w.rows, o);
    if (lane >= o) {
      w.rel += r;
      w.need += t;
      w.rows += a;
    }
  }
  const int prev = max(warp - 1, 0);
  const Sums before{__shfl_sync(0xffffffffu, w.rel, prev), __shfl_sync(0xffffffffu, w.need, prev),
                    __shfl_sync(0xffffffffu, w.rows, prev)};
  *total = Sums{__shfl_sync(0xffffffffu, w.rel, 31), __shfl_sync(0xffffffffu, w.need, 31),
                __shfl_sync(0xffffffffu, w.rows, 31)};
  if (warp > 0) {
    v.rel += before.rel;
    v.need += before.need;
    v.rows += before.rows;
  }
  return v;
}

// The pool row of slot `pos` of request b, or -1 (an unserved request's, or one behind its table).
__device__ __forceinline__ long long slot_of(const ReserveParams& p, int b, long long pos, bool* bad) {
  const int blk = p.table[(size_t)b * p.max_blocks + (pos >> p.bs_shift)];
  if (blk < 0 || blk >= p.num_blocks) {
    *bad = true;
    return -1;
  }
  return ((long long)blk << p.bs_shift) + (pos & (p.bs - 1));
}
__device__ __forceinline__ bool served(const ReserveParams& p, int b, int len, int add) {
  const int nb = p.n_blocks[b];
  return len >= 0 && add >= 0 && nb >= 0 && nb <= p.max_blocks && (long long)len + add <= ((long long)nb << p.bs_shift);
}

}  // namespace

// One cluster (of one CTA for small calls): every CTA scans the requests, all share the entries.
// With `map` (single CTA only) the slot map is written here as well.
__global__ void __launch_bounds__(1024) kv_reserve_kernel(const ReserveParams p, int map) {
  extern __shared__ int s_plan[];
  __shared__ Sums s_warp[32];
  const int B = p.B, T = blockDim.x, tid = threadIdx.x;
  int* s_base = s_plan;             // min(held, want): where what is given back or taken begins; -1 = refused
  int* s_rel = s_base + B;          // [B + 1] blocks given back before b
  int* s_need = s_rel + B + 1;      // [B + 1] blocks taken before b
  int* s_row = s_need + B + 1;      // [B + 1] new rows before b
  pdl_wait();  // what comes before in the stream may still be ending: nothing of it is read ahead of this
  pdl_launch_dependents();  // the slot map's kernel may be launched
  const int f = *p.free_count;
  // ---- scan ----
  const int per = (B + T - 1) / T;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  int refused = 0;
  Sums mine{0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const int len = p.seq_len[b], add = p.n_new[b], held = p.n_blocks[b];
    const long long want = ((long long)len + add + p.bs - 1) >> p.bs_shift;
    const bool ok = len >= 0 && add >= 0 && want <= p.max_blocks && held >= 0 && held <= p.max_blocks;
    refused |= !ok;
    s_base[b] = ok ? min(held, (int)want) : -1;
    const int r = ok ? max(held - (int)want, 0) : 0, t = ok ? max((int)want - held, 0) : 0;
    s_rel[b] = r;
    s_need[b] = t;
    s_row[b] = max(add, 0);
    mine.rel += r;
    mine.need += t;
    mine.rows += max(add, 0);
  }
  Sums all;
  const Sums incl = block_scan(mine, s_warp, &all);
  int rel0 = incl.rel - mine.rel, need0 = incl.need - mine.need;
  long long row0 = incl.rows - mine.rows;
  const int R = all.rel, A = all.need;
  const long long total = all.rows;
  const long long row_cap = p.slot_map ? p.slot_cap : 0x7fffffffLL;
  const bool fatal = f < 0 || f > p.num_blocks || (long long)f + R > p.num_blocks || total > row_cap;
  for (int b = b0; b < b1; ++b) {
    const int r = s_rel[b], t = s_need[b], a = s_row[b];
    s_rel[b] = rel0;
    s_need[b] = need0;
    s_row[b] = fatal ? 0 : (int)row0;
    rel0 += r;
    need0 += t;
    row0 += a;
  }
  if (tid == 0) {
    s_rel[B] = R;
    s_need[B] = A;
    s_row[B] = fatal ? 0 : (int)total;
  }
  const int top = f + R;
  const uint32_t rank = map ? 0 : cluster_rank();
  const int ncta = gridDim.x, gt = (int)rank * T + tid, gn = ncta * T;
  if (__syncthreads_or(refused) || fatal || A > top) {
    if (gt == 0) set_status(p.dev_status, SPEC_ERR_CAPACITY);
  }
  if (!fatal) {
    // ---- give back ----
    for (int r = gt; r < R; r += gn) {
      const int b = owner_of(s_rel, B, r);
      int32_t* e = p.table + (size_t)b * p.max_blocks + s_base[b] + (r - s_rel[b]);
      p.free_list[top - 1 - r] = *e;
      *e = -1;
    }
  }
  // every CTA has read the counts, and what was given back is on the list
  if (ncta > 1) cluster_sync_all(); else __syncthreads();
  if (!fatal) {
    // ---- take; requests are served while the running sum of what they want is within the stack ----
    for (int a = gt; a < min(A, top); a += gn) {
      const int b = owner_of(s_need, B, a);
      if (s_need[b + 1] <= top)
        p.table[(size_t)b * p.max_blocks + s_base[b] + (a - s_need[b])] = p.free_list[top - 1 - a];
    }
    for (int b = gt; b < B; b += gn) {
      const int t = s_need[b + 1] - s_need[b];
      if (s_base[b] >= 0 && (t == 0 || s_need[b + 1] <= top)) p.n_blocks[b] = s_base[b] + t;
    }
    // what is taken: the largest of the running sums within the stack
    if (gt == 0) *p.free_count = top - s_need[owner_of(s_need, B + 1, top)];
  }
  if (p.row_start)
    for (int b = gt; b <= B; b += gn) p.row_start[b] = s_row[b];
  if (!map || !p.slot_map) return;
  __syncthreads();
  // ---- slot map ----
  bool bad = false;
  const int n = s_row[B];
  for (long long i = tid; i < p.slot_cap; i += T) {
    long long slot = -1;
    if (i < n) {
      const int b = owner_of(s_row, B, (int)i);
      const int len = p.seq_len[b];
      if (served(p, b, len, s_row[b + 1] - s_row[b])) slot = slot_of(p, b, (long long)len + (int)i - s_row[b], &bad);
    }
    p.slot_map[i] = slot;
  }
  if (bad) set_status(p.dev_status, SPEC_ERR_CAPACITY);
}

// The slot map of a large call: every thread finds the request of its run of rows once and follows it.
__global__ void __launch_bounds__(256) kv_slot_map_kernel(const ReserveParams p) {
  extern __shared__ int s_row[];
  pdl_wait();
  for (int b = threadIdx.x; b <= p.B; b += blockDim.x) s_row[b] = p.row_start[b];
  __syncthreads();
  const int n = s_row[p.B];
  bool bad = false;
  const long long step = (long long)gridDim.x * blockDim.x * kRowsPerThread;
  for (long long i0 = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * kRowsPerThread; i0 < p.slot_cap; i0 += step) {
    long long slot[kRowsPerThread];
    int b = i0 < n ? owner_of(s_row, p.B, (int)i0) : 0, len = 0;
    bool ok = false, fresh = true;
#pragma unroll
    for (int j = 0; j < kRowsPerThread; ++j) {
      const long long i = i0 + j;
      slot[j] = -1;
      if (i >= n) continue;
      while (i >= s_row[b + 1]) {  // requests without rows are passed over
        ++b;
        fresh = true;
      }
      if (fresh) {
        len = p.seq_len[b];
        ok = served(p, b, len, s_row[b + 1] - s_row[b]);
        fresh = false;
      }
      if (ok) slot[j] = slot_of(p, b, (long long)len + (int)i - s_row[b], &bad);
    }
    if (i0 + kRowsPerThread <= p.slot_cap) {  // slot_map is 16-byte aligned
#pragma unroll
      for (int j = 0; j < kRowsPerThread; j += 2)
        *reinterpret_cast<longlong2*>(p.slot_map + i0 + j) = make_longlong2(slot[j], slot[j + 1]);
    } else {
      for (int j = 0; j < kRowsPerThread; ++j)
        if (i0 + j < p.slot_cap) p.slot_map[i0 + j] = slot[j];
    }
  }
  if (bad) set_status(p.dev_status, SPEC_ERR_CAPACITY);
}

cudaError_t launch_kv_reserve(const ReserveParams& p, int num_sms, cudaStream_t stream) {
  const size_t plan = (size_t)(4 * p.B + 3) * sizeof(int), rows = (size_t)(p.B + 1) * sizeof(int);
  // (512 threads: 32 requests, two calls, 14.8 us with a cold cache; 256 threads 16.9, 128 21.0)
  const bool small = p.B <= 64 && p.slot_cap <= 16384;
  cudaError_t err = cudaFuncSetAttribute(kv_reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (4 * SPEC_MAX_RESERVE_BATCH + 3) * (int)sizeof(int));
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(small ? 1 : 8);
  cfg.blockDim = dim3(small ? 512 : 1024);
  cfg.dynamicSmemBytes = plan;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = small ? 1 : 8;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, kv_reserve_kernel, p, small ? 1 : 0);
  if (err != cudaSuccess || small || !p.slot_map || p.slot_cap == 0) return err;
  const long long want = (p.slot_cap + 256 * kRowsPerThread - 1) / (256 * kRowsPerThread);
  const unsigned grid = (unsigned)(want < (long long)num_sms * 8 ? want : (long long)num_sms * 8);
  return launch_dependent(kv_slot_map_kernel, dim3(grid), dim3(256), rows, stream, p);
}

}  // namespace spectree
