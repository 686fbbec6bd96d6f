// K13: the rows of each prompt that a budget leaves in the cache.
//
// Two kernels, the choice and the copying of the chosen rows (ahead of them, for large batches, the counts).
//
// The choice is a radix selection.  Weights become 32-bit keys in their order; three passes of 11, 11 and 10 bits
// count the keys that share what is known of the threshold, and the bin in which the budget runs out is the
// threshold's next piece.  Then a row stays if its key is above the threshold, or equal to it and among the first of
// the equal ones; warps walk disjoint stretches in order, four neighbouring keys to a lane, so a row's place is the
// number of rows that stay before it: sums over the lanes, the warps and the CTAs before.  One cluster works on a
// request and KV head: its CTAs hold the keys in shared memory (one read of the weights; stretches past 40960 keys per
// CTA are read again in each pass), and each adds up a slice of all CTAs' counts through distributed shared memory.  All
// counts are integers: no order of additions changes the result.
//
// The copy reads and writes every kept row once, with 16-byte accesses, four rows of K and V in flight per thread.
//
// What bounds it: the choice by its chain of passes and meetings of the cluster (three of each a pass, some 500 cycles
// apiece), 14 to 19 us whatever the bytes; the copy by memory, at 0.88 of a plain copy's rate.  16 prompts of up to 8192
// rows at a budget of 1024: 37.8 us; one of 131072 rows on 8 heads, a cluster of 8 each: 29.0 us (36.1 with every CTA adding
// up all the bins).

#include "pdl.cuh"
#include "prompt.cuh"
#include "tc_ptx.cuh"
#include "topk.cuh"

namespace spectree {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 40960;        // keys a CTA holds
constexpr int kCopyThreads = 256;
constexpr int kCopies = 4;          // (row, head)s per thread
constexpr int kBatch = 8;           // keys of a thread on their way at once
constexpr int kCountedBatch = 1024; // requests from which the counts have a kernel of their own

// Rows kept before request `upto` and in all (-1 where they are refused), by all threads of the block.
struct Kept {
  long long before, total;
};
__device__ __forceinline__ int rows_kept(const KeepParams& p, int b) {
  const int n = p.row_start[b + 1] - p.row_start[b];
  return n < p.budget ? n : p.budget;
}
__device__ __forceinline__ Kept count_kept(const KeepParams& p, int upto, long long (*s_sum)[2]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool ok = row_start_ok(p.row_start, p.B, p.n_rows);
  long long before = 0, total = 0;
  if (ok)
    for (int b = tid; b < p.B; b += kThreads) {
      const int n = rows_kept(p, b);
      total += n;
      if (b < upto) before += n;
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (lane == 0) {
    s_sum[warp][0] = before;
    s_sum[warp][1] = total;
  }
  __syncthreads();
  Kept k = {0, 0};
  const int warps = p.B < kThreads ? (p.B + 31) / 32 : kWarps;  // those with a request
  for (int w = 0; w < warps; ++w) {
    k.before += s_sum[w][0];
    k.total += s_sum[w][1];
  }
  if (!ok || k.total > p.rows_out) k.before = k.total = -1;
  return k;
}

// The counts of a large batch, once for all (a small one's are worked out by every CTA of the choice).
__global__ void __launch_bounds__(kThreads) keep_counts_kernel(const KeepParams p) {
  __shared__ long long s_sum[kWarps][2];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  // thread t takes requests [t * per, (t + 1) * per): their sums, then a scan over the threads
  const Kept k = count_kept(p, 0, s_sum);
  const bool ok = k.total >= 0;
  if (!ok && tid == 0) set_status(p.dev_status, SPEC_ERR_CAPACITY);
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = tid * per, b1 = b0 + per < p.B ? b0 + per : p.B;
  long long mine = 0;
  if (ok)
    for (int b = b0; b < b1; ++b) mine += rows_kept(p, b);
  const int lane = tid & 31, warp = tid >> 5;
  long long v = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) s_sum[warp][0] = v;
  __syncthreads();
  long long before = v - mine;
  for (int w = 0; w < warp; ++w) before += s_sum[w][0];
  for (int b = b0; b < b1; ++b) {
    const int n = ok ? rows_kept(p, b) : 0;
    p.n_keep[b] = n;
    p.keep_start[b] = ok ? (int)before : 0;
    before += n;
  }
  if (tid == 0) p.keep_start[p.B] = ok ? (int)k.total : 0;
}

__device__ __forceinline__ int cluster_ld(const int* at, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(at, rank)) : "memory");
  return v;
}

__device__ __forceinline__ void cluster_st(int* at, uint32_t rank, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(cluster_addr(at, rank)), "r"(v) : "memory");
}

struct SelectShared {
  int part[4][2048];    // a pass's counts, by warp & 3
  int bins[3][2048];    // their sums, one set per pass (other CTAs read them)
  int warp_sum[kWarps];
  int totals[2];        // keys above and at the threshold
  int warp_n[kWarps][2];
  int bin, left;        // written by the CTA that finds them, in every CTA of the cluster
  int slice[8];         // keys in each CTA's slice of the bins
  long long sum[kWarps][2];
};

static_assert(sizeof(SelectShared) % 16 == 0, "the keys behind it are read four at a time");

__global__ void __launch_bounds__(kThreads, 1) keep_select_kernel(const KeepParams p, int32_t* source, int cluster, int counted) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  SelectShared& s = *reinterpret_cast<SelectShared*>(s_raw);
  uint32_t* s_key = reinterpret_cast<uint32_t*>(s_raw + sizeof(SelectShared));  // [kHeld]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster > 1 ? (int)cluster_rank() : 0;
  const int seg = blockIdx.x / cluster;
  const int b = seg / p.Hkv, g = seg % p.Hkv;
  pdl_wait();
  pdl_launch_dependents();
  int keep;
  long long out0;
  if (counted) {
    keep = p.n_keep[b];
    out0 = p.keep_start[b];
  } else {
    const Kept k = count_kept(p, b, s.sum);
    keep = k.total < 0 ? 0 : rows_kept(p, b);
    out0 = k.total < 0 ? 0 : k.before;
    if (rank == 0 && g == 0 && tid == 0) {
      p.n_keep[b] = keep;
      p.keep_start[b] = (int)out0;
      if (b == 0) {
        p.keep_start[p.B] = k.total < 0 ? 0 : (int)k.total;
        if (k.total < 0) set_status(p.dev_status, SPEC_ERR_CAPACITY);
      }
    }
  }
  if (keep == 0) return;  // (the whole cluster)
  const int r0 = p.row_start[b], n = p.row_start[b + 1] - r0;
  auto put = [&](int place, int j) {
    const long long at = (out0 + place) * p.Hkv + g;
    p.index[at] = j;
    source[at] = r0 + j;
  };
  if (n <= p.budget) {
    for (long long j = (long long)rank * kThreads + tid; j < n; j += (long long)cluster * kThreads) put((int)j, (int)j);
    return;
  }
  if (rank == 0) {
    for (int j = tid; j < p.first; j += kThreads) put(j, j);
    for (int j = tid; j < p.last; j += kThreads) put(p.budget - p.last + j, n - p.last + j);
  }
  int left = p.budget - p.first - p.last;  // rows to choose
  if (left == 0) return;
  // candidates [first, n - last); this CTA's are [c0, c1)
  const int cands = n - p.first - p.last;
  const int per = (int)(((long long)cands + cluster - 1) / cluster);
  const long long lo = (long long)rank * per, hi = lo + per < cands ? lo + per : cands;
  const int mine = hi > lo ? (int)(hi - lo) : 0;
  const float* weight = p.weight + (size_t)g * p.n_rows + r0 + p.first + (mine ? lo : 0);
  auto key_at = [&](int i) { return i < kHeld ? s_key[i] : order_u(weight[i]); };
  uint32_t known = 0;  // the threshold's upper bits
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < 4 * 2048; i += kThreads) (&s.part[0][0])[i] = 0;
    __syncthreads();
    int* part = s.part[warp & 3];
    for (int i0 = tid; i0 < mine; i0 += kThreads * kBatch) {
      uint32_t key[kBatch];  // (all reads first)
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int i = i0 + e * kThreads;
        key[e] = i < mine ? (pass == 0 ? __float_as_uint(weight[i]) : key_at(i)) : 0u;
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int i = i0 + e * kThreads;
        if (i >= mine) break;
        if (pass == 0) {
          key[e] = order_u(__uint_as_float(key[e]));
          if (i < kHeld) s_key[i] = key[e];
        }
        if (pass == 0 || (key[e] >> (shift + bits)) == known) atomicAdd(&part[(key[e] >> shift) & ((1u << bits) - 1)], 1);
      }
    }
    __syncthreads();
    for (int i = tid; i < 2048; i += kThreads) s.bins[pass][i] = s.part[0][i] + s.part[1][i] + s.part[2][i] + s.part[3][i];
    if (cluster > 1)
      cluster_sync_all();
    else
      __syncthreads();
    // The bin, from above, in which the rows to choose run out.  Each CTA sums a slice of the bins over the cluster (all of
    // them in every CTA took 8000 cycles a pass), rank 0 the uppermost; a thread looks at two neighbouring bins of it.
    const int slice = 2048 / cluster, top_bin = 2047 - rank * slice - 2 * tid;
    const bool mine_bins = 2 * tid < slice;
    int x[2] = {0, 0};
    if (mine_bins) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (cluster > 1) {
#pragma unroll 8
          for (int r = 0; r < cluster; ++r) x[e] += cluster_ld(&s.bins[pass][top_bin - e], (uint32_t)r);
        } else {
          x[e] = s.bins[pass][top_bin - e];
        }
      }
    }
    int v = x[0] + x[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) s.warp_sum[warp] = v;
    __syncthreads();
    int above = v - x[0] - x[1];
    {  // every warp scans the warps' sums for itself
      int y = s.warp_sum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      const int before = __shfl_sync(0xffffffffu, y, (warp + 31) & 31), all = __shfl_sync(0xffffffffu, y, 31);
      if (warp > 0) above += before;
      if (cluster > 1) {
        if (tid < cluster) cluster_st(&s.slice[rank], (uint32_t)tid, all);
        cluster_sync_all();
        for (int r = 0; r < rank; ++r) above += s.slice[r];
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (mine_bins && above < left && above + x[e] >= left) {
        for (int r = 0; r < cluster; ++r) {
          if (cluster > 1) {
            cluster_st(&s.bin, (uint32_t)r, top_bin - e);
            cluster_st(&s.left, (uint32_t)r, left - above);
          } else {
            s.bin = top_bin - e;
            s.left = left - above;
          }
        }
      }
      above += x[e];
    }
    if (cluster > 1)
      cluster_sync_all();
    else
      __syncthreads();
    known = (known << bits) | (uint32_t)s.bin;
    left = s.left;
    __syncthreads();
  }
  // `known` is the threshold, `left` the number of keys equal to it that stay.  Warps walk stretches, four neighbouring keys
  // per lane; keys above and at the threshold are counted in the halves of a word (128 a step) and summed apart.
  const int stretch = ((mine + kWarps - 1) / kWarps + 127) & ~127;
  const int w0 = warp * stretch < mine ? warp * stretch : mine, w1 = w0 + stretch < mine ? w0 + stretch : mine;
  auto four = [&](int i, uint32_t (&key)[4]) {
    if (i + 4 <= w1 && i + 4 <= kHeld) {
      const uint4 k = *reinterpret_cast<const uint4*>(s_key + i);
      key[0] = k.x, key[1] = k.y, key[2] = k.z, key[3] = k.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) key[e] = i + e < w1 ? key_at(i + e) : 0u;
    }
  };
  // (known == 0: NaN alone are at the threshold, and places behind the stretch are not keys)
  auto count = [&](int i, const uint32_t (&key)[4]) {
    uint32_t n = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < w1) n += key[e] > known ? 1u : (key[e] == known ? 0x10000u : 0u);
    return n;
  };
  int above = 0, equal = 0;
  for (int i = w0 + lane * 4; i < w1; i += 128) {
    uint32_t key[4];
    four(i, key);
    const uint32_t n = count(i, key);
    above += n & 0xffffu;
    equal += n >> 16;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    above += __shfl_xor_sync(0xffffffffu, above, o);
    equal += __shfl_xor_sync(0xffffffffu, equal, o);
  }
  if (lane == 0) {
    s.warp_n[warp][0] = above;
    s.warp_n[warp][1] = equal;
  }
  __syncthreads();
  {  // sums over the warps before this one, and over the CTAs before
    int n[2] = {s.warp_n[lane][0], s.warp_n[lane][1]};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      int y = n[e];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      const int all = __shfl_sync(0xffffffffu, y, 31);
      if (tid == 0) s.totals[e] = all;
      const int before = __shfl_sync(0xffffffffu, y - n[e], warp);
      (e ? equal : above) = before;
    }
  }
  if (cluster > 1) {
    cluster_sync_all();
    for (int r = 0; r < rank; ++r) {
      above += cluster_ld(&s.totals[0], (uint32_t)r);
      equal += cluster_ld(&s.totals[1], (uint32_t)r);
    }
  }
  for (int i0 = w0; i0 < w1; i0 += 128) {
    const int i = i0 + lane * 4;
    uint32_t key[4];
    four(i, key);
    const uint32_t n = count(i, key);
    uint32_t sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t z = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += z;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, sum, 31);
    int up = above + (int)((sum - n) & 0xffffu), eq = equal + (int)((sum - n) >> 16);
    if (n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (i + e >= w1) break;
        const bool is_up = key[e] > known, is_eq = key[e] == known;
        if (is_up || (is_eq && eq < left)) put(p.first + up + (eq < left ? eq : left), p.first + (int)lo + i + e);
        up += is_up;
        eq += is_eq;
      }
    }
    above += all & 0xffffu;
    equal += all >> 16;
  }
  if (cluster > 1) cluster_sync_all();  // no CTA leaves while another may still read its counts
}

// Copies K and V of every kept (row, head): `vecs` lanes of 16 bytes per row.
__global__ void __launch_bounds__(kCopyThreads) keep_copy_kernel(const KeepParams p, const int32_t* source, int vecs) {
  pdl_wait();
  const long long units = (long long)p.keep_start[p.B] * p.Hkv;
  const int per_block = kCopyThreads / vecs;  // units side by side
  const int lane = threadIdx.x % vecs, at = threadIdx.x / vecs;
  const long long u0 = (long long)blockIdx.x * per_block * kCopies + at;
  uint4 kv[kCopies][2];
#pragma unroll
  for (int f = 0; f < kCopies; ++f) {
    const long long u = u0 + (long long)f * per_block;
    if (u < units) {
      const long long row = source[u];
      const int g = (int)(u % p.Hkv);
      kv[f][0] = *reinterpret_cast<const uint4*>(p.k + row * p.k_stride + (size_t)g * p.row_bytes + lane * 16);
      kv[f][1] = *reinterpret_cast<const uint4*>(p.v + row * p.v_stride + (size_t)g * p.row_bytes + lane * 16);
    }
  }
#pragma unroll
  for (int f = 0; f < kCopies; ++f) {
    const long long u = u0 + (long long)f * per_block;
    if (u < units) {
      *reinterpret_cast<uint4*>(p.k_out + (size_t)u * p.row_bytes + lane * 16) = kv[f][0];
      *reinterpret_cast<uint4*>(p.v_out + (size_t)u * p.row_bytes + lane * 16) = kv[f][1];
    }
  }
}

}  // namespace

cudaError_t launch_kv_keep(const KeepParams& p, int32_t* source, int num_sms, cudaStream_t stream) {
  // Each CTA of the choice reads the whole of row_start: 1 us up to a request per thread, against 4 us for a kernel ahead.
  const bool copies = p.n_rows > 0 && p.rows_out > 0;
  const int counted = p.B > kCountedBatch || !copies;
  cudaError_t err = cudaSuccess;
  if (counted) err = launch_dependent(keep_counts_kernel, dim3(1), dim3(kThreads), 0, stream, p);
  if (err != cudaSuccess || !copies) return err;
  // CTAs per request and head: as many as there are SMs for, and 2048 rows for each.
  const long long segs = (long long)p.B * p.Hkv;
  int cluster = 1;
  while (cluster < 8 && segs * cluster * 2 <= num_sms && (long long)cluster * 2 * 2048 <= p.n_rows) cluster *= 2;
  err = cudaFuncSetAttribute(keep_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(SelectShared) + kHeld * 4);
  if (err != cudaSuccess) return err;
  const long long longest = p.n_rows < kHeld ? p.n_rows : kHeld;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(segs * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(SelectShared) + (size_t)longest * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, keep_select_kernel, p, source, cluster, counted);
  if (err != cudaSuccess) return err;
  const int vecs = p.row_bytes / 16;
  const long long per_block = (long long)(kCopyThreads / vecs) * kCopies;
  const long long most = p.rows_out < p.n_rows ? p.rows_out : p.n_rows;  // a request keeps no more rows than it has
  const long long blocks = (most * p.Hkv + per_block - 1) / per_block;
  return launch_dependent(keep_copy_kernel, dim3((unsigned)blocks), dim3(kCopyThreads), 0, stream, p, source, vecs);
}

}  // namespace spectree
