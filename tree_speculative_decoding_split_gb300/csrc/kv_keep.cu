// K13: the rows of each prompt that a budget leaves in the cache.
//
// Two kernels, the choice and the copying of the chosen rows (ahead of them, for large batches, the counts).
//
// The choice is a radix selection.  Weights become 32-bit keys in their order; three passes of 11, 11 and 10 bits
// count the keys that share what is known of the threshold, and the bin in which the budget runs out is the
// threshold's next piece.  Then a row stays if its key is above the threshold, or equal to it and among the first of
// the equal ones; threads have neighbouring keys, so a row's place is the number of rows that stay before it: sums
// over the threads, the warps and the CTAs before.  One cluster works on a request and KV head: its CTAs hold the keys in
// shared memory (one read of the weights; stretches past 40960 keys per CTA are read again in each pass), tell one another
// how many counts lie in each slice of the bins, and the one whose slice has the threshold adds it up through
// distributed shared memory.  All counts are integers: no order of additions changes the result.
//
// The copy reads and writes every kept row once, 16 bytes of K and of V per thread; what it reads makes way in the L2 for
// what it writes, which the cache's append reads next (16 prompts 32.2 us without; two rows a thread 32.8, four 34.8).
//
// What bounds it: the choice by its chain of passes and meetings of the cluster (two a pass), 10 to 14 us whatever the
// bytes; the copy by memory.  16 prompts of up to 8192 rows at a budget of 1024: 29.1 us; one of 131072 rows on 8 heads, a
// cluster of 8 each: 22.6 us (with an earlier copy, 36.1 with every CTA adding up all the bins, 29.0 with every CTA adding up
// a slice, a third meeting and the last walk in steps of 128 keys a warp, 22.9 as it is).  These are graph replays over the
// same outputs; Python calls, which make new ones, take 33.6 and 24.0.  512 prompts of 200 rows at a budget of 64 take 233 us
// where their bytes take 40: a CTA of the choice per request and head, one to an SM, cleared and walked for 200 keys.

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

// Request b as a CTA of the choice needs it: rows kept of it, before it and in all (-1 where they are refused).
struct Request {
  int keep, before, total, r0, n;
};
// Up to 32 requests, by every warp for itself, with one read and no meeting of the block (1 us less than count_kept).  Rows
// kept are rows there are: sums stay below 2^31.
__device__ __forceinline__ Request request_in_warp(const KeepParams& p, int b) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = 0;
  if (lane < p.B) {
    lo = p.row_start[lane];
    hi = p.row_start[lane + 1];
  }
  const bool ok = !__any_sync(0xffffffffu, lo < 0 || hi < lo || hi > p.n_rows);
  const int kept = !ok ? 0 : (hi - lo < p.budget ? hi - lo : p.budget);
  Request r;
  r.total = __reduce_add_sync(0xffffffffu, kept);
  r.before = __reduce_add_sync(0xffffffffu, lane < b ? kept : 0);
  r.keep = __shfl_sync(0xffffffffu, kept, b);
  r.r0 = __shfl_sync(0xffffffffu, lo, b);
  r.n = __shfl_sync(0xffffffffu, hi, b) - r.r0;
  if (!ok || r.total > p.rows_out) r.total = -1;
  return r;
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

struct alignas(16) SelectShared {
  int part[4][2048];    // the first pass's counts, by warp & 3
  int bins[3][2048];    // each pass's counts (other CTAs read them)
  int warp_sum[kWarps];
  int warp_n[kWarps][2];
  int bin, left;        // written by the CTA that finds them, in every CTA of the cluster
  int slice[8][8];      // [CTA][slice of the bins] its counts there, in every CTA
  int totals[8][2];     // [CTA] its keys above and at the threshold, in every CTA
  long long sum[kWarps][2];
};

__global__ void __launch_bounds__(kThreads, 1)
    keep_select_kernel(const KeepParams p, int32_t* source, int log_cluster, int counted) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  SelectShared& s = *reinterpret_cast<SelectShared*>(s_raw);
  uint32_t* s_key = reinterpret_cast<uint32_t*>(s_raw + sizeof(SelectShared));  // [kHeld]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cluster = 1 << log_cluster, rank = cluster > 1 ? (int)cluster_rank() : 0;
  const int seg = (int)(blockIdx.x >> log_cluster);
  const int b = seg / p.Hkv, g = seg % p.Hkv;
  pdl_wait();
  pdl_launch_dependents();
  Request r;
  if (counted) {
    r.keep = p.n_keep[b];
    r.before = p.keep_start[b];
  } else {
    if (p.B <= 32) {
      r = request_in_warp(p, b);
    } else {
      const Kept k = count_kept(p, b, s.sum);
      r.total = (int)k.total;
      r.before = (int)k.before;
      r.keep = r.total < 0 ? 0 : rows_kept(p, b);
    }
    if (r.total < 0) r.keep = r.before = 0;
    if (rank == 0 && g == 0 && tid == 0) {
      p.n_keep[b] = r.keep;
      p.keep_start[b] = r.before;
      if (b == 0) {
        p.keep_start[p.B] = r.total < 0 ? 0 : r.total;
        if (r.total < 0) set_status(p.dev_status, SPEC_ERR_CAPACITY);
      }
    }
  }
  if (r.keep == 0) return;  // (the whole cluster)
  if (counted || p.B > 32) {
    r.r0 = p.row_start[b];
    r.n = p.row_start[b + 1] - r.r0;
  }
  const int r0 = r.r0, n = r.n;
  const long long out0 = r.before;
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
  __syncwarp();
  if (cluster > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // (it runs: others may write to it)
  // candidates [first, n - last); this CTA's are [c0, c1)
  const int cands = n - p.first - p.last;
  const int per = (int)(((long long)cands + cluster - 1) >> log_cluster);
  const long long lo = (long long)rank * per, hi = lo + per < cands ? lo + per : cands;
  const int mine = hi > lo ? (int)(hi - lo) : 0;
  const float* weight = p.weight + (size_t)g * p.n_rows + r0 + p.first + (mine ? lo : 0);
  const int held = mine < kHeld ? mine : kHeld;
  for (int i = tid; i < 4 * 2048; i += kThreads) (&s.part[0][0])[i] = 0;
  for (int i = tid; i < 2 * 2048; i += kThreads) s.bins[1][i] = 0;  // (and the last)
  uint32_t known = 0;  // the threshold's upper bits
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bits = pass == 2 ? 10 : 11;
    const uint32_t mask = (1u << bits) - 1;
    if (pass == 0) {
      __syncthreads();
      int* part = s.part[warp & 3];
      for (int i0 = tid; i0 < mine; i0 += kThreads * kBatch) {
        float w[kBatch];  // (all reads first)
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const int i = i0 + e * kThreads;
          w[e] = i < mine ? weight[i] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const int i = i0 + e * kThreads;
          if (i >= mine) break;
          const uint32_t key = order_u(w[e]);
          if (i < kHeld) s_key[i] = key;
          atomicAdd(&part[key >> 21], 1);
        }
      }
    } else {
      // few keys share what is known: one set of counts, keys read four at a time
      int* bins = s.bins[pass];
      auto add = [&](uint32_t key) {
        if (key >> (shift + bits) == known) atomicAdd(&bins[(key >> shift) & mask], 1);
      };
      for (int i = tid * 4; i < held; i += kThreads * 4) {
        if (i + 4 <= held) {
          const uint4 k = *reinterpret_cast<const uint4*>(s_key + i);
          add(k.x), add(k.y), add(k.z), add(k.w);
        } else {
          for (int e = i; e < held; ++e) add(s_key[e]);
        }
      }
      for (int i0 = kHeld + tid; i0 < mine; i0 += kThreads * kBatch) {
        float w[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) w[e] = i0 + e * kThreads < mine ? weight[i0 + e * kThreads] : 0.f;
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
          if (i0 + e * kThreads < mine) add(order_u(w[e]));
      }
    }
    __syncthreads();
    // The bin, from above, in which the rows to choose run out.  A thread has two neighbouring bins, in falling order.
    int top_bin = 2047 - 2 * tid, above = 0;
    int x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = top_bin - e;
      if (pass == 0) s.bins[0][i] = s.part[0][i] + s.part[1][i] + s.part[2][i] + s.part[3][i];
      x[e] = s.bins[pass][i];
    }
    bool finds = true;
    if (cluster > 1) {
      // Every CTA tells all others what it has in each of `cluster` slices of the bins.  So each knows of its own slice (rank
      // 0 has the uppermost) whether the rows run out there, and that one alone adds up the bins of it over the cluster (all
      // bins in every CTA took 8000 cycles a pass, a slice in every CTA and a third meeting 5200 where this takes 3500).
      const int sum = __reduce_add_sync(0xffffffffu, x[0] + x[1]);
      if (lane == 0) s.warp_sum[warp] = sum;
      __syncthreads();
      if (pass == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      if (tid < cluster * cluster) {
        const int to = tid >> log_cluster, slice = tid & (cluster - 1), warps = kWarps >> log_cluster;
        int n_slice = 0;
        for (int w = 0; w < warps; ++w) n_slice += s.warp_sum[slice * warps + w];
        cluster_st(&s.slice[rank][slice], (uint32_t)to, n_slice);
      }
      cluster_sync_all();
      int before = 0, inside = 0;
      for (int i = lane; i < cluster * cluster; i += 32) {
        const int slice = i & (cluster - 1), v = s.slice[i >> log_cluster][slice];
        if (slice < rank) before += v;
        if (slice == rank) inside += v;
      }
      above = __reduce_add_sync(0xffffffffu, before);
      inside = __reduce_add_sync(0xffffffffu, inside);
      finds = above < left && above + inside >= left;
      const int slice = 2048 >> log_cluster;
      top_bin -= rank * slice;
      x[0] = x[1] = 0;
      if (finds && 2 * tid < slice) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll 8
          for (int c = 0; c < cluster; ++c) x[e] += cluster_ld(&s.bins[pass][top_bin - e], (uint32_t)c);
      }
    }
    if (finds) {  // (the whole block)
      int v = x[0] + x[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      if (lane == 31) s.warp_sum[warp] = v;
      __syncthreads();
      above += v - x[0] - x[1] + __reduce_add_sync(0xffffffffu, lane < warp ? s.warp_sum[lane] : 0);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (above < left && above + x[e] >= left) {
          for (int c = 0; c < cluster; ++c) {
            if (cluster > 1) {
              cluster_st(&s.bin, (uint32_t)c, top_bin - e);
              cluster_st(&s.left, (uint32_t)c, left - above);
            } else {
              s.bin = top_bin - e;
              s.left = left - above;
            }
          }
        }
        above += x[e];
      }
    }
    if (cluster > 1)
      cluster_sync_all();
    else
      __syncthreads();
    known = (known << bits) | (uint32_t)s.bin;
    left = s.left;
  }
  // `known` is the threshold, `left` the number of keys equal to it that stay.  Every thread has neighbouring keys, as many
  // as make 16 bytes times an odd number (so that a warp's reads spread over the banks); keys above and at the threshold
  // are counted in the halves of a word (40960 of each at most).  Keys that are not held are walked by warps behind them.
  const int fours = (held + 4 * kThreads - 1) / (4 * kThreads) | 1;
  const int t0 = tid * fours * 4 < held ? tid * fours * 4 : held, t1 = t0 + fours * 4 < held ? t0 + fours * 4 : held;
  auto of = [&](uint32_t key) { return key > known ? 1u : (key == known ? 0x10000u : 0u); };
  uint32_t n_mine = 0, there = 0;  // there: a bit for each four keys with one that may stay
  for (int i = t0, bit = 1; i < t1; i += 4, bit <<= 1) {
    uint32_t n_four = 0;
    if (i + 4 <= t1) {
      const uint4 k = *reinterpret_cast<const uint4*>(s_key + i);
      n_four = of(k.x) + of(k.y) + of(k.z) + of(k.w);
    } else {
      for (int e = i; e < t1; ++e) n_four += of(s_key[e]);
    }
    n_mine += n_four;
    if (n_four) there |= bit;
  }
  uint32_t n_sum = n_mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, n_sum, o);
    if (lane >= o) n_sum += y;
  }
  if (lane == 31) s.warp_sum[warp] = (int)n_sum;
  const int rest = mine - held, stretch = ((rest + kWarps - 1) / kWarps + 31) & ~31;
  const int w0 = held + (warp * stretch < rest ? warp * stretch : rest), w1 = mine - w0 > stretch ? w0 + stretch : mine;
  if (rest > 0) {
    int up = 0, eq = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint32_t key = order_u(weight[i]);
      up += key > known;
      eq += key == known;
    }
    up = __reduce_add_sync(0xffffffffu, up);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) s.warp_n[warp][0] = up, s.warp_n[warp][1] = eq;
  }
  __syncthreads();
  const uint32_t warp_sum = (uint32_t)s.warp_sum[lane];
  const uint32_t all = __reduce_add_sync(0xffffffffu, warp_sum);
  const uint32_t n_before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum : 0u) + n_sum - n_mine;
  int above = 0, equal = 0;  // in the CTAs before this one
  int rest_up = (int)(all & 0xffffu), rest_eq = (int)(all >> 16), up_all = rest_up, eq_all = rest_eq;
  if (rest > 0) {
    const int up = s.warp_n[lane][0], eq = s.warp_n[lane][1];
    up_all += __reduce_add_sync(0xffffffffu, up);
    eq_all += __reduce_add_sync(0xffffffffu, eq);
    rest_up += __reduce_add_sync(0xffffffffu, lane < warp ? up : 0);
    rest_eq += __reduce_add_sync(0xffffffffu, lane < warp ? eq : 0);
  }
  if (cluster > 1) {
    if (tid < cluster) {
      cluster_st(&s.totals[rank][0], (uint32_t)tid, up_all);
      cluster_st(&s.totals[rank][1], (uint32_t)tid, eq_all);
    }
    cluster_sync_all();  // (the last: no CTA touches another's memory from here on)
    for (int c = 0; c < rank; ++c) {
      above += s.totals[c][0];
      equal += s.totals[c][1];
    }
  }
  int up = above + (int)(n_before & 0xffffu), eq = equal + (int)(n_before >> 16);
  for (; there; there &= there - 1) {
    const int i0 = t0 + 4 * (__ffs(there) - 1), i1 = i0 + 4 < t1 ? i0 + 4 : t1;
    for (int i = i0; i < i1; ++i) {
      const uint32_t key = s_key[i];
      const bool is_up = key > known, is_eq = key == known;
      if (is_up || (is_eq && eq < left)) put(p.first + up + (eq < left ? eq : left), p.first + (int)lo + i);
      up += is_up;
      eq += is_eq;
    }
  }
  if (rest > 0) {
    above += rest_up;
    equal += rest_eq;
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t key = i < w1 ? order_u(weight[i]) : 0u;
      const bool is_up = i < w1 && key > known, is_eq = i < w1 && key == known;
      const uint32_t ups = __ballot_sync(0xffffffffu, is_up), eqs = __ballot_sync(0xffffffffu, is_eq), low = (1u << lane) - 1;
      const int up = above + __popc(ups & low), eq = equal + __popc(eqs & low);
      if (is_up || (is_eq && eq < left)) put(p.first + up + (eq < left ? eq : left), p.first + (int)lo + i);
      above += __popc(ups);
      equal += __popc(eqs);
    }
  }
}

// Copies K and V of every kept (row, head), 2^log_vecs lanes of 16 bytes per row.
__global__ void __launch_bounds__(kCopyThreads) keep_copy_kernel(const KeepParams p, const int32_t* source, int log_vecs) {
  pdl_wait();
  const long long units = (long long)p.keep_start[p.B] * p.Hkv;
  const int vecs = 1 << log_vecs;
  const int lane = threadIdx.x & (vecs - 1);
  const long long u = ((long long)blockIdx.x * kCopyThreads + threadIdx.x) >> log_vecs;
  if (u >= units) return;
  const int row = source[u];
  const int g = u <= 0xffffffffLL ? (int)((unsigned)u % (unsigned)p.Hkv) : (int)(u % p.Hkv);
  const size_t in = (size_t)g * p.row_bytes + lane * 16, out = (size_t)u * p.row_bytes + lane * 16;
  const uint4 k = __ldcs(reinterpret_cast<const uint4*>(p.k + row * p.k_stride + in));
  const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p.v + row * p.v_stride + in));
  *reinterpret_cast<uint4*>(p.k_out + out) = k;
  *reinterpret_cast<uint4*>(p.v_out + out) = v;
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
  int log_cluster = 0;
  while (log_cluster < 3 && (segs << (log_cluster + 1)) <= num_sms && (2LL * 2048 << log_cluster) <= p.n_rows) ++log_cluster;
  const int cluster = 1 << log_cluster;
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
  err = cudaLaunchKernelEx(&cfg, keep_select_kernel, p, source, log_cluster, counted);
  if (err != cudaSuccess) return err;
  const int log_vecs = p.row_bytes == 128 ? 3 : (p.row_bytes == 256 ? 4 : 5), vecs = 1 << log_vecs;
  const long long per_block = kCopyThreads / vecs;
  const long long most = p.rows_out < p.n_rows ? p.rows_out : p.n_rows;  // a request keeps no more rows than it has
  const long long blocks = (most * p.Hkv + per_block - 1) / per_block;
  return launch_dependent(keep_copy_kernel, dim3((unsigned)blocks), dim3(kCopyThreads), 0, stream, p, source, log_vecs);
}

}  // namespace spectree
