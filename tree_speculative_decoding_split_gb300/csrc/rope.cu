// K10: positions of prompt rows and tree nodes, and the rotation of q and k by them.
//
// Positions.  A prompt's row j sits at pos0 + j, a tree's node at pos0 + its depth, as the nodes of one depth are
// candidates for the same place in the text (tech-tldr "多トークン予測（Medusa・EAGLE）", section "ツリー検証").  Depths
// come from pointer jumping in shared memory: 8 rounds cover 255 levels.
//
// Rotation.  Pair i of a head's first rot_dim channels turns by positions[r] * f_i.  The frequency is kept as a
// 64-bit fraction of a turn, so the product modulo 2^64 *is* the angle modulo a turn, exact at every position (in
// float32 the angle of position 100000 would be off by 0.004).  Its upper 32 bits are split into a quarter turn
// and a rest of at most an eighth, which float32 holds to 2^-24 of itself.
//
// Both are bound by memory: the rotation reads and writes q and k once.  One block takes a few rows: rot_dim / 2
// angles per row go to shared memory first, then every thread turns 8 (bf16) or 4 (fp32) pairs of a head, two
// 16-byte loads and stores.  It has two (row, head)s of them in flight in bf16 and four in fp32, where a unit is half as
// many pairs (four in bf16 took 9.8 us at the trees below, as more blocks no longer fit an SM; loads ahead of the
// angles took 80.4 us at the prompts).
//
// Measured: 4 fp32 prompts of 4096 to 16384 rows, 24 heads of 64, 76.7 us (0.97 of a plain copy's rate), as bf16 with 40
// heads of 128 132 us (0.93); 32 trees of 63
// bf16 nodes, 8.8 us of which 6.1 are the bytes'; one token 2.3 us, a launch.  Positions take a launch: 1.9 us for 32
// trees, and 4.7 us for 512 prompts, where every block looks row_start over and searches it.

#include "pdl.cuh"
#include "prompt.cuh"

namespace spectree {

namespace {

constexpr int kPosThreads = 256;
constexpr int kPosRows = 4 * kPosThreads;  // packed rows per block
constexpr int kRopeThreads = 256;

__global__ void __launch_bounds__(kPosThreads) positions_rows_kernel(const PositionsParams p) {
  pdl_wait();
  const int tid = threadIdx.x;
  const long long first = (long long)blockIdx.x * kPosRows;
  auto none = [&](long long r) {
    if (p.fill && r < p.n_rows) p.positions[r] = -1;
  };
  if (!row_start_ok(p.row_start, p.B, p.n_rows)) {
    if (blockIdx.x == 0 && tid == 0) set_status(p.dev_status, SPEC_ERR_CAPACITY);
    for (int u = 0; u < kPosRows / kPosThreads; ++u) none(first + u * kPosThreads + tid);
    return;
  }
  const long long behind = p.row_start[p.B], front = p.row_start[0];
  __shared__ int s_lo, s_hi;
  if (tid < 2) {  // the block's first and last request; each thread then searches between them
    const long long r = tid == 0 ? first : first + kPosRows - 1;
    const int b = request_of(p.row_start, 0, p.B, r);
    if (tid == 0)
      s_lo = b;
    else
      s_hi = b;
  }
  __syncthreads();
  const int lo = s_lo, hi = s_hi + 1;
#pragma unroll
  for (int u = 0; u < kPosRows / kPosThreads; ++u) {
    const long long r = first + u * kPosThreads + tid;
    if (r < front || r >= behind) {
      none(r);
      continue;
    }
    const int b = request_of(p.row_start, lo, hi, r);
    const int p0 = p.pos0[b], start = p.row_start[b], n = p.row_start[b + 1] - start;
    const bool bad = p0 < 0 || (long long)p0 + n - 1 > 0x7fffffffLL;
    if (bad && r == start) set_status(p.dev_status, SPEC_ERR_CAPACITY);
    p.positions[r] = bad ? -1 : p0 + (int)(r - start);
  }
}

__global__ void __launch_bounds__(kPosThreads) positions_tree_kernel(const PositionsParams p) {
  __shared__ int s_jmp[kMaxNodes], s_dep[kMaxNodes];
  pdl_wait();
  const int b = blockIdx.x, c = threadIdx.x;
  const int n = p.n_nodes[b], p0 = p.pos0[b];
  int err = 0;
  if (n < 1 || n > p.N) err = SPEC_ERR_BAD_TREE;
  if (!err && c < n) {
    const int par = p.parent[(size_t)b * p.N + c];
    if (c == 0 ? par != -1 : (par < 0 || par >= c)) err = SPEC_ERR_BAD_TREE;
    s_jmp[c] = par;
    s_dep[c] = c > 0;
  }
  const int bad_tree = __syncthreads_or(err);
  int depth = 0;
  if (!bad_tree) {
    for (int round = 0; round < 8; ++round) {
      int j = -1, more_depth = 0, next = -1;
      if (c < n && (j = s_jmp[c]) >= 0) {
        more_depth = s_dep[j];
        next = s_jmp[j];
      }
      __syncthreads();
      if (j >= 0) {
        s_dep[c] += more_depth;
        s_jmp[c] = next;
      }
      if (!__syncthreads_or(next >= 0)) break;
    }
    if (c < n) depth = s_dep[c];
  }
  const int bad_pos = __syncthreads_or(!bad_tree && c < n && (p0 < 0 || (long long)p0 + depth > 0x7fffffffLL));
  if (c == 0 && bad_tree) set_status(p.dev_status, SPEC_ERR_BAD_TREE);
  if (c == 0 && bad_pos) set_status(p.dev_status, SPEC_ERR_CAPACITY);
  if (c < p.N) p.positions[(size_t)b * p.N + c] = (bad_tree || bad_pos || c >= n) ? -1 : p0 + depth;
}

// cos and sin of the fraction of a turn `t` / 2^32.
__device__ __forceinline__ float2 turn_cos_sin(uint32_t t) {
  const uint32_t quarter = (t + 0x20000000u) >> 30;      // nearest quarter turn
  const int rest = (int)(t - (quarter << 30));           // at most 2^29 away from it
  float s, c;
  sincospif((float)rest * 4.6566128730773926e-10f, &s, &c);  // 2^-31: in half turns
  const float a = (quarter & 1u) ? -s : c, b = (quarter & 1u) ? c : s;
  return (quarter & 2u) ? make_float2(-a, -b) : make_float2(a, b);
}

// A 16-byte vector of a row as float numbers, and back.
template <bool BF16>
struct Vec {
  static constexpr int kN = BF16 ? 8 : 4;
  float x[kN];
  __device__ __forceinline__ void unpack(const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BF16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        x[i] = __uint_as_float(w[i]);
      }
    }
  }
  __device__ __forceinline__ uint4 pack() const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = BF16 ? pack_bf16x2(x[2 * i], x[2 * i + 1]) : __float_as_uint(x[i]);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int rows_block, int units, int rot_units) {
  using V = Vec<BF16>;
  constexpr int kN = V::kN;      // elements of a 16-byte vector = pairs of a unit
  constexpr int kFlight = BF16 ? 2 : 4;     // (row, head)s of a thread whose loads are under way at once
  extern __shared__ float2 s_cs[];  // [rows_block][rot / 2] cos, sin times the amplitude
  __shared__ int s_pos[64];
  const int tid = threadIdx.x;
  const int half = p.rot >> 1;
  const long long row0 = (long long)blockIdx.x * rows_block;
  const int rows = (int)(p.n_rows - row0 < rows_block ? p.n_rows - row0 : rows_block);
  pdl_wait();
  for (int i = tid; i < rows * half; i += kRopeThreads) {
    const int r = i / half, c = i - r * half;
    const int pos = p.positions[row0 + r];
    if (c == 0) s_pos[r] = pos;
    const unsigned long long turn = (unsigned long long)(uint32_t)pos * (unsigned long long)p.turns[c];
    const float2 cs = turn_cos_sin((uint32_t)(turn >> 32));
    s_cs[i] = make_float2(cs.x * p.amplitude, cs.y * p.amplitude);
  }
  __syncthreads();
  constexpr size_t kSize = BF16 ? 2 : 4;
  const int heads = p.Hq + p.Hk, work = rows * heads;
  // thread -> one unit (a pair of vectors that turn together, or pass on) of every lanes-th (row, head)
  const int lanes = kRopeThreads / units;
  const int u = tid % units, lane = tid / units;
  if (lane >= lanes) return;
  const bool turns = u < rot_units;
  const int a_off = turns ? (INTER ? u * 2 * kN : u * kN) : p.rot + (u - rot_units) * 2 * kN;
  const int b_off = turns && !INTER ? a_off + half : a_off + kN;
  for (int w0 = lane; w0 < work; w0 += lanes * kFlight) {
    uint4 va[kFlight], vb[kFlight];
    char* dst[kFlight];
    int at[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int w = w0 + f * lanes;
      at[f] = -1;
      if (w < work) {
        const int r = w / heads, h = w - r * heads;
        if (s_pos[r] >= 0) {
          const long long row = row0 + r;
          const bool is_q = h < p.Hq;
          const long long hd = (long long)(is_q ? h : h - p.Hq) * p.d;
          const char* src = is_q ? static_cast<const char*>(p.q) + (row * p.q_stride + hd) * kSize
                                 : static_cast<const char*>(p.k) + (row * p.k_stride + hd) * kSize;
          dst[f] = is_q ? static_cast<char*>(p.q_out) + (row * p.q_out_stride + hd) * kSize
                        : static_cast<char*>(p.k_out) + (row * p.k_out_stride + hd) * kSize;
          va[f] = *reinterpret_cast<const uint4*>(src + a_off * kSize);
          vb[f] = *reinterpret_cast<const uint4*>(src + b_off * kSize);
          at[f] = r;
        }
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (at[f] < 0) continue;
      if (turns) {
        V a, b;
        a.unpack(va[f]);
        b.unpack(vb[f]);
        const float4* cs4 = reinterpret_cast<const float4*>(s_cs + at[f] * half + u * kN);
        V oa, ob;
#pragma unroll
        for (int i = 0; i < kN; i += 2) {
          const float4 cs = cs4[i >> 1];  // cos, sin of pairs i and i + 1
          if (INTER) {  // pair i: elements 2 i, 2 i + 1 of the unit's two vectors side by side
            V& in = i < kN / 2 ? a : b;
            V& to = i < kN / 2 ? oa : ob;
            const int e = (2 * i) % kN;
            to.x[e] = in.x[e] * cs.x - in.x[e + 1] * cs.y;
            to.x[e + 1] = in.x[e] * cs.y + in.x[e + 1] * cs.x;
            to.x[e + 2] = in.x[e + 2] * cs.z - in.x[e + 3] * cs.w;
            to.x[e + 3] = in.x[e + 2] * cs.w + in.x[e + 3] * cs.z;
          } else {
            oa.x[i] = a.x[i] * cs.x - b.x[i] * cs.y;
            ob.x[i] = a.x[i] * cs.y + b.x[i] * cs.x;
            oa.x[i + 1] = a.x[i + 1] * cs.z - b.x[i + 1] * cs.w;
            ob.x[i + 1] = a.x[i + 1] * cs.w + b.x[i + 1] * cs.z;
          }
        }
        va[f] = oa.pack();
        vb[f] = ob.pack();
      }
      *reinterpret_cast<uint4*>(dst[f] + a_off * kSize) = va[f];
      *reinterpret_cast<uint4*>(dst[f] + b_off * kSize) = vb[f];
    }
  }
}

template <bool BF16, bool INTER>
cudaError_t launch_rope_as(const RopeParams& p, int num_sms, cudaStream_t stream) {
  const int unit = 2 * Vec<BF16>::kN;
  const int units = p.d / unit, rot_units = p.rot / unit;
  // Rows per block: as many as give every thread kFlight (row, head)s twice, fewer where the rows would not fill
  // the GPU four times over; at most 64, and 32 KB of angles.
  const int lanes = kRopeThreads / units, heads = p.Hq + p.Hk;
  long long rows = (8LL * lanes + heads - 1) / heads;
  const long long fill = p.n_rows / (4LL * num_sms);
  if (rows > fill) rows = fill;
  if (rows > 4096 / (p.rot / 2)) rows = 4096 / (p.rot / 2);
  if (rows > 64) rows = 64;
  if (rows < 1) rows = 1;
  const long long blocks = (p.n_rows + rows - 1) / rows;
  return launch_dependent(rope_kernel<BF16, INTER>, dim3((unsigned)blocks), dim3(kRopeThreads),
                          (size_t)rows * (p.rot / 2) * sizeof(float2), stream, p, (int)rows, units, rot_units);
}

}  // namespace

cudaError_t launch_rope_positions(const PositionsParams& p, cudaStream_t stream) {
  if (p.parent)
    return launch_dependent(positions_tree_kernel, dim3(p.B), dim3(kPosThreads), 0, stream, p);
  const long long blocks = p.n_rows > 0 ? (p.n_rows + kPosRows - 1) / kPosRows : 1;
  return launch_dependent(positions_rows_kernel, dim3((unsigned)blocks), dim3(kPosThreads), 0, stream, p);
}

cudaError_t launch_rope(const RopeParams& p, int num_sms, cudaStream_t stream) {
  if (p.is_bf16)
    return p.interleaved ? launch_rope_as<true, true>(p, num_sms, stream) : launch_rope_as<true, false>(p, num_sms, stream);
  return p.interleaved ? launch_rope_as<false, true>(p, num_sms, stream) : launch_rope_as<false, false>(p, num_sms, stream);
}

}  // namespace spectree
