// Device helpers shared by the attention kernels over the 8-bit paged cache.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.cuh"

namespace spectree {

constexpr float kKv8MinScale = 5.4210108624275222e-20f;  // 2^-64
constexpr float kKv8MaxScale = 1.329227995784916e36f;    // 2^120

__device__ __forceinline__ float kv8_clamp_scale(float s) { return fminf(fmaxf(s, kKv8MinScale), kKv8MaxScale); }

// How a request's prefix is cut into splits of whole steps (2^unit_shift keys): as many splits as the launch
// has, but none shorter than 256 keys.  The merge evaluates the same function.
struct Kv8Split {
  int n;      // splits in use, >= 1
  int steps;  // steps per split
};
__host__ __device__ __forceinline__ Kv8Split kv8_split(long long len, int n_split, int unit_shift) {
  const int total = (int)((len + (1 << unit_shift) - 1) >> unit_shift);
  int steps = (total + n_split - 1) / n_split;
  if (steps < (256 >> unit_shift)) steps = 256 >> unit_shift;
  Kv8Split s;
  s.steps = steps;
  s.n = total > 0 ? (total + steps - 1) / steps : 1;
  return s;
}

// Index of row (node row / G, head h G + row % G) of request b in [B][N][Hq].
__device__ __forceinline__ int kv8_node(const Kv8AttnParams& p, int row) {
  return p.G == 1 ? row : (int)__umulhi((uint32_t)row, p.g_magic);
}
__device__ __forceinline__ size_t kv8_row(const Kv8AttnParams& p, int b, int h, int row) {
  const int i = kv8_node(p, row);
  return ((size_t)b * p.N + i) * p.Hq + h * p.G + (row - i * p.G);
}

// Verdict on request b from its counts alone; `len` is the prefix length every kernel goes on with.
__device__ __forceinline__ int kv8_counts(const Kv8AttnParams& p, int b, long long* len, int* n) {
  *len = p.prefix_len[b];
  *n = p.n_nodes[b];
  int err = 0;
  if (*n < 1 || *n > p.N) {
    err = SPEC_ERR_BAD_TREE;
    *n = 0;
  }
  if (*len < 0 || *len > p.L_cap) {
    if (!err) err = SPEC_ERR_CAPACITY;
    *len = 0;
  }
  return err;
}

}  // namespace spectree
