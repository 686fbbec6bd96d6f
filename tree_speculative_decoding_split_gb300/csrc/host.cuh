// Host-side helpers shared by the C ABI files: workspace carving, device queries, tensor maps and the
// checks of a paged cache's sizes.
#pragma once

#include <cstring>

#include "common.cuh"

namespace spectree {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// Sequential carve-out of a caller-provided workspace (or a pure size count when base is null).
struct Carver {
  char* base;
  size_t off = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  template <typename T>
  T* take(size_t count) {
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off += align_up(count * sizeof(T));
    return p;
  }
};

inline int num_sms_current() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 148;
  return sms;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver entry point is looked up once per process (immutable after the first call).
inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  }
  return fn;
}

// bf16 tensor map with 128-byte swizzle.  dims/box are innermost first; strides (bytes) are for
// dims 1.. (rank - 1).
inline bool make_map_bf16(CUtensorMap* m, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  if (rank < 1 || rank > 5) return false;
  std::memset(m, 0, sizeof(*m));
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of an e4m3 pool [num_blocks][Hkv][bs][d]: (d, bs, num_blocks * Hkv) bytes, boxes of `box_rows`
// rows of one block and head, swizzled over the row's own d bytes (128 or 64).
inline bool make_map_kv8(CUtensorMap* m, const void* pool, int d, int bs, long long heads, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)bs, (cuuint64_t)heads};
  const cuuint64_t strides[2] = {(cuuint64_t)d, (cuuint64_t)d * bs};
  const cuuint32_t box[3] = {(cuuint32_t)d, (cuuint32_t)box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  std::memset(m, 0, sizeof(*m));
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(pool), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Packed K/V rows [n_rows][Hkv][d] in bf16 or float32: boxes of `box_rows` rows of one head, dense.
inline bool make_map_rows(CUtensorMap* m, const void* rows, bool bf16, int d, int Hkv, long long n_rows, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)Hkv, (cuuint64_t)n_rows};
  const cuuint64_t row = (cuuint64_t)d * (bf16 ? 2 : 4);
  const cuuint64_t strides[2] = {row, row * Hkv};
  const cuuint32_t box[3] = {(cuuint32_t)d, 1, (cuuint32_t)box_rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  std::memset(m, 0, sizeof(*m));
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(rows), dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Paged KV: block size a power of two in [16, 256], kv_capacity = max_blocks * block_size, and
// pool coordinates that fit the tensor map.
inline spec_status check_paged(int bs, int max_blocks, int num_blocks, int Hkv, long long L_cap) {
  if (bs != 16 && bs != 32 && bs != 64 && bs != 128 && bs != 256) return SPEC_ERR_UNSUPPORTED;
  if (max_blocks < 1 || num_blocks < 1) return SPEC_ERR_INVALID_ARGUMENT;
  if ((long long)max_blocks * bs != L_cap) return SPEC_ERR_INVALID_ARGUMENT;
  if ((long long)num_blocks * Hkv >= 0x7fffffffLL) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

inline int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

}  // namespace spectree
