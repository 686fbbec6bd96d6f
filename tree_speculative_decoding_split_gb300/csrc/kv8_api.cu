// C ABI of the 8-bit paged KV cache (see include/spectree.h): argument checks, workspace, tensor maps and
// launches of the block tables, the appending of rows and the attention over the cache.

#include <cmath>
#include <cstring>

#include "common.cuh"
#include "host.cuh"
#include "kernels.cuh"

using namespace spectree;

namespace {

spec_status check_reserve(const spec_kv_reserve_args* a) {
  if (!a) return SPEC_ERR_INVALID_ARGUMENT;
  if (a->batch < 1 || a->slot_cap < 0) return SPEC_ERR_INVALID_ARGUMENT;
  const spec_status ps =
      check_paged(a->block_size, a->max_blocks, a->num_blocks, 1, (long long)a->max_blocks * a->block_size);
  if (ps != SPEC_OK) return ps;
  if (a->batch > SPEC_MAX_RESERVE_BATCH || a->slot_cap > 0x7fffffffLL ||
      (long long)a->batch * a->max_blocks > 0x7fffffffLL)
    return SPEC_ERR_UNSUPPORTED;
  if (!a->seq_len || !a->n_new || !a->block_table || !a->n_blocks || !a->free_list || !a->free_count)
    return SPEC_ERR_INVALID_ARGUMENT;
  if (a->slot_map && (!a->row_start || (a->slot_cap > 0 && !aligned16(a->slot_map)))) return SPEC_ERR_INVALID_ARGUMENT;
  return SPEC_OK;
}

spec_status check_append(const spec_kv8_append_args* a) {
  if (!a) return SPEC_ERR_INVALID_ARGUMENT;
  if (a->dtype != SPEC_DTYPE_F32 && a->dtype != SPEC_DTYPE_BF16) return SPEC_ERR_UNSUPPORTED;
  if (a->head_dim != 64 && a->head_dim != 128) return SPEC_ERR_UNSUPPORTED;
  if (a->batch < 1 || a->num_kv_heads < 1 || a->reserved0 != 0) return SPEC_ERR_INVALID_ARGUMENT;
  const spec_status ps = check_paged(a->block_size, a->max_blocks, a->num_blocks, a->num_kv_heads,
                                     (long long)a->max_blocks * a->block_size);
  if (ps != SPEC_OK) return ps;
  if (!a->k_new || !a->v_new || !a->seq_len || !a->block_table || !a->k_cache || !a->v_cache || !a->k_scale ||
      !a->v_scale || a->new_len == a->seq_len)
    return SPEC_ERR_INVALID_ARGUMENT;
  if (!aligned16(a->k_new) || !aligned16(a->v_new) || !aligned16(a->k_cache) || !aligned16(a->v_cache))
    return SPEC_ERR_INVALID_ARGUMENT;
  if (a->path) {
    if (!a->accept_len || a->row_start || a->n_rows != 0 || a->n_max < 1 || a->path_cap < 1)
      return SPEC_ERR_INVALID_ARGUMENT;
    if (a->n_max > SPEC_MAX_NODES) return SPEC_ERR_UNSUPPORTED;
  } else {
    if (!a->row_start || a->accept_len || a->n_rows < 0 || a->n_max != 0 || a->path_cap != 0)
      return SPEC_ERR_INVALID_ARGUMENT;
    if (a->n_rows > 0x7fffffffLL) return SPEC_ERR_UNSUPPORTED;
  }
  return SPEC_OK;
}

Kv8AppendParams append_params(const spec_kv8_append_args* a, int32_t* dev_status) {
  Kv8AppendParams p;
  std::memset(&p, 0, sizeof(p));
  p.B = a->batch; p.Hkv = a->num_kv_heads; p.d = a->head_dim;
  p.bs = a->block_size; p.bs_shift = log2_of(a->block_size);
  p.max_blocks = a->max_blocks; p.num_blocks = a->num_blocks;
  p.is_bf16 = a->dtype == SPEC_DTYPE_BF16;
  p.N = a->n_max; p.path_cap = a->path_cap; p.n_rows = a->n_rows;
  p.k_new = a->k_new; p.v_new = a->v_new; p.row_start = a->row_start; p.path = a->path; p.accept_len = a->accept_len;
  p.seq_len = a->seq_len; p.table = a->block_table;
  p.k_cache = a->k_cache; p.v_cache = a->v_cache; p.k_scale = a->k_scale; p.v_scale = a->v_scale;
  p.new_len = a->new_len;
  p.dev_status = dev_status;
  // n rows at any offset touch at most floor((n + bs - 2) / bs) + 1 blocks; a path has at most n_max rows
  const int rows = a->path_cap < a->n_max ? a->path_cap : a->n_max;
  p.units_per_req = (rows + a->block_size - 2) / a->block_size + 1;
  return p;
}

spec_status check_attn_kv8(const spec_attn_kv8_args* a) {
  if (!a) return SPEC_ERR_INVALID_ARGUMENT;
  if (a->dtype != SPEC_DTYPE_BF16) return SPEC_ERR_UNSUPPORTED;
  if (a->head_dim != 64 && a->head_dim != 128) return SPEC_ERR_UNSUPPORTED;
  if (a->batch < 1 || a->n_max < 1 || a->num_q_heads < 1 || a->num_kv_heads < 1) return SPEC_ERR_INVALID_ARGUMENT;
  if (a->n_max > SPEC_MAX_NODES) return SPEC_ERR_UNSUPPORTED;
  if (a->num_q_heads % a->num_kv_heads) return SPEC_ERR_INVALID_ARGUMENT;
  if ((long long)a->batch * a->num_kv_heads > 65535) return SPEC_ERR_UNSUPPORTED;  // CTAs stay within 32 bits
  const spec_status ps = check_paged(a->block_size, a->max_blocks, a->num_blocks, a->num_kv_heads,
                                     (long long)a->max_blocks * a->block_size);
  if (ps != SPEC_OK) return ps;
  if ((long long)a->max_blocks * a->block_size > 0x7fffffffLL - 128) return SPEC_ERR_UNSUPPORTED;
  if ((long long)a->n_max * a->num_q_heads * a->batch > 0x7fffffffLL) return SPEC_ERR_UNSUPPORTED;
  if (a->num_q_heads / a->num_kv_heads > 256) return SPEC_ERR_UNSUPPORTED;
  if (!a->q || !a->k_tree || !a->v_tree || !a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale || !a->prefix_len ||
      !a->n_nodes || !a->parent || !a->block_table || !a->out)
    return SPEC_ERR_INVALID_ARGUMENT;
  if (!aligned16(a->q) || !aligned16(a->k_tree) || !aligned16(a->v_tree) || !aligned16(a->k_cache) ||
      !aligned16(a->v_cache) || !aligned16(a->out))
    return SPEC_ERR_INVALID_ARGUMENT;
  return SPEC_OK;
}

struct AttnKv8Layout {
  float* part_o;
  float2* part_ml;
  int2* used;
  Kv8AttnPlan plan;
  size_t bytes;
};

AttnKv8Layout layout_attn_kv8(const spec_attn_kv8_args* a, void* ws) {
  AttnKv8Layout l;
  l.plan = plan_attention_kv8(a->batch, a->n_max, a->num_q_heads / a->num_kv_heads, a->num_kv_heads,
                              (long long)a->max_blocks * a->block_size, num_sms_current());
  const size_t ctas = (size_t)(a->batch * l.plan.base + l.plan.extra) * a->num_kv_heads * l.plan.n_rt;
  const size_t rows = l.plan.merge() ? ctas * l.plan.rows_cta : 0;
  Carver c(ws);
  l.used = c.take<int2>(a->batch);
  l.part_ml = c.take<float2>(rows);
  l.part_o = c.take<float>(rows * a->head_dim);
  l.bytes = c.off;
  return l;
}

}  // namespace

extern "C" {

spec_status spec_kv_reserve(const spec_kv_reserve_args* a, int32_t* dev_status, void* stream) {
  const spec_status st = check_reserve(a);
  if (st != SPEC_OK) return st;
  ReserveParams p;
  std::memset(&p, 0, sizeof(p));
  p.B = a->batch; p.bs = a->block_size; p.bs_shift = log2_of(a->block_size);
  p.max_blocks = a->max_blocks; p.num_blocks = a->num_blocks;
  p.slot_cap = a->slot_map ? a->slot_cap : 0;
  p.seq_len = a->seq_len; p.n_new = a->n_new; p.table = a->block_table; p.n_blocks = a->n_blocks;
  p.free_list = a->free_list; p.free_count = a->free_count; p.slot_map = a->slot_map; p.row_start = a->row_start;
  p.dev_status = dev_status;
  return launch_kv_reserve(p, num_sms_current(), static_cast<cudaStream_t>(stream)) == cudaSuccess ? SPEC_OK
                                                                                                  : SPEC_ERR_CUDA;
}

spec_status spec_kv8_append(const spec_kv8_append_args* a, int32_t* dev_status, void* stream) {
  const spec_status st = check_append(a);
  if (st != SPEC_OK) return st;
  const Kv8AppendParams p = append_params(a, dev_status);
  if (kv8_append_grid(p) == 0) return SPEC_ERR_UNSUPPORTED;
  CUtensorMap tm[2];
  const bool boxes = kv8_append_boxes(p);
  if (boxes && (!make_map_rows(&tm[0], p.k_new, p.is_bf16, p.d, p.Hkv, p.n_rows, p.bs) ||
                !make_map_rows(&tm[1], p.v_new, p.is_bf16, p.d, p.Hkv, p.n_rows, p.bs)))
    return SPEC_ERR_CUDA;
  return launch_kv8_append(boxes ? tm : nullptr, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SPEC_OK
                                                                                                    : SPEC_ERR_CUDA;
}

size_t spec_tree_attention_kv8_workspace(const spec_attn_kv8_args* a) {
  if (check_attn_kv8(a) != SPEC_OK) return 0;
  return layout_attn_kv8(a, nullptr).bytes;
}

spec_status spec_tree_attention_kv8(const spec_attn_kv8_args* a, void* workspace, size_t workspace_bytes,
                                    int32_t* dev_status, void* stream_ptr) {
  const spec_status st = check_attn_kv8(a);
  if (st != SPEC_OK) return st;
  if (!workspace || !aligned16(workspace)) return SPEC_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < layout_attn_kv8(a, nullptr).bytes) return SPEC_ERR_WORKSPACE_TOO_SMALL;
  const AttnKv8Layout l = layout_attn_kv8(a, workspace);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  Kv8AttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(a->q);
  p.k_tree = static_cast<const uint16_t*>(a->k_tree);
  p.v_tree = static_cast<const uint16_t*>(a->v_tree);
  p.k_scale = a->k_scale; p.v_scale = a->v_scale;
  p.prefix_len = a->prefix_len; p.n_nodes = a->n_nodes; p.parent = a->parent; p.table = a->block_table;
  p.out = static_cast<uint16_t*>(a->out); p.lse = a->lse;
  p.part_o = l.part_o; p.part_ml = l.part_ml; p.used = l.plan.merge() ? l.used : nullptr;
  p.dev_status = dev_status;
  p.B = a->batch; p.N = a->n_max; p.Hq = a->num_q_heads; p.Hkv = a->num_kv_heads; p.G = p.Hq / p.Hkv;
  p.g_magic = p.G > 1 ? (uint32_t)((1ull << 32) / (uint32_t)p.G) + 1u : 0u;
  p.d = a->head_dim; p.bs = a->block_size; p.bs_shift = log2_of(a->block_size);
  p.max_blocks = a->max_blocks; p.num_blocks = a->num_blocks;
  p.L_cap = (long long)a->max_blocks * a->block_size;
  p.base = l.plan.base; p.extra = l.plan.extra; p.rows_cta = l.plan.rows_cta; p.n_rt = l.plan.n_rt;
  const float scale = a->scale > 0.f ? a->scale : 1.f / std::sqrt((float)a->head_dim);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.unit_shift = l.plan.unit_shift;
  p.inv_slots = 1.f / (float)l.plan.slots;
  p.fixed_steps = l.plan.fixed_steps;
  CUtensorMap tm[4];
  const long long heads = (long long)a->num_blocks * a->num_kv_heads;
  const int box = l.plan.groups == 0 ? 16 : (p.bs < 128 ? p.bs : 128);
  if (!make_map_kv8(&tm[0], a->k_cache, p.d, p.bs, heads, box) || !make_map_kv8(&tm[1], a->v_cache, p.d, p.bs, heads, box))
    return SPEC_ERR_CUDA;
  if (l.plan.groups == 0) {
    if (launch_attention_kv8_rows(&tm[0], &tm[1], p, stream) != cudaSuccess) return SPEC_ERR_CUDA;
  } else {
    // the tree's rows as (d, Hkv, N, B): boxes of 64 dimensions of 64 nodes of one head
    const cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)p.Hkv, (cuuint64_t)p.N, (cuuint64_t)p.B};
    const cuuint64_t row = (cuuint64_t)p.d * 2;
    const cuuint64_t strides[3] = {row, row * p.Hkv, row * p.Hkv * p.N};
    const cuuint32_t tbox[4] = {64, 1, 64, 1};
    if (!make_map_bf16(&tm[2], a->k_tree, 4, dims, strides, tbox) ||
        !make_map_bf16(&tm[3], a->v_tree, 4, dims, strides, tbox))
      return SPEC_ERR_CUDA;
    if (launch_attention_kv8_tc(tm, p, l.plan.groups, stream) != cudaSuccess) return SPEC_ERR_CUDA;
  }
  if (p.used && launch_attention_kv8_merge(p, stream) != cudaSuccess) return SPEC_ERR_CUDA;
  return SPEC_OK;
}

}  // extern "C"
