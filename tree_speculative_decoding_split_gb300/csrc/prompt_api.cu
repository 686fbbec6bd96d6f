// C ABI of the calls that take prompts to the cache (see include/spectree.h): argument checks, workspace, tensor maps
// and launches of positions, rotation, prompt attention, key weights and the rows kept for a budget.

#include <cmath>
#include <cstring>

#include "common.cuh"
#include "host.cuh"
#include "prompt.cuh"

using namespace spectree;

namespace {

constexpr long long kMaxRows = 0x7fffffffLL - 256;  // tiles may reach 255 rows past the last one

constexpr long long kMaxKeepRows = 0x7fffffffLL - 16384;  // the choice counts up to two batches of a block past the last one

// Rows of `heads` heads of d elements, `stride` elements apart: long enough, and multiples of 16 bytes.
bool row_stride_ok(long long stride, long long heads, int d, int size) {
  return stride >= heads * d && (stride * size) % 16 == 0 && stride < (1LL << 38);
}

spec_status check_positions(const spec_rope_positions_args* a) {
  if (!a || a->batch < 1 || !a->pos0) return SPEC_ERR_INVALID_ARGUMENT;
  if ((a->row_start != nullptr) == (a->parent != nullptr)) return SPEC_ERR_INVALID_ARGUMENT;
  if (a->fill < 0 || a->fill > 1 || (a->fill && a->parent) || a->reserved0 != 0) return SPEC_ERR_INVALID_ARGUMENT;
  if (a->parent) {
    if (!a->n_nodes || a->n_rows != 0 || a->n_max < 1 || !a->positions) return SPEC_ERR_INVALID_ARGUMENT;
    if (a->n_max > SPEC_MAX_NODES) return SPEC_ERR_UNSUPPORTED;
  } else {
    if (a->n_nodes || a->n_max != 0 || a->n_rows < 0 || (!a->positions && a->n_rows > 0)) return SPEC_ERR_INVALID_ARGUMENT;
    if (a->n_rows > 0x7fffffffLL || a->batch > SPEC_MAX_RESERVE_BATCH) return SPEC_ERR_UNSUPPORTED;
  }
  return SPEC_OK;
}

spec_status check_rope(const spec_rope_args* a) {
  if (!a) return SPEC_ERR_INVALID_ARGUMENT;
  if (a->dtype != SPEC_DTYPE_F32 && a->dtype != SPEC_DTYPE_BF16) return SPEC_ERR_UNSUPPORTED;
  if (a->layout != SPEC_ROPE_HALF && a->layout != SPEC_ROPE_INTERLEAVED) return SPEC_ERR_UNSUPPORTED;
  if (a->num_q_heads < 1 || a->num_k_heads < 1 || a->head_dim < 1 || a->rot_dim < 1 || a->n_rows < 0 || a->reserved0 != 0 ||
      !std::isfinite(a->amplitude))
    return SPEC_ERR_INVALID_ARGUMENT;
  if (a->head_dim % 16 || a->head_dim > 256 || a->rot_dim % 16 || a->rot_dim > a->head_dim || a->n_rows > 0x7fffffffLL ||
      (long long)a->num_q_heads + a->num_k_heads > 65535)
    return SPEC_ERR_UNSUPPORTED;
  const int size = a->dtype == SPEC_DTYPE_BF16 ? 2 : 4;
  if (!row_stride_ok(a->q_stride, a->num_q_heads, a->head_dim, size) ||
      !row_stride_ok(a->q_out_stride, a->num_q_heads, a->head_dim, size) ||
      !row_stride_ok(a->k_stride, a->num_k_heads, a->head_dim, size) ||
      !row_stride_ok(a->k_out_stride, a->num_k_heads, a->head_dim, size))
    return SPEC_ERR_INVALID_ARGUMENT;
  if (a->n_rows == 0) return SPEC_OK;
  if (!a->q || !a->k || !a->positions || !a->turns || !a->q_out || !a->k_out) return SPEC_ERR_INVALID_ARGUMENT;
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->q_out) || !aligned16(a->k_out)) return SPEC_ERR_INVALID_ARGUMENT;
  if ((a->q_out == a->q && a->q_out_stride != a->q_stride) || (a->k_out == a->k && a->k_out_stride != a->k_stride))
    return SPEC_ERR_INVALID_ARGUMENT;
  return SPEC_OK;
}

// What prompt attention and key weights ask of their sizes alike.
spec_status check_prompt(int dtype, int B, int Hq, int Hkv, int d, long long n_rows, long long q_stride, long long k_stride,
                         float scale) {
  if (dtype != SPEC_DTYPE_BF16) return SPEC_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return SPEC_ERR_UNSUPPORTED;
  if (B < 1 || Hq < 1 || Hkv < 1 || n_rows < 0 || Hq % Hkv || !std::isfinite(scale)) return SPEC_ERR_INVALID_ARGUMENT;
  if (B > SPEC_MAX_RESERVE_BATCH || Hq / Hkv > 128 || n_rows > kMaxRows) return SPEC_ERR_UNSUPPORTED;
  if (!row_stride_ok(q_stride, Hq, d, 2) || !row_stride_ok(k_stride, Hkv, d, 2)) return SPEC_ERR_INVALID_ARGUMENT;
  return SPEC_OK;
}

int attn_step(const spec_prompt_attn_args* a) { return 2 * (128 / (a->num_q_heads / a->num_kv_heads)); }

// Do the pieces of all heads count in 32 bits?
bool pieces_ok(long long n_rows, int B, int step, int Hkv) { return plan_items(n_rows, B, step) * Hkv <= 0x7fffffffLL; }

spec_status check_prompt_attn(const spec_prompt_attn_args* a) {
  if (!a) return SPEC_ERR_INVALID_ARGUMENT;
  const spec_status st = check_prompt(a->dtype, a->batch, a->num_q_heads, a->num_kv_heads, a->head_dim, a->n_rows, a->q_stride,
                                      a->k_stride, a->scale);
  if (st != SPEC_OK) return st;
  if (!row_stride_ok(a->v_stride, a->num_kv_heads, a->head_dim, 2) || !a->row_start) return SPEC_ERR_INVALID_ARGUMENT;
  if (!pieces_ok(a->n_rows, a->batch, attn_step(a), a->num_kv_heads)) return SPEC_ERR_UNSUPPORTED;
  if (a->n_rows == 0) return SPEC_OK;
  if (!a->q || !a->k || !a->v || !a->out) return SPEC_ERR_INVALID_ARGUMENT;
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->out)) return SPEC_ERR_INVALID_ARGUMENT;
  return SPEC_OK;
}

spec_status check_key_weights(const spec_key_weights_args* a) {
  if (!a) return SPEC_ERR_INVALID_ARGUMENT;
  const spec_status st = check_prompt(a->dtype, a->batch, a->num_q_heads, a->num_kv_heads, a->head_dim, a->n_rows, a->q_stride,
                                      a->k_stride, a->scale);
  if (st != SPEC_OK) return st;
  if (a->window < 1 || a->reserved0 != 0 || !a->row_start) return SPEC_ERR_INVALID_ARGUMENT;
  if (!pieces_ok(a->n_rows, a->batch, kWeightKeys, a->num_kv_heads)) return SPEC_ERR_UNSUPPORTED;
  if (a->n_rows == 0) return SPEC_OK;
  if (!a->q || !a->k || !a->lse || !a->weight || !aligned16(a->q) || !aligned16(a->k)) return SPEC_ERR_INVALID_ARGUMENT;
  return SPEC_OK;
}

spec_status check_keep(const spec_kv_keep_args* a) {
  if (!a) return SPEC_ERR_INVALID_ARGUMENT;
  if (a->dtype != SPEC_DTYPE_F32 && a->dtype != SPEC_DTYPE_BF16) return SPEC_ERR_UNSUPPORTED;
  if (a->head_dim != 64 && a->head_dim != 128) return SPEC_ERR_UNSUPPORTED;
  if (a->batch < 1 || a->num_kv_heads < 1 || a->n_rows < 0 || a->rows_out < 0 || a->budget < 1 || a->first < 0 || a->last < 0 ||
      (long long)a->first + a->last > a->budget || a->reserved0 != 0)
    return SPEC_ERR_INVALID_ARGUMENT;
  if (a->n_rows > kMaxKeepRows || a->rows_out > 0x7fffffffLL || a->batch > SPEC_MAX_RESERVE_BATCH ||
      (long long)a->batch * a->num_kv_heads >= (1LL << 27))
    return SPEC_ERR_UNSUPPORTED;
  if (a->rows_out * a->num_kv_heads >= (1LL << 33)) return SPEC_ERR_UNSUPPORTED;  // the copy's grid
  const int size = a->dtype == SPEC_DTYPE_BF16 ? 2 : 4;
  if (!row_stride_ok(a->k_stride, a->num_kv_heads, a->head_dim, size) ||
      !row_stride_ok(a->v_stride, a->num_kv_heads, a->head_dim, size))
    return SPEC_ERR_INVALID_ARGUMENT;
  if (!a->row_start || !a->keep_start || !a->n_keep) return SPEC_ERR_INVALID_ARGUMENT;
  if (a->n_rows > 0 && (!a->k || !a->v || !a->weight || !aligned16(a->k) || !aligned16(a->v))) return SPEC_ERR_INVALID_ARGUMENT;
  if (a->rows_out > 0 && (!a->k_out || !a->v_out || !a->index || !aligned16(a->k_out) || !aligned16(a->v_out)))
    return SPEC_ERR_INVALID_ARGUMENT;
  return SPEC_OK;
}

// The plan of a call: how many rows an item takes, and the list's place in the workspace.
struct PlanLayout {
  int32_t* count;
  PromptItem* items;
  size_t bytes;
};
PlanLayout layout_plan(long long n_rows, int B, int step, void* ws) {
  PlanLayout l;
  Carver c(ws);
  l.count = c.take<int32_t>(1);
  l.items = c.take<PromptItem>((size_t)plan_items(n_rows, B, step));
  l.bytes = c.off;
  return l;
}

// Rows [n_rows][H][d], `stride` elements apart, as (d, H, n_rows): boxes of 64 dimensions, `heads` heads and `rows` rows.
bool make_map_heads(CUtensorMap* m, const void* x, int d, int H, long long n_rows, long long stride, int heads, int rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)n_rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)rows};
  return make_map_bf16(m, x, 3, dims, strides, box);
}

float scale_of(float scale, int d) { return scale > 0.f ? scale : 1.f / std::sqrt((float)d); }

// Launches the plan where the call needs one (n_rows 0: its checks alone) and says where the kernel finds it.
spec_status plan(long long n_rows, int B, int step, int by_work, const int32_t* row_start, const PlanLayout& l, PlanView* view,
                 int32_t* dev_status, cudaStream_t stream) {
  const bool list = B > (by_work ? 1 : kPlanInKernel) || n_rows == 0;
  view->items = list ? l.items : nullptr;
  view->count = l.count;
  view->row_start = row_start;
  view->n_rows = n_rows;
  view->B = B;
  view->step = step;
  view->by_work = by_work;
  if (!list) return SPEC_OK;
  PlanParams p;
  p.B = B; p.step = step; p.by_work = by_work; p.n_rows = n_rows; p.row_start = row_start;
  p.items = l.items; p.count = l.count; p.dev_status = dev_status;
  return launch_prompt_plan(p, stream) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

int grid_for(long long items, int Hkv) {
  const long long most = items * Hkv;
  const int sms = num_sms_current();
  return most < sms ? (int)most : sms;
}


}  // namespace

extern "C" {

spec_status spec_rope_table(int32_t rot_dim, double base, int32_t kind, double factor, int64_t original_len, double low,
                            double high, int64_t* turns) {
  if (!turns || rot_dim < 2 || rot_dim % 2 || !std::isfinite(base) || base <= 1.0 || !std::isfinite(factor) || factor <= 0.0)
    return SPEC_ERR_INVALID_ARGUMENT;
  if (kind < SPEC_ROPE_NONE || kind > SPEC_ROPE_RAMP) return SPEC_ERR_UNSUPPORTED;
  const bool by_turns = kind == SPEC_ROPE_BANDS || kind == SPEC_ROPE_RAMP;
  if (by_turns && (original_len < 1 || !std::isfinite(low) || !std::isfinite(high) || low <= 0.0 || high <= low))
    return SPEC_ERR_INVALID_ARGUMENT;
  if (kind == SPEC_ROPE_BASE && rot_dim == 2) return SPEC_ERR_INVALID_ARGUMENT;
  const double two_pi = 6.283185307179586476925;
  const int half = rot_dim / 2;
  if (kind == SPEC_ROPE_BASE) {
    base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    if (!std::isfinite(base)) return SPEC_ERR_INVALID_ARGUMENT;
  }
  // the (real) index whose frequency makes r turns over the original length
  auto index_of = [&](double r) { return rot_dim * std::log((double)original_len / (r * two_pi)) / (2.0 * std::log(base)); };
  double i_high = 0.0, i_low = 0.0;
  if (kind == SPEC_ROPE_RAMP) {
    // (the ramp may end, or lie, behind the last index: after a long trained length no frequency is scaled in full, or at all)
    i_high = std::fmin(std::fmax(std::floor(index_of(high)), 0.0), rot_dim - 1.0);
    i_low = std::fmin(std::fmax(std::ceil(index_of(low)), 0.0), rot_dim - 1.0);
    if (i_low < i_high + 0.001) i_low = i_high + 0.001;
  }
  for (int pass = 0; pass < 2; ++pass)  // (nothing is written before every frequency is known to fit)
    for (int i = 0; i < half; ++i) {
      double f = std::pow(base, -2.0 * i / rot_dim);
      double share = 0.0;  // of f / factor
      if (kind == SPEC_ROPE_LINEAR) share = 1.0;
      if (kind == SPEC_ROPE_BANDS) {
        const double r = (double)original_len * f / two_pi;
        share = std::fmin(std::fmax((high - r) / (high - low), 0.0), 1.0);
      }
      if (kind == SPEC_ROPE_RAMP) share = std::fmin(std::fmax((i - i_high) / (i_low - i_high), 0.0), 1.0);
      f = share == 1.0 ? f / factor : f * (1.0 - share) + f / factor * share;
      const double turn = f / two_pi;
      if (!(turn < 0.5)) return SPEC_ERR_UNSUPPORTED;
      if (pass) turns[i] = (int64_t)std::floor(turn * 18446744073709551616.0);  // 2^64
    }
  return SPEC_OK;
}

spec_status spec_rope_positions(const spec_rope_positions_args* a, int32_t* dev_status, void* stream) {
  const spec_status st = check_positions(a);
  if (st != SPEC_OK) return st;
  PositionsParams p;
  p.B = a->batch; p.N = a->n_max; p.n_rows = a->n_rows; p.pos0 = a->pos0; p.row_start = a->row_start;
  p.parent = a->parent; p.n_nodes = a->n_nodes; p.positions = a->positions; p.fill = a->fill; p.dev_status = dev_status;
  return launch_rope_positions(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_rope(const spec_rope_args* a, void* stream) {
  const spec_status st = check_rope(a);
  if (st != SPEC_OK || a->n_rows == 0) return st;
  RopeParams p;
  p.is_bf16 = a->dtype == SPEC_DTYPE_BF16; p.interleaved = a->layout == SPEC_ROPE_INTERLEAVED;
  p.Hq = a->num_q_heads; p.Hk = a->num_k_heads; p.d = a->head_dim; p.rot = a->rot_dim; p.n_rows = a->n_rows;
  p.q_stride = a->q_stride; p.k_stride = a->k_stride; p.q_out_stride = a->q_out_stride; p.k_out_stride = a->k_out_stride;
  p.amplitude = a->amplitude; p.q = a->q; p.k = a->k; p.positions = a->positions; p.turns = a->turns;
  p.q_out = a->q_out; p.k_out = a->k_out;
  return launch_rope(p, num_sms_current(), static_cast<cudaStream_t>(stream)) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

size_t spec_prompt_attention_workspace(const spec_prompt_attn_args* a) {
  if (check_prompt_attn(a) != SPEC_OK) return 0;
  return layout_plan(a->n_rows, a->batch, attn_step(a), nullptr).bytes;
}

spec_status spec_prompt_attention(const spec_prompt_attn_args* a, void* workspace, size_t workspace_bytes,
                                  int32_t* dev_status, void* stream_ptr) {
  const spec_status st = check_prompt_attn(a);
  if (st != SPEC_OK) return st;
  if (!workspace || !aligned16(workspace)) return SPEC_ERR_INVALID_ARGUMENT;
  const int step = attn_step(a);
  const PlanLayout l = layout_plan(a->n_rows, a->batch, step, workspace);
  if (workspace_bytes < l.bytes) return SPEC_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  PromptAttnParams p;
  p.Hq = a->num_q_heads; p.Hkv = a->num_kv_heads; p.G = p.Hq / p.Hkv; p.tg = step / 2;
  p.scale_log2 = scale_of(a->scale, a->head_dim) * 1.4426950408889634f;
  p.head = p.scale_log2 > 1e-30f ? kPromptHead / p.scale_log2 : 0.f;  // (none where it might leave float32)
  p.v = static_cast<const uint16_t*>(a->v); p.v_stride = a->v_stride;
  p.out = static_cast<uint16_t*>(a->out); p.out32 = (reinterpret_cast<uintptr_t>(a->out) & 31u) == 0;
  p.lse = a->lse; p.dev_status = dev_status;
  CUtensorMap tm[3];
  if (a->n_rows > 0 &&
      (!make_map_heads(&tm[0], a->q, a->head_dim, p.Hq, a->n_rows, a->q_stride, p.G, p.tg) ||
       !make_map_heads(&tm[1], a->k, a->head_dim, p.Hkv, a->n_rows, a->k_stride, 1, 128) ||
       !make_map_heads(&tm[2], a->v, a->head_dim, p.Hkv, a->n_rows, a->v_stride, 1, 128)))
    return SPEC_ERR_CUDA;
  const spec_status ps = plan(a->n_rows, a->batch, step, 1, a->row_start, l, &p.plan, dev_status, stream);
  if (ps != SPEC_OK || a->n_rows == 0) return ps;
  const int grid = grid_for(plan_items(a->n_rows, a->batch, step), p.Hkv);
  return launch_prompt_attention(a->head_dim, &tm[0], &tm[1], &tm[2], p, grid, stream) == cudaSuccess ? SPEC_OK
                                                                                                      : SPEC_ERR_CUDA;
}

size_t spec_prompt_key_weights_workspace(const spec_key_weights_args* a) {
  if (check_key_weights(a) != SPEC_OK) return 0;
  return layout_plan(a->n_rows, a->batch, kWeightKeys, nullptr).bytes;
}

spec_status spec_prompt_key_weights(const spec_key_weights_args* a, void* workspace, size_t workspace_bytes,
                                    int32_t* dev_status, void* stream_ptr) {
  const spec_status st = check_key_weights(a);
  if (st != SPEC_OK) return st;
  if (!workspace || !aligned16(workspace)) return SPEC_ERR_INVALID_ARGUMENT;
  const PlanLayout l = layout_plan(a->n_rows, a->batch, kWeightKeys, workspace);
  if (workspace_bytes < l.bytes) return SPEC_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  KeyWeightsParams p;
  p.Hq = a->num_q_heads; p.Hkv = a->num_kv_heads; p.G = p.Hq / p.Hkv; p.tc = 128 / p.G; p.window = a->window;
  p.scale_log2 = scale_of(a->scale, a->head_dim) * 1.4426950408889634f;
  p.n_rows = a->n_rows; p.lse = a->lse; p.weight = a->weight; p.dev_status = dev_status;
  CUtensorMap tm[2];
  if (a->n_rows > 0 && (!make_map_heads(&tm[0], a->q, a->head_dim, p.Hq, a->n_rows, a->q_stride, p.G, p.tc) ||
                        !make_map_heads(&tm[1], a->k, a->head_dim, p.Hkv, a->n_rows, a->k_stride, 1, 128)))
    return SPEC_ERR_CUDA;
  const spec_status ps = plan(a->n_rows, a->batch, kWeightKeys, 0, a->row_start, l, &p.plan, dev_status, stream);
  if (ps != SPEC_OK || a->n_rows == 0) return ps;
  // Every head has as many CTAs of its own, where that idles an eighth of the SMs at most (8 prompts of 0.5K to 32K: 89.1 us,
  // 89.6 with shares over heads; one of 16K 13.2 and 14.2)
  int grid = grid_for(plan_items(a->n_rows, a->batch, kWeightKeys), p.Hkv);
  p.per_head = grid % p.Hkv * 8 <= grid ? grid / p.Hkv : 0;
  if (p.per_head) grid = p.per_head * p.Hkv;
  return launch_key_weights(a->head_dim, &tm[0], &tm[1], p, grid, stream) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

size_t spec_kv_keep_workspace(const spec_kv_keep_args* a) {
  if (check_keep(a) != SPEC_OK) return 0;
  return align_up(((size_t)a->rows_out * a->num_kv_heads + 1) * sizeof(int32_t));
}

spec_status spec_kv_keep(const spec_kv_keep_args* a, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                         void* stream) {
  const spec_status st = check_keep(a);
  if (st != SPEC_OK) return st;
  if (!workspace || !aligned16(workspace)) return SPEC_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < spec_kv_keep_workspace(a)) return SPEC_ERR_WORKSPACE_TOO_SMALL;
  const int size = a->dtype == SPEC_DTYPE_BF16 ? 2 : 4;
  KeepParams p;
  p.B = a->batch; p.Hkv = a->num_kv_heads; p.row_bytes = a->head_dim * size;
  p.budget = a->budget; p.first = a->first; p.last = a->last; p.n_rows = a->n_rows; p.rows_out = a->rows_out;
  p.k_stride = a->k_stride * size; p.v_stride = a->v_stride * size;
  p.k = static_cast<const uint8_t*>(a->k); p.v = static_cast<const uint8_t*>(a->v);
  p.weight = a->weight; p.row_start = a->row_start;
  p.k_out = static_cast<uint8_t*>(a->k_out); p.v_out = static_cast<uint8_t*>(a->v_out);
  p.index = a->index; p.keep_start = a->keep_start; p.n_keep = a->n_keep; p.dev_status = dev_status;
  return launch_kv_keep(p, static_cast<int32_t*>(workspace), num_sms_current(), static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

}  // extern "C"
