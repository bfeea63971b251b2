// lora_base_abi.hip -- the extern "C" entry points of the base side declared in
// include/lora_mi355x.h: expert routing, row quantisation, 8-bit products, weighted sum.
// Every check that can fail runs before the first HIP call.
#include "../../include/lora_mi355x.h"
#include "lora_base_host.h"

namespace lora {

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
bool dtype_ok(lora_dtype d) { return d == LORA_F32 || d == LORA_BF16; }
lora_status launched(hipError_t e) { return e == hipSuccess ? LORA_OK : LORA_ERR_HIP; }

lora_status check_meta(const lora_meta *m) {
  if (m->num_tokens < 0 || m->num_slots < 1 || m->num_slots > kMaxSlots || m->x_row_div < 1) return LORA_ERR_INVALID_ARG;
  if (!m->sorted || !m->sorted_slot || !m->seg_slot || !m->seg_count || !m->seg_start || !m->info || !m->tiles)
    return LORA_ERR_INVALID_ARG;
  return LORA_OK;
}

constexpr int64_t kMaxRows = (int64_t)1 << 24;
constexpr int64_t kMaxWidth = (int64_t)1 << 24;
constexpr int64_t kMaxDepth = 131056;  // products of -128 with -128: 16384 each, below 2^31 in all

lora_status check_weight(const lora_int8_weight *w) {
  if (!w || w->reserved != 0 || !w->ptr || !aligned16(w->ptr) || !w->scale || !aligned4(w->scale) || !aligned4(w->bias))
    return LORA_ERR_INVALID_ARG;
  if (w->num_experts < 1 || w->d_in < 16 || w->d_in % 16 || w->d_out < 8 || w->d_out % 8) return LORA_ERR_INVALID_ARG;
  if (w->row_stride % 16 || w->row_stride < w->d_in || w->expert_stride % 16) return LORA_ERR_INVALID_ARG;
  if (w->num_experts > kMaxSlots || w->d_in > kMaxDepth || w->d_out > kMaxWidth || w->row_stride >= (1 << 23))
    return LORA_ERR_UNSUPPORTED;
  if (w->num_experts > 1) {
    // matrices that do not overlap: one after the other, or side by side in longer rows
    const bool apart = w->expert_stride >= (w->d_out - 1) * w->row_stride + w->d_in;
    const bool beside = !apart && w->expert_stride >= w->d_in && w->row_stride >= (w->num_experts - 1) * w->expert_stride + w->d_in;
    if (!apart && !beside) return LORA_ERR_INVALID_ARG;
  }
  return LORA_OK;
}

}  // namespace

}  // namespace lora

using namespace lora;

extern "C" {

lora_status lora_moe_route(const lora_routing *r, const void *d_logits, int64_t ld, int64_t num_tokens,
                           lora_dtype dtype, int32_t *d_topk_ids, float *d_weights, void *stream) {
  if (!r || num_tokens < 0) return LORA_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || (r->score != LORA_SCORE_SOFTMAX && r->score != LORA_SCORE_SIGMOID)) return LORA_ERR_UNSUPPORTED;
  if (r->num_experts < 1 || r->topk < 1 || r->num_groups < 1) return LORA_ERR_INVALID_ARG;
  if (r->num_experts > 1024 || r->topk > kMaxTopk || r->num_groups > kMaxGroups) return LORA_ERR_UNSUPPORTED;
  if (r->num_experts % r->num_groups) return LORA_ERR_INVALID_ARG;
  const int32_t size = r->num_experts / r->num_groups;
  int32_t kept = 1;
  if (r->num_groups > 1) {
    kept = r->topk_groups;
    if (kept < 1 || kept > r->num_groups || r->group_top < 1 || r->group_top > 2 || r->group_top > size)
      return LORA_ERR_INVALID_ARG;
  }
  if (r->topk > kept * size || ld < r->num_experts || !aligned4(r->d_bias)) return LORA_ERR_INVALID_ARG;
  if (num_tokens == 0) return LORA_OK;
  const int64_t esize = dtype == LORA_F32 ? 4 : 2;
  if (!d_logits || reinterpret_cast<uintptr_t>(d_logits) % esize || !d_topk_ids || !aligned4(d_topk_ids) || !d_weights ||
      !aligned4(d_weights))
    return LORA_ERR_INVALID_ARG;
  RouteArgs a{};
  a.logits = static_cast<const char *>(d_logits);
  a.ld = ld;
  a.tokens = num_tokens;
  a.bias = r->d_bias;
  a.ids = d_topk_ids;
  a.weights = d_weights;
  a.scale = r->scale;
  a.experts = r->num_experts;
  a.topk = r->topk;
  a.sigmoid = r->score == LORA_SCORE_SIGMOID;
  // groups that all stay are no groups
  a.groups = kept < r->num_groups ? r->num_groups : 1;
  a.kept = kept;
  a.group_top = r->group_top;
  a.renorm = r->renormalize != 0;
  a.aligned = aligned16(d_logits) && ld * esize % 16 == 0;
  return launched(launch_route(a, dtype == LORA_BF16, static_cast<hipStream_t>(stream)));
}

lora_status lora_quantize(const void *d_x, int64_t ldx, int64_t num_rows, int64_t width, lora_dtype dtype,
                          lora_activation activation, const lora_meta *meta, int8_t *d_q, int64_t ldq, float *d_scale,
                          void *d_act, int64_t ldact, void *stream) {
  if (!dtype_ok(dtype) || (activation != LORA_ACT_NONE && activation != LORA_ACT_SILU_MUL)) return LORA_ERR_UNSUPPORTED;
  if (num_rows < 0 || width < 16 || width % 16 || (d_act && activation == LORA_ACT_NONE)) return LORA_ERR_INVALID_ARG;
  if (num_rows > kMaxRows * 64 || width > kMaxWidth) return LORA_ERR_UNSUPPORTED;
  const int64_t in = activation == LORA_ACT_SILU_MUL ? 2 * width : width;
  if (ldx < in || ldx % 8 || ldq < width || ldq % 16 || (d_act && (ldact < width || ldact % 8))) return LORA_ERR_INVALID_ARG;
  if (meta) {
    const lora_status st = check_meta(meta);
    if (st != LORA_OK) return st;
    if (meta->num_tokens != num_rows || meta->x_row_div != 1) return LORA_ERR_INVALID_ARG;
  }
  if (!aligned16(d_x) || !aligned16(d_q) || !aligned4(d_scale) || !aligned16(d_act)) return LORA_ERR_INVALID_ARG;
  if (num_rows == 0) return LORA_OK;
  if (!d_x || !d_q || !d_scale) return LORA_ERR_INVALID_ARG;
  QuantArgs a{};
  a.x = static_cast<const char *>(d_x);
  a.q = d_q;
  a.scale = d_scale;
  a.act = static_cast<char *>(d_act);
  if (meta) {
    a.sorted = meta->sorted;
    a.sorted_slot = meta->sorted_slot;
  }
  a.ldx = ldx;
  a.ldq = ldq;
  a.ldact = ldact;
  a.rows = num_rows;
  a.width = (int32_t)width;
  a.gated = activation == LORA_ACT_SILU_MUL;
  return launched(launch_quantize(a, dtype == LORA_BF16, static_cast<hipStream_t>(stream)));
}

lora_status lora_int8_matmul_workspace_bytes(int64_t num_rows, const lora_int8_weight *w, size_t *bytes) {
  if (!bytes || num_rows < 0) return LORA_ERR_INVALID_ARG;
  const lora_status st = check_weight(w);
  if (st != LORA_OK) return st;
  if (num_rows > kMaxRows) return LORA_ERR_UNSUPPORTED;
  *bytes = 0;
  return LORA_OK;
}

lora_status lora_int8_matmul(const lora_meta *meta, const int8_t *d_x, int64_t ldx, const float *d_x_scale,
                             int64_t num_rows, const lora_int8_weight *w, void *d_y, int64_t ldy, lora_dtype dtype,
                             void *, size_t, void *stream) {  // no form needs a workspace
  size_t need = 0;
  lora_status st = lora_int8_matmul_workspace_bytes(num_rows, w, &need);
  if (st != LORA_OK) return st;
  if (!dtype_ok(dtype)) return LORA_ERR_UNSUPPORTED;
  if (ldx < w->d_in || ldx % 16 || ldy < w->d_out || ldy % 8 || !aligned16(d_x) || !aligned16(d_y) || !aligned4(d_x_scale))
    return LORA_ERR_INVALID_ARG;
  if (meta) {
    st = check_meta(meta);
    if (st != LORA_OK) return st;
    if (meta->num_tokens != num_rows || meta->num_slots != w->num_experts) return LORA_ERR_INVALID_ARG;
  } else if (w->num_experts != 1) {
    return LORA_ERR_INVALID_ARG;
  }
  if (num_rows == 0) return LORA_OK;
  if (!d_x || !d_x_scale || !d_y) return LORA_ERR_INVALID_ARG;
  Int8Args a{};
  a.x = d_x;
  a.w = w->ptr;
  a.x_scale = d_x_scale;
  a.w_scale = w->scale;
  a.bias = w->bias;
  a.y = static_cast<char *>(d_y);
  a.ldx = ldx;
  a.ldy = ldy;
  a.rows = num_rows;
  a.expert_stride = w->expert_stride;
  a.row_stride = w->row_stride;
  a.d_in = (int32_t)w->d_in;
  a.d_out = (int32_t)w->d_out;
  a.experts = w->num_experts;
  if (meta) {
    a.meta.sorted = meta->sorted;
    a.meta.sorted_slot = meta->sorted_slot;
    a.meta.seg_slot = meta->seg_slot;
    a.meta.seg_count = meta->seg_count;
    a.meta.seg_start = meta->seg_start;
    a.meta.info = meta->info;
    a.meta.tiles = meta->tiles;
    a.meta.T = meta->num_tokens;
    a.meta.S = meta->num_slots;
    a.meta.x_row_div = meta->x_row_div;
  }
  return launched(launch_int8(a, dtype == LORA_BF16, static_cast<hipStream_t>(stream)));
}

lora_status lora_moe_combine(const void *d_y, int64_t ldy, int64_t width, lora_dtype dtype, const int32_t *d_topk_ids,
                             const float *d_weights, int64_t num_tokens, int32_t topk, int32_t num_experts,
                             int32_t num_local_experts, const int32_t *d_expert_map, const void *d_add, int64_t ldadd,
                             void *d_out, int64_t ldout, void *stream) {
  if (!dtype_ok(dtype)) return LORA_ERR_UNSUPPORTED;
  if (num_tokens < 0 || topk < 1 || num_experts < 1 || num_local_experts < 1 || width < 8 || width % 8)
    return LORA_ERR_INVALID_ARG;
  if (topk > 64 || width > kMaxWidth || num_tokens > kMaxRows) return LORA_ERR_UNSUPPORTED;
  if (ldy < width || ldy % 8 || ldout < width || ldout % 8 || (d_add && (ldadd < width || ldadd % 8)))
    return LORA_ERR_INVALID_ARG;
  if (!aligned16(d_y) || !aligned16(d_add) || !aligned16(d_out) || !aligned4(d_topk_ids) || !aligned4(d_weights) ||
      !aligned4(d_expert_map))
    return LORA_ERR_INVALID_ARG;
  // in place means the same rows: any other stride would read rows that are written
  if (d_add == d_out && d_add && ldadd != ldout) return LORA_ERR_INVALID_ARG;
  if (num_tokens == 0) return LORA_OK;
  if (!d_y || !d_topk_ids || !d_weights || !d_out) return LORA_ERR_INVALID_ARG;
  CombineArgs a{};
  a.y = static_cast<const char *>(d_y);
  a.add = static_cast<const char *>(d_add);
  a.out = static_cast<char *>(d_out);
  a.ids = d_topk_ids;
  a.map = d_expert_map;
  a.weights = d_weights;
  a.ldy = ldy;
  a.ldadd = ldadd;
  a.ldout = ldout;
  a.tokens = num_tokens;
  a.width = (int32_t)width;
  a.topk = topk;
  a.experts = num_experts;
  a.local = num_local_experts;
  return launched(launch_combine(a, dtype == LORA_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
