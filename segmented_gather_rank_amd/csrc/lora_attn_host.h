// lora_attn_host.h -- argument blocks and launchers of the attention and append
// kernels, shared by their translation units.  Internal to the library.
#pragma once

#include <hip/hip_runtime.h>

#include "lora_attn_plan.h"

namespace lora {

hipError_t launch_attn_plan(const AttnPlanArgs &a, hipStream_t s);

struct AttnArgs {
  CacheView cache;
  const char *q;
  char *out;
  float *lse;                // [T][q_heads] or NULL
  const float *slopes;       // [q_heads] or NULL
  const int32_t *limits, *info, *few_items, *slots, *tile_items, *join_list;
  int64_t ldq, ldo, tokens;  // elements
  int64_t max_units;
  float *part;               // partial results: see part_row
  float *part_ml;
  float scale, cap;
  int32_t heads, group, q_heads, dim;
  Divisor by_heads, by_group, by_q_heads, by_kv_parts;  // kv_parts: head groups per key head
  int32_t few_waves, tile_blocks;  // slices times head groups, workgroups of tile items (0: few rows only)
};

// Kind of the cache's elements (and with it of q and out).
enum AttnKind { kAttnBf16 = 0, kAttnE4m3 = 1, kAttnF32 = 2 };

hipError_t launch_attn(const AttnArgs &a, AttnKind kind, hipStream_t s);
hipError_t launch_attn_join(const AttnArgs &a, AttnKind kind, hipStream_t s);

struct AppendArgs {
  const char *x;
  char *q, *k, *v;
  int64_t ldx, ldq, tokens;        // elements
  int64_t off_q, off_k, off_v;     // columns
  int64_t page_stride, head_stride, pos_stride;  // elements
  int64_t num_slots;
  const int64_t *slot;
  const int32_t *pos;
  const float *table;
  int64_t num_pos;
  const float *k_scale, *v_scale;
  int32_t *num_bad;
  int32_t q_heads, kv_heads, dim, page_size, half, axes, interleaved;
  int32_t axis_end[4];
  Divisor units[3];                // units per head: turned, copied, v
  Divisor by_page;
};
hipError_t launch_append(const AppendArgs &a, AttnKind kind, hipStream_t s);

}  // namespace lora
