// lora_base_host.h -- argument blocks and launchers of the base side's kernels
// (routing, row quantisation, 8-bit products, weighted sum), shared by their
// translation units.  Internal to the library.
#pragma once

#include "lora_host.h"

namespace lora {

constexpr int kMaxTopk = 32;     // choices of a token in lora_moe_route
constexpr int kMaxGroups = 64;

struct RouteArgs {
  const char *logits;
  int64_t ld, tokens;
  const float *bias;
  int32_t *ids;
  float *weights;
  float scale;
  int32_t experts, topk, sigmoid, groups, kept, group_top, renorm, aligned;
  int32_t group_lanes;           // set by the launcher: lanes of a group, 0 where groups are not whole lanes
};
hipError_t launch_route(const RouteArgs &a, bool bf16, hipStream_t s);

struct QuantArgs {
  const char *x;
  int8_t *q;
  float *scale;
  char *act;                     // or NULL
  const int32_t *sorted, *sorted_slot;  // NULL: every row
  int64_t ldx, ldq, ldact, rows;
  int32_t width, gated;
};
hipError_t launch_quantize(const QuantArgs &a, bool bf16, hipStream_t s);

struct Int8Args {
  const int8_t *x, *w;
  const float *x_scale, *w_scale, *bias;
  char *y;
  int64_t ldx, ldy, rows;
  int64_t expert_stride, row_stride;
  int32_t d_in, d_out, experts;
  MetaView meta;                 // sorted == NULL: dense
};
hipError_t launch_int8(const Int8Args &a, bool bf16, hipStream_t s);
// Rows in tiles of 64; with metadata, the segments of fewest .. most rows.
hipError_t launch_int8_mid(const Int8Args &a, bool bf16, int fewest, int most, hipStream_t s);
// Rows in tiles of 256; with metadata, the segments of at least `fewest` rows.
hipError_t launch_int8_tile(const Int8Args &a, bool bf16, int fewest, hipStream_t s);

struct CombineArgs {
  const char *y, *add;           // add: NULL or rows
  char *out;
  const int32_t *ids, *map;
  const float *weights;
  int64_t ldy, ldadd, ldout, tokens;
  int32_t width, topk, experts, local;
};
hipError_t launch_combine(const CombineArgs &a, bool bf16, hipStream_t s);

}  // namespace lora
