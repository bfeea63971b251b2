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
// A dense batch in tiles of 64 rows.
hipError_t launch_int8_mid(const Int8Args &a, bool bf16, hipStream_t s);
// A dense batch in tiles of 128 or 256 rows; by expert, the segments that are not few_kernel's, in either.
hipError_t launch_int8_tile(const Int8Args &a, bool bf16, hipStream_t s);

// By expert, rows decide who takes a segment, and only the device knows them.  Every kernel
// that may be the one asks the same rule, whose answers follow from the metadata's counts:
//   few   most rows of a segment that few_kernel takes: 64 in a decode step (16 rows a
//         segment or fewer on average), 128 where tiles would not fill the chip: it splits
//         d_in over a workgroup's waves, which answers soonest; else 16
//   large whether the others take tiles of 256, else of 128: from 160 rows a segment on.
//         (Long and short segments in tiles of their own, one kernel after the other, are
//         slower than either for all: 113 rows a segment on average 178 us for 165, all in
//         tiles of 256: 169; 226 rows 240 us for 207.  Between 113 and 226 rows, and with
//         counts more uneven than a normal router's, nothing was timed.)
constexpr int kFewRows = 64;
struct ExpertRule {
  int few;
  bool large;
  __device__ __forceinline__ ExpertRule(const MetaView &m, int d_out) {
    const int none = m.info[3];                   // rows without a key come first, as a segment of their own
    const int64_t segments = m.info[0] - (none > 0), rows = m.T - none;
    few = rows <= 16 * segments ? kFewRows : segments * ((d_out + 127) / 128) >= 512 ? 16 : 2 * kFewRows;
    large = rows > 160 * segments;
  }
};

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
