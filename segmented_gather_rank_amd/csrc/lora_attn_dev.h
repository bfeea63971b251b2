// lora_attn_dev.h -- device helpers shared by the attention kernels.
#pragma once

#include "lora_attn_host.h"
#include "lora_common.h"

namespace lora {

typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 *lds_i16x4_ptr;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The thread's index, opaque to the optimiser: what a work item derives from it is
// computed per item instead of being kept in registers across items (and across
// the variants of the item's code).
__device__ __forceinline__ int thread_of_item() {
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  return tid;
}

// Instruction kinds of __builtin_amdgcn_sched_group_barrier.
constexpr int kSchedMfma = 0x8, kSchedDsRead = 0x100;

// Maximum of three in one instruction; a NaN among them stays, so that no operand
// has to be quieted first, as fmaxf would.  Where a score is NaN its row's weights
// are too, whatever maximum they refer to.  The operands come from matrix products,
// whose results may be read only some cycles later: the compiler sees to that for
// operations it knows, not for an inline assembly statement.
__device__ __forceinline__ float max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}
// Maximum and sum over the lanes l and l ^ 32, and over l, l ^ 16, l ^ 32, l ^ 48:
// swapping a register's halves (rows of 16) with a copy of itself gives one
// register with each half's value everywhere.
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_rows(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum_rows(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return sum_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Four keys of one column: lane l of a 16-lane group gives the address of row
// l / 4, columns 4 (l % 4) .. + 3, and receives column l of the group's 4 rows.
__device__ __forceinline__ u32x2 lds_read_tr(const uint16_t *p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_ptr)(p)));
}

// Two e4m3 values (half of a 32-bit word) as a bf16 pair; exact.
__device__ __forceinline__ u32x4 e4m3x8_to_bf16(uint32_t lo, uint32_t hi) {
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
  return r;
}

// Whether any of 8 bf16 values is infinite or NaN.
__device__ __forceinline__ bool any_nonfinite(u32x4 v) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= (v[i] & 0x7f80u) == 0x7f80u || (v[i] & 0x7f800000u) == 0x7f800000u;
  return bad;
}

// A weight of zero does not hide an infinite or NaN value: 0 * inf = NaN would
// reach the rows that do not see the key.  Where a step has both hidden keys and
// such values its products with V run three times: with those values as zeros,
// and with 1 for a seen key against 1 for a +inf (-inf) value, NaN counting as
// both.  A positive count adds that infinity.
enum VPart { kVFinite = 0, kVPosInf = 1, kVNegInf = 2 };
__device__ __forceinline__ u32x4 v_part(u32x4 v, int part) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t x = (v[i] >> (16 * h)) & 0xffffu, mag = x & 0x7fffu;
      uint32_t y;
      if (part == kVFinite) y = mag >= 0x7f80u ? 0u : x;
      else if (part == kVPosInf) y = x == 0x7f80u || mag > 0x7f80u ? 0x3f80u : 0u;
      else y = x == 0xff80u || mag > 0x7f80u ? 0x3f80u : 0u;
      w |= y << (16 * h);
    }
    r[i] = w;
  }
  return r;
}
__device__ __forceinline__ float add_counted_infs(float o, float pos, float neg) {
  if (pos > 0.f) o += __builtin_inff();
  if (neg > 0.f) o -= __builtin_inff();
  return o;
}

// The running maximum that the weights refer to is only raised when a score
// exceeds it by more than 2^kSlack: the weights stay below 2^kSlack and their
// sum and O are exact up to that factor, while O, half of a wave's registers, is
// hardly ever rescaled.
constexpr float kSlack = 8.f;

// Scores to base-2 logits.  Plain: the factor alone.  General: cap * tanh(x / cap),
// then the distance bias.
struct ScoreArgs {
  float mul;        // scale * k_scale (general), times log2 e (plain)
  float cap, quarter_cap, over_cap, two_over_cap;  // over_cap = 1 / cap, two_over_cap = 2 log2(e) / cap
  float slope;      // of this lane's row
};
// cap * tanh(x / cap) with y = x / cap.  Below 1/4 the series of tanh in y, off by less
// than 1e-8 of x, since the other form loses what is small against the cap: tanh(y) =
// 1 - 2 / (exp(2y) + 1), off by about 3e-7.
__device__ __forceinline__ float cap_small(const ScoreArgs &s, float x) {
  const float y = x * s.over_cap, z = y * y;
  float p = __builtin_fmaf(z, 62.f / 2835.f, -17.f / 315.f);
  p = __builtin_fmaf(z, p, 2.f / 15.f);
  p = __builtin_fmaf(z, p, -1.f / 3.f);
  return __builtin_fmaf(x * z, p, x);
}
__device__ __forceinline__ float cap_large(const ScoreArgs &s, float x) {
  return s.cap * __builtin_fmaf(-2.f, __builtin_amdgcn_rcpf(exp2_fast(x * s.two_over_cap) + 1.f), 1.f);
}
// The scores of a lane capped.  Most batches of them need the series alone, which has
// no exponential and no reciprocal.  A prompt of 4096 tokens (32 / 8 heads of 128) takes
// 258 us with a cap that few scores come near, 307 where most pass a quarter of it (235
// and 226 with the exponential alone, which is wrong for large caps); decode is bound by
// HBM all the same.
template <int N, typename V>
__device__ __forceinline__ void cap_scores(const ScoreArgs &s, V &st) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 2) top = max3(top, fabsf(st[i]), fabsf(st[i + 1]));
  if (__any(!(top < s.quarter_cap))) {
#pragma unroll
    for (int i = 0; i < N; ++i) st[i] = fabsf(st[i]) < s.quarter_cap ? cap_small(s, st[i]) : cap_large(s, st[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) st[i] = cap_small(s, st[i]);
  }
}
// N matrix products of a lane to general logits; distance(i) is of the i-th.
template <int N, typename V, typename F>
__device__ __forceinline__ void general_logits(const ScoreArgs &s, V &st, F &&distance) {
#pragma unroll
  for (int i = 0; i < N; ++i) st[i] *= s.mul;
  if (s.cap > 0.f) cap_scores<N>(s, st);
#pragma unroll
  for (int i = 0; i < N; ++i) st[i] = (st[i] - s.slope * fabsf((float)distance(i))) * kLog2e;
}
template <bool GENERAL>
__device__ __forceinline__ ScoreArgs score_args(const AttnArgs &a, int kvh, int q_head) {
  ScoreArgs s;
  const float ks = a.cache.k_scale ? a.cache.k_scale[kvh] : 1.f;
  s.mul = a.scale * ks * (GENERAL ? 1.f : kLog2e);
  s.cap = a.cap;
  s.quarter_cap = 0.25f * a.cap;
  // (finite for the smallest caps too: 0 * inf would be NaN)
  s.over_cap = GENERAL && a.cap > 0.f ? fminf(1.f / a.cap, 3e38f) : 0.f;
  s.two_over_cap = GENERAL && a.cap > 0.f ? fminf(2.f * kLog2e / a.cap, 3e38f) : 0.f;
  s.slope = GENERAL && a.slopes ? a.slopes[q_head] : 0.f;
  return s;
}

__device__ __forceinline__ AttnItem load_item(const int32_t *items, int i) {
  // uniform index: scalar loads
  const int32_t *p = items + (int64_t)i * kAttnItemInts;
  return AttnItem{p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7]};
}

// Row `row` (of kUnitRows) of partial-result unit `unit`, head group h.  A head
// group's units lie together: the parts of a row are close in memory (one after
// the other for a decode token), which spares address translations.
__device__ __forceinline__ int64_t part_row(const AttnArgs &a, int64_t unit, int h, int row) {
  return (h * a.max_units + unit) * kUnitRows + row;
}

}  // namespace lora
