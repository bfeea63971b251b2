// lora_int8.hip -- products of 8-bit rows and weights, with a scale for each token and
// channel: the base product of a dense layer, or of a MoE layer's experts.
//
// The sum over d_in is exact in 32-bit integers (v_mfma_i32_16x16x64_i8), so neither the
// order nor a split of it changes a result.  The weight's rows are the first operand, so
// that a lane ends with four neighbouring outputs of one row of x.
//
// few_kernel: a workgroup takes 16 NT output columns of up to 64 rows at a time and its
// waves take d_in in turn, 128 bytes of every row a step, straight from memory to the
// matrix cores' registers (few rows use a weight once, there is nothing to share); the
// waves' sums meet in LDS.  Bound: HBM reads of the weights.  The experts of a decode step
// (256 tokens, an eighth of their 8 choices of 256 here, 7168 x 4096 each): 165 us a call,
// 5.4 TB/s; one row x 4096 x 4096: 5.4 us, 3.1 TB/s, the chain of loads, sums and barrier.
// Dense batches x 4096 x 6144: 1 row 8 us, 16 rows 11, 32 rows 14, and 64 rows 21, as beyond
// 32 rows registers let a wave load one step ahead only.  Loads by buffer take 32-bit
// offsets, which leaves registers for two workgroups a CU (by address 183 us).  Segments of
// a workgroup's own number that others take cost a workgroup that ends at once, 2 ns each;
// a workgroup for four segments ends them sooner, but evens the load of a decode step out
// less (181 us for 165).
#include <algorithm>

#include "lora_base_host.h"

namespace lora {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;  // bytes of d_in a step takes: two matrix instructions

// The rows that a workgroup works on: a segment of the metadata, or all.
struct Rows {
  const int32_t *sorted;  // NULL: row i is i
  int count, expert;
  uint32_t div;
  __device__ __forceinline__ int64_t at(int i) const { return sorted ? sorted[i] : i; }
  __device__ __forceinline__ int64_t x_row(int64_t row) const { return div == 1 ? row : (int64_t)((uint32_t)row / div); }
};

// Segment `i` of the metadata; count 0 where there is none, or it is the rows' without a key.
__device__ __forceinline__ Rows segment(const Int8Args &a, int i) {
  const int n = a.meta.info[0], slot = a.meta.seg_slot[i], count = a.meta.seg_count[i], start = a.meta.seg_start[i];
  return Rows{a.meta.sorted + start, i < n && slot >= 0 ? count : 0, slot, (uint32_t)a.meta.x_row_div};
}

// y of 4 neighbouring columns of one row
template <typename Y>
__device__ __forceinline__ void store4(char *y, int64_t at, const float v[4]) {
  if constexpr (sizeof(Y) == 2) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    typedef __attribute__((address_space(1))) u32x2 g_u32x2;
    *(g_u32x2 *)(y + 2 * at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  } else {
    gstore16f(y + 4 * at, f32x4{v[0], v[1], v[2], v[3]});
  }
}

__device__ __forceinline__ i32x4 product(u32x4 w, u32x4 x, i32x4 sum) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), sum, 0, 0, 0);
}

// An offset past the end of every buffer: a load from there gives zeros.
constexpr uint32_t kNowhere = 0xffffffffu;

// Where a lane reads a row of x from: 32 bits from x's start, or an address where x is
// larger than that.
template <bool WIDE> struct XRow;
template <> struct XRow<false> {
  uint32_t at;
  __device__ __forceinline__ void aim(const int8_t *, int64_t offset) { at = (uint32_t)offset; }
  __device__ __forceinline__ u32x4 load(rsrc_t x, int k, bool in) const {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(x, (int)(in ? at : kNowhere), k, 0));
  }
};
template <> struct XRow<true> {
  const int8_t *at;
  __device__ __forceinline__ void aim(const int8_t *x, int64_t offset) { at = x + offset; }
  __device__ __forceinline__ u32x4 load(rsrc_t, int k, bool in) const { return in ? gload16(at + k) : u32x4{0, 0, 0, 0}; }
};

// Output columns n0 .. n0 + 16 NT - 1 of rows r0 .. r0 + 16 MT - 1.
template <typename Y, bool WIDE, int MT, int NT, int WAVES, int AHEAD>
__device__ __forceinline__ void few_block(const Int8Args &a, const Rows &rows, int r0, int n0, i32x4 *lds) {
  static_assert(MT * NT <= WAVES, "a wave adds up one block");
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int l16 = lane % 16, quarter = lane / 16;
  // past the last row and column: the last one again, not stored
  int64_t row[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) row[m] = rows.at(min(r0 + 16 * m + l16, rows.count - 1));
  const rsrc_t w = make_rsrc(a.w + rows.expert * a.expert_stride + n0 * a.row_stride, kNowhere - 1);
  const rsrc_t x = make_rsrc(a.x, kNowhere - 1);
  uint32_t wo[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    wo[n] = (uint32_t)min(16 * n + l16, a.d_out - 1 - n0) * (uint32_t)a.row_stride + 16 * quarter;
  XRow<WIDE> xo[MT];

  i32x4 sum[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) sum[m][n] = i32x4{0, 0, 0, 0};

  u32x4 wv[AHEAD][NT][2], xv[AHEAD][MT][2];
  // a step's bytes of the weights, and of x; pieces past the end of d_in are zeros
  auto load_w = [&](int d, int step) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = step * kStep + 64 * h;
      const bool in = k + 16 * quarter < a.d_in;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        wv[d][n][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(w, (int)(in ? wo[n] : kNowhere), k, 0));
    }
  };
  auto load_x = [&](int d, int step) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = step * kStep + 64 * h;
      const bool in = k + 16 * quarter < a.d_in;
#pragma unroll
      for (int m = 0; m < MT; ++m) xv[d][m][h] = xo[m].load(x, k, in);
    }
  };
  auto multiply = [&](int d) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) sum[m][n] = product(wv[d][n][h], xv[d][m][h], sum[m][n]);
  };
  const int steps = (a.d_in + kStep - 1) / kStep;
#pragma unroll
  for (int d = 0; d < AHEAD; ++d)
    if (wave + d * WAVES < steps) load_w(d, wave + d * WAVES);
  int64_t from[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    from[m] = rows.x_row(row[m]);
    xo[m].aim(a.x, from[m] * a.ldx + 16 * quarter);
  }
#pragma unroll
  for (int d = 0; d < AHEAD; ++d)
    if (wave + d * WAVES < steps) load_x(d, wave + d * WAVES);
  for (int s = wave; s < steps; s += AHEAD * WAVES) {
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) {
      if (s + d * WAVES < steps) multiply(d);
      if (s + (d + AHEAD) * WAVES < steps) {
        load_w(d, s + (d + AHEAD) * WAVES);
        load_x(d, s + (d + AHEAD) * WAVES);
      }
    }
  }

  // the waves' sums together: wave b adds up block b
  __syncthreads();  // what the workgroup's block before this one left is read
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) lds[((m * NT + n) * WAVES + wave) * 64 + lane] = sum[m][n];
  __syncthreads();
  if (wave >= MT * NT) return;
  const int m = wave / NT, n = wave % NT;
  const int r = r0 + 16 * m + l16, c = n0 + 16 * n + 4 * quarter;
  if (r >= rows.count || c >= a.d_out) return;
  const int64_t en = (int64_t)rows.expert * a.d_out + c;
  const int64_t to = rows.at(r);
  f32x4 ws, bs = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    ws[e] = a.w_scale[en + e];
    if (a.bias) bs[e] = a.bias[en + e];
  }
  const float xs = a.x_scale[rows.x_row(to)];
  i32x4 t = lds[wave * WAVES * 64 + lane];
#pragma unroll
  for (int o = 1; o < WAVES; ++o) t += lds[(wave * WAVES + o) * 64 + lane];
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = (float)t[e] * (xs * ws[e]) + bs[e];
  store4<Y>(a.y, to * a.ldy + c, v);
}

template <typename Y, bool WIDE, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 4) void few_kernel(Int8Args a, int group0, bool all) {
  __shared__ i32x4 lds[4 * NT * WAVES * 64];
  const int n0 = blockIdx.x * 16 * NT;
  Rows rows{nullptr, (int)a.rows, 0, 1};
  int r0 = 0, end = rows.count;
  if (a.meta.sorted) {
    rows = segment(a, group0 + blockIdx.y);
    end = all || rows.count <= ExpertRule(a.meta, a.d_out).few ? rows.count : 0;
  } else {
    r0 = (group0 + blockIdx.y) * 64;
    end = min(end, r0 + 64);
  }
  for (; r0 < end; r0 += 64) {
    if (end - r0 <= 16) few_block<Y, WIDE, 1, NT, WAVES, 4>(a, rows, r0, n0, lds);
    else if (end - r0 <= 32) few_block<Y, WIDE, 2, NT, WAVES, 2>(a, rows, r0, n0, lds);
    else few_block<Y, WIDE, 4, NT, WAVES, 1>(a, rows, r0, n0, lds);
  }
}

// With metadata, all segments or those of few rows.
template <typename Y, bool WIDE, int NT>
hipError_t launch_few(const Int8Args &a, bool all, hipStream_t s) {
  constexpr int kWaves = 8;
  const int64_t groups = a.meta.sorted ? std::min<int64_t>(a.rows, a.experts) + 1 : (a.rows + 63) / 64;
  const int64_t cols = (a.d_out + 16 * NT - 1) / (16 * NT);
  // a launch holds fewer than 2^32 threads, and 2^16 rows of its grid
  const int64_t rows = std::max<int64_t>(1, std::min<int64_t>(32768, ((int64_t)1 << 22) / cols));
  for (int64_t g0 = 0; g0 < groups; g0 += rows) {
    const dim3 grid((unsigned)cols, (unsigned)std::min(groups - g0, rows));
    few_kernel<Y, WIDE, NT, kWaves><<<grid, dim3(64 * kWaves), 0, s>>>(a, (int)g0, all);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <typename Y>
hipError_t launch_few(const Int8Args &a, bool all, bool wide, hipStream_t s) {
  if (wide) return launch_few<Y, true, 2>(a, all, s);
  // 16 columns a workgroup where 32 would leave CUs without one
  const int64_t groups = a.meta.sorted ? std::min<int64_t>(a.rows, a.experts) : (a.rows + 63) / 64;
  if (groups * a.d_out < 512 * 32) return launch_few<Y, false, 1>(a, all, s);
  return launch_few<Y, false, 2>(a, all, s);
}

}  // namespace

hipError_t launch_int8(const Int8Args &a, bool bf16, hipStream_t s) {
  // x is addressed in 32 bits: all of it, or in tiles of a dense batch their 256 rows.  Where that does not reach,
  // few_kernel takes all, 64 rows of a segment after the other, in the time of that.
  const int64_t x_rows = a.meta.sorted ? (a.rows - 1) / a.meta.x_row_div + 1 : a.rows;
  const bool wide = x_rows * a.ldx >= ((int64_t)1 << 32) - 256;
  const bool tiles = a.meta.sorted ? !wide : 256 * a.ldx < ((int64_t)1 << 32) - 256;
  if (!tiles || a.meta.sorted || a.rows <= kFewRows) {
    const hipError_t err = bf16 ? launch_few<uint16_t>(a, !tiles, wide, s) : launch_few<float>(a, !tiles, wide, s);
    if (err != hipSuccess || !tiles || a.rows <= 16 || (!a.meta.sorted && a.rows <= kFewRows)) return err;
  }
  // A dense batch of up to three workgroups a CU takes tiles of 64 x 64, more take larger ones:
  // 256 rows x 4096 x 6144 (384 tiles) 16.5 us here, 22.7 in tiles of 128; 512 x 4096 x 28672 (3584) 116 and 64.
  const int64_t tiles64 = (a.rows + 63) / 64 * ((a.d_out + 63) / 64);
  return !a.meta.sorted && tiles64 <= 768 ? launch_int8_mid(a, bf16, s) : launch_int8_tile(a, bf16, s);
}

}  // namespace lora
