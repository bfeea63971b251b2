// lora_int8.hip -- products of 8-bit rows and weights, with a scale for each token and
// channel: the base product of a dense layer, or of a MoE layer's experts.
//
// The sum over d_in is exact in 32-bit integers (v_mfma_i32_16x16x64_i8), so neither the
// order nor a split of it changes a result.  The weight's rows are the first operand, so
// that a lane ends with four neighbouring outputs of one row of x.
//
// few_kernel: a workgroup takes 16 NT output columns of up to 64 rows at a time and its
// waves take d_in in turn, 128 bytes of every row a step, straight from memory to the
// matrix cores' registers (few rows use a weight once, there is nothing to share).
#include <algorithm>

#include "lora_base_host.h"

namespace lora {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kFewRows = 64;  // most rows of a segment (or a dense batch) that few_kernel takes
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

// Output columns n0 .. n0 + 16 NT - 1 of rows r0 .. r0 + 16 MT - 1.
template <typename Y, int MT, int NT, int WAVES, int AHEAD>
__device__ __forceinline__ void few_block(const Int8Args &a, const Rows &rows, int r0, int n0, i32x4 *lds) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, l16 = lane % 16, quarter = lane / 16;
  // past the last row and column: the last one again, not stored
  const int8_t *wp[NT], *xp[MT];
  const int8_t *w = a.w + (int64_t)rows.expert * a.expert_stride + 16 * quarter;
#pragma unroll
  for (int n = 0; n < NT; ++n) wp[n] = w + (int64_t)min(n0 + 16 * n + l16, a.d_out - 1) * a.row_stride;
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xp[m] = a.x + rows.x_row(rows.at(min(r0 + 16 * m + l16, rows.count - 1))) * a.ldx + 16 * quarter;

  i32x4 sum[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) sum[m][n] = i32x4{0, 0, 0, 0};

  u32x4 wv[AHEAD][NT][2], xv[AHEAD][MT][2];
  auto load = [&](int d, int step) {
    const int k = step * kStep;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int n = 0; n < NT; ++n) wv[d][n][h] = gload16(wp[n] + k + 64 * h);
#pragma unroll
      for (int m = 0; m < MT; ++m) xv[d][m][h] = gload16(xp[m] + k + 64 * h);
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
  const int steps = a.d_in / kStep;
#pragma unroll
  for (int d = 0; d < AHEAD; ++d)
    if (wave + d * WAVES < steps) load(d, wave + d * WAVES);
  for (int s = wave; s < steps; s += AHEAD * WAVES) {
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) {
      if (s + d * WAVES < steps) multiply(d);
      if (s + (d + AHEAD) * WAVES < steps) load(d, s + (d + AHEAD) * WAVES);
    }
  }
  // the last bytes of d_in, a multiple of 16: pieces past the end are zeros
  if (a.d_in % kStep && wave == steps % WAVES) {
    const int k = steps * kStep;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = k + 64 * h + 16 * quarter < a.d_in;
      const u32x4 none = {0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < NT; ++n) wv[0][n][h] = in ? gload16(wp[n] + k + 64 * h) : none;
#pragma unroll
      for (int m = 0; m < MT; ++m) xv[0][m][h] = in ? gload16(xp[m] + k + 64 * h) : none;
    }
    multiply(0);
  }

  // the waves' sums together: wave w adds up the blocks w, w + WAVES, ...
  __syncthreads();  // what the workgroup's block before this one left is read
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) lds[((m * NT + n) * WAVES + wave) * 64 + lane] = sum[m][n];
  __syncthreads();
#pragma unroll
  for (int b = 0; b < MT * NT; ++b) {
    if (b % WAVES != wave) continue;
    const int m = b / NT, n = b % NT;
    i32x4 t = lds[b * WAVES * 64 + lane];
#pragma unroll
    for (int o = 1; o < WAVES; ++o) t += lds[(b * WAVES + o) * 64 + lane];
    const int r = r0 + 16 * m + l16, c = n0 + 16 * n + 4 * quarter;
    if (r < rows.count && c < a.d_out) {
      const int64_t row = rows.at(r);
      const float xs = a.x_scale[rows.x_row(row)];
      const int64_t en = (int64_t)rows.expert * a.d_out + c;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = (float)t[e] * (xs * a.w_scale[en + e]);
        if (a.bias) v[e] += a.bias[en + e];
      }
      store4<Y>(a.y, row * a.ldy + c, v);
    }
  }
}

template <typename Y, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void few_kernel(Int8Args a, int group0, int most) {
  __shared__ i32x4 lds[4 * NT * WAVES * 64];
  const int n0 = blockIdx.x * 16 * NT;
  Rows rows{nullptr, (int)a.rows, 0, 1};
  int r0 = 0, end = rows.count;
  if (a.meta.sorted) {
    rows = segment(a, group0 + blockIdx.y);
    end = rows.count <= most ? rows.count : 0;
  } else {
    r0 = (group0 + blockIdx.y) * 64;
    end = min(end, r0 + 64);
  }
  for (; r0 < end; r0 += 64) {
    if (end - r0 <= 16) few_block<Y, 1, NT, WAVES, 4>(a, rows, r0, n0, lds);
    else if (end - r0 <= 32) few_block<Y, 2, NT, WAVES, 2>(a, rows, r0, n0, lds);
    else few_block<Y, 4, NT, WAVES, 2>(a, rows, r0, n0, lds);
  }
}

// With metadata, the segments of at most `most` rows.
template <typename Y>
hipError_t launch_few(const Int8Args &a, int most, hipStream_t s) {
  const int64_t groups = a.meta.sorted ? std::min<int64_t>(a.rows, a.experts) + 1 : (a.rows + 63) / 64;
  constexpr int kNT = 2, kWaves = 8;
  const int64_t cols = (a.d_out + 16 * kNT - 1) / (16 * kNT);
  // a launch holds fewer than 2^32 threads, and 2^16 rows of its grid
  const int64_t rows = std::max<int64_t>(1, std::min<int64_t>(32768, ((int64_t)1 << 22) / cols));
  for (int64_t g0 = 0; g0 < groups; g0 += rows) {
    const dim3 grid((unsigned)cols, (unsigned)std::min(groups - g0, rows));
    few_kernel<Y, kNT, kWaves><<<grid, dim3(64 * kWaves), 0, s>>>(a, (int)g0, most);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_int8(const Int8Args &a, bool bf16, hipStream_t s) {
  // tiles address x in 32 bits: all of it where rows are gathered, 256 rows else
  const int64_t x_rows = a.meta.sorted ? (a.rows - 1) / a.meta.x_row_div + 1 : 256;
  const bool tiles = a.rows > kFewRows && x_rows * a.ldx < ((int64_t)1 << 32);
  const int most = tiles ? kFewRows : INT32_MAX;
  if (a.meta.sorted || !tiles) {
    const hipError_t err = bf16 ? launch_few<uint16_t>(a, most, s) : launch_few<float>(a, most, s);
    if (err != hipSuccess) return err;
  }
  return tiles ? launch_int8_tile(a, bf16, kFewRows + 1, s) : hipSuccess;
}

}  // namespace lora
