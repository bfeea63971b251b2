// lora_quant.hip -- rows (or the gated activation of rows) to 8-bit integers with a
// scale each.
//
// Bound: HBM; a row is read once and stays in registers between its maximum and its
// rounding, THREADS threads a row, CH pieces of 8 values a thread.  Rows too long for
// that are read twice.  17705 rows of 4096 bf16: 35.7 us, 6.1 TB/s (read and write: the
// call before left part of the rows in the last-level cache); the activation of 36864
// rows of 2 x 2048 bf16, written too: 113 us, 4.7 TB/s (a large copy: 5.1).  In fp32: 65 us,
// 5.6 TB/s, and 165 us, 5.9.
//
// The rounding is that of the real number 127 v / m.  In 32 bits v * (127 / m) is within
// 2^-23 * 127 of it, so that the nearest integer stands unless the product is that near
// to a half; then the quotient is taken in 64 bits, whose 53 are enough: 254 v is either an
// odd multiple of m or differs from it by 2^-32 of itself at least.
#include <algorithm>
#include <cmath>

#include "lora_base_host.h"

namespace lora {

namespace {

template <typename X> __device__ __forceinline__ const X *row_of(const char *x, int64_t row, int64_t ld) {
  return reinterpret_cast<const X *>(x) + row * ld;
}

// Largest of the magnitudes' bit patterns: those of infinities and NaN are above all others.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

template <int CTRL>
__device__ __forceinline__ uint32_t turned(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
__device__ __forceinline__ uint32_t wave_most(uint32_t v) {
  v = max(v, turned<0x121>(v));
  v = max(v, turned<0x122>(v));
  v = max(v, turned<0x124>(v));
  v = max(v, turned<0x128>(v));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}

// x / (1 + exp(-x)) * u.  exp(-|x|), which does not overflow, as the square of its root,
// which the hardware's exponential does not flush to 0 before the square does; what the
// root's argument loses to its rounding (-|x| - 2 ln 2 times the argument, up to 4e-6: ln 2
// as two float32 numbers) corrects the square.  In all 12 * 2^-24 at most: 6 of e, a rounding
// of 1 + e, a step of the hardware's inverse, three products.
__device__ __forceinline__ float gated(float x, float u) {
  const float m = fabsf(x);
  const float z = m * -0.72134752f;                     // -m / (2 ln 2)
  const float left = fmaf(z, 3.8094e-9f, fmaf(z, -1.38629436f, -m));
  const float root = __builtin_amdgcn_exp2f(z), square = root * root;
  // (of an infinity `left` is no number, and e 0)
  const float e = fminf(fmaxf(fmaf(square, left, square), 0.f), 1.f);
  return x * (x < 0.f ? e : 1.f) * __builtin_amdgcn_rcpf(1.f + e) * u;
}

template <typename X, bool ACT>
__device__ __forceinline__ void values(const X *row, int width, int at, float v[8]) {
  load8(row + at, v);
  if constexpr (ACT) {
    float u[8];
    load8(row + width + at, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = gated(v[e], u[e]);
  }
}

struct Step {
  float m, by;       // the largest magnitude, 127 / m
  bool finite, exact_only;
  __device__ __forceinline__ explicit Step(uint32_t most) {
    m = __uint_as_float(most);
    finite = most < 0x7f800000u;
    by = finite && most ? 127.f / m : 0.f;
    exact_only = !(by < INFINITY);
  }
  __device__ __forceinline__ float scale() const { return finite ? m / 127.f : __builtin_nanf(""); }
  __device__ __forceinline__ int nearest(float v) const { return (int)rint((double)v * 127. / (double)m); }
};

__device__ __forceinline__ void put(int8_t *q, const Step &s, const float v[8]) {
  // adding 1.5 * 2^23 rounds to an integer, which the low bits then hold
  constexpr float kRound = 12582912.f;
  float t[8], off = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float p = v[e] * s.by;
    t[e] = p + kRound;
    off = fmaxf(off, fabsf(p - (t[e] - kRound)));
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 1]), __float_as_uint(t[4 * h]), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 3]), __float_as_uint(t[4 * h + 2]), 0x04000c0cu);
    w[h] = lo | hi;
  }
  if (s.exact_only || off > 0.5f - 0x1p-15f) {
    w[0] = w[1] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e / 4] |= ((uint32_t)s.nearest(v[e]) & 0xffu) << (8 * (e % 4));
  }
  if (!s.finite) w[0] = w[1] = 0;
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(1))) u32x2 g_u32x2;
  *(g_u32x2 *)q = u32x2{w[0], w[1]};
}

// A row's maximum over its THREADS threads (a wave, or the whole workgroup).
template <int THREADS>
__device__ __forceinline__ uint32_t row_most(uint32_t v, uint32_t *lds) {
  v = wave_most(v);
  if constexpr (THREADS > 64) {
    if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) v = max(v, lds[w]);
  }
  return v;
}

// CH = 0: a row of any length, read twice.
template <typename X, bool ACT, int THREADS, int CH>
__global__ __launch_bounds__(256) void quantize_kernel(QuantArgs a) {
  __shared__ uint32_t most_of[4];
  constexpr int kRows = 256 / THREADS;
  const int tid = threadIdx.x % THREADS;
  const int64_t i = (int64_t)blockIdx.x * kRows + threadIdx.x / THREADS;
  bool live = i < a.rows;
  int64_t row = live ? i : a.rows - 1;
  if (a.sorted) {
    live = live && a.sorted_slot[row] >= 0;
    row = a.sorted[row];
  }
  // the same for all threads of a row, so none waits at a barrier for one that left
  if (!live) return;
  const X *x = row_of<X>(a.x, row, a.ldx);
  int8_t *q = a.q + row * a.ldq;
  X *act = ACT && a.act ? reinterpret_cast<X *>(a.act) + row * a.ldact : nullptr;
  uint32_t most = 0;
  if constexpr (CH > 0) {
    float v[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = 8 * (tid + c * THREADS);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = 0.f;
      if (at < a.width) values<X, ACT>(x, a.width, at, v[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) most = max(most, magnitude(v[c][e]));
    const Step s(row_most<THREADS>(most, most_of));
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = 8 * (tid + c * THREADS);
      if (at < a.width) {
        put(q + at, s, v[c]);
        if (act) store8(act + at, v[c]);
      }
    }
    if (tid == 0) a.scale[row] = s.scale();
  } else {
    float v[8];
    for (int at = 8 * tid; at < a.width; at += 8 * THREADS) {
      values<X, ACT>(x, a.width, at, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) most = max(most, magnitude(v[e]));
    }
    const Step s(row_most<THREADS>(most, most_of));
    for (int at = 8 * tid; at < a.width; at += 8 * THREADS) {
      values<X, ACT>(x, a.width, at, v);
      put(q + at, s, v);
      if (act) store8(act + at, v);
    }
    if (tid == 0) a.scale[row] = s.scale();
  }
}

template <typename X, bool ACT, int THREADS, int CH>
hipError_t launch_as(const QuantArgs &a, hipStream_t s) {
  constexpr int kRows = 256 / THREADS;
  // at most 2^30 rows: a launch of 2^23 workgroups covers 2^23 or more of them
  constexpr int64_t kMost = (int64_t)1 << 23;
  for (int64_t r0 = 0; r0 < a.rows; r0 += kMost) {
    QuantArgs b = a;
    b.rows = std::min(a.rows - r0, kMost);
    if (a.sorted) {
      b.sorted += r0;
      b.sorted_slot += r0;
    } else {
      b.x += r0 * a.ldx * (int64_t)sizeof(X);
      b.q += r0 * a.ldq;
      b.scale += r0;
      if (b.act) b.act += r0 * a.ldact * (int64_t)sizeof(X);
    }
    quantize_kernel<X, ACT, THREADS, CH><<<dim3((unsigned)((b.rows + kRows - 1) / kRows)), dim3(256), 0, s>>>(b);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <typename X, bool ACT>
hipError_t launch_for(const QuantArgs &a, hipStream_t s) {
  if (a.width <= 512) return launch_as<X, ACT, 64, 1>(a, s);
  if (a.width <= 1024) return launch_as<X, ACT, 64, 2>(a, s);
  if (a.width <= 2048) return launch_as<X, ACT, 256, 1>(a, s);
  if (a.width <= 4096) return launch_as<X, ACT, 256, 2>(a, s);
  if (a.width <= 8192) return launch_as<X, ACT, 256, 4>(a, s);
  if (a.width <= 16384) return launch_as<X, ACT, 256, 8>(a, s);
  return launch_as<X, ACT, 256, 0>(a, s);
}

}  // namespace

hipError_t launch_quantize(const QuantArgs &a, bool bf16, hipStream_t s) {
  if (a.gated) return bf16 ? launch_for<uint16_t, true>(a, s) : launch_for<float, true>(a, s);
  return bf16 ? launch_for<uint16_t, false>(a, s) : launch_for<float, false>(a, s);
}

}  // namespace lora
