// lora_route.hip -- expert choices from a router's logits.
//
// 16 lanes (or a wave, beyond 256 experts) hold a token's values as integers that order
// like them, PER consecutive experts a lane, so that equal values go to the lowest id by
// going to the lowest lane.  Each of topk rounds takes the largest: a lane's own by its
// registers, a token's by rotations inside a row of 16 lanes.
//
// What decides a choice is compared exactly.  Without bias (and where a group's rank is
// its largest value) the logits themselves are ordered.  With it c = s + bias is
// rounded, and two values that differ in 64 bits may agree or change places in 32: a
// token whose neighbours in the chosen order (or whose last kept and first dropped
// group) come within the error bound of each other is done again in 64 bits.  That is
// one token in some hundred; where all biases are equal and logits repeat (bf16), up to
// all of them.
#include <algorithm>
#include <cmath>

#include "lora_base_host.h"

namespace lora {

namespace {

typedef unsigned int u32x2r __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------- values as ordered integers

template <typename S> struct Ordered;
template <> struct Ordered<float> {
  typedef int32_t key;
  static constexpr key kGone = INT32_MIN;  // below every value's key
  static __device__ __forceinline__ key of(float v) {
    const int32_t b = __float_as_int(v + 0.f);  // -0 is 0
    return b ^ ((b >> 31) & 0x7fffffff);
  }
  static __device__ __forceinline__ float value(key k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }
};
template <> struct Ordered<double> {
  typedef int64_t key;
  static constexpr key kGone = INT64_MIN;
  static __device__ __forceinline__ key of(double v) {
    const int64_t b = __double_as_longlong(v + 0.);
    return b ^ ((b >> 63) & 0x7fffffffffffffffll);
  }
  static __device__ __forceinline__ double value(key k) {
    return __longlong_as_double(k ^ ((k >> 63) & 0x7fffffffffffffffll));
  }
};

// ---------------------------------------------------------------- over the lanes of a token

template <int CTRL>
__device__ __forceinline__ int32_t turned(int32_t v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, false); }
template <int CTRL>
__device__ __forceinline__ int64_t turned(int64_t v) {
  const uint32_t lo = (uint32_t)turned<CTRL>((int32_t)(uint32_t)v), hi = (uint32_t)turned<CTRL>((int32_t)(uint32_t)(v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}
template <int CTRL>
__device__ __forceinline__ float turned(float v) { return __int_as_float(turned<CTRL>(__float_as_int(v))); }
template <int CTRL>
__device__ __forceinline__ double turned(double v) { return __longlong_as_double(turned<CTRL>((int64_t)__double_as_longlong(v))); }

// The value of the lane 16 (then 32) further round the wave.
template <typename T> __device__ __forceinline__ T across(T v, int by) { return __shfl_xor(v, by, 64); }

// f over the LANES lanes of a token, in all of them; every lane folds the same values in
// an order of its own, so f has to give the same whatever the order, or to be a sum whose
// last bits do not decide anything.
template <int LANES, typename T, typename F>
__device__ __forceinline__ T fold(T v, F f) {
  v = f(v, turned<0x121>(v));  // row_ror:1
  v = f(v, turned<0x122>(v));
  v = f(v, turned<0x124>(v));
  v = f(v, turned<0x128>(v));
  if constexpr (LANES == 64) {
    v = f(v, across(v, 16));
    v = f(v, across(v, 32));
  }
  return v;
}
template <typename T> __device__ __forceinline__ T larger(T a, T b) { return a > b ? a : b; }
template <typename T> __device__ __forceinline__ T smaller(T a, T b) { return a < b ? a : b; }
template <int LANES, typename T> __device__ __forceinline__ T most(T v) {
  return fold<LANES>(v, [](T a, T b) { return larger(a, b); });
}
template <int LANES, typename T> __device__ __forceinline__ T least(T v) {
  return fold<LANES>(v, [](T a, T b) { return smaller(a, b); });
}
template <int LANES, typename T> __device__ __forceinline__ T total(T v) {
  return fold<LANES>(v, [](T a, T b) { return a + b; });
}

// LDS written by this wave is read by this wave: operations of one wave stay in order,
// the compiler has to keep them so.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

template <typename X>
__device__ __forceinline__ float logit_at(const char *row, int e) {
  if constexpr (sizeof(X) == 2) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(row)[e] << 16);
  else return reinterpret_cast<const float *>(row)[e];
}

// ---------------------------------------------------------------- one token

template <int LANES, int PER>
struct Token {
  float x[PER];                  // logits of experts base .. base + PER - 1; -inf past the last
  int base, lane;                // lane of the token's
  float top;                     // largest logit (NaN aside)
};

// How near two values in 32 bits may be for their order to stand: twice a value's error.
// s is within (30 + 104) * 2^-24 of its size (the exponential, sums of 16 a lane and of the
// lanes, the division; then the exponent's argument, rounded, up to where the exponential
// ends).  With a bias, whose sum adds half a step, the argument's part is at most
// |z| e^-|z| < 0.4 steps of 1, and s at most 1.
__device__ __forceinline__ float near(float v, bool biased) {
  return biased ? 64.f * 0x1p-24f * (1.f + fabsf(v)) : 320.f * 0x1p-24f * fabsf(v) + 1e-36f;
}

// The chosen experts of the token: lane j % LANES keeps choice j in id[j / LANES].
// Returns whether 32 bits could not tell (S = double: never).
template <typename S, int LANES, int PER, int KEEP>
__device__ __forceinline__ bool choose(const RouteArgs &a, const Token<LANES, PER> &t, S *lds, int id[KEEP]) {
  typedef Ordered<S> O;
  typedef typename O::key key;
  constexpr bool kExact = std::is_same<S, double>::value;
  const bool by_value = a.bias != nullptr || (a.groups > 1 && a.group_top > 1);  // the order needs s
  bool unsure = false;
  key k[PER];
  // the order of experts without bias
#pragma unroll
  for (int i = 0; i < PER; ++i) k[i] = O::of(t.x[i] == t.x[i] ? (S)t.x[i] : -(S)INFINITY);
  if (by_value) {
    S sum = 0;
    S s[PER];
    const S top = (S)t.top;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const S x = (S)t.x[i];
      if (a.sigmoid) {
        s[i] = (S)1 / ((S)1 + exp_of(-x));
      } else {
        s[i] = x == top ? (S)1 : exp_of(x - top);
        sum += x == x ? s[i] : (S)0;
      }
    }
    // one lane's sum for all: equal logits have equal scores
    if (!a.sigmoid) sum = __shfl(total<LANES>(sum), 0, LANES);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = t.base + i;
      S c = a.sigmoid ? s[i] : s[i] / sum;
      if (a.bias && e < a.experts) c += (S)a.bias[e];
      // masked, NaN
      if (!(t.x[i] > -INFINITY) || c != c) c = -(S)INFINITY;
      if (a.bias) k[i] = O::of(c);
      if (a.groups > 1) lds[e] = c;
    }
  } else if (a.groups > 1) {
#pragma unroll
    for (int i = 0; i < PER; ++i) lds[t.base + i] = O::value(k[i]);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (t.base + i >= a.experts) k[i] = O::kGone;

  if (a.groups > 1) {
    // ranks: the token's values are in LDS, a group a lane
    const int size = a.experts / a.groups;
    S *rank = lds + LANES * PER;
    wave_sync();
    for (int g = t.lane; g < a.groups; g += LANES) {
      S first = -(S)INFINITY, second = -(S)INFINITY;
      for (int i = 0; i < size; ++i) {
        const S v = lds[g * size + i];
        second = larger(second, smaller(first, v));
        first = larger(first, v);
      }
      rank[g] = a.group_top > 1 ? first + second : first;
    }
    wave_sync();
    // a group stays if fewer than `kept` come before it
    uint64_t stays = 0;
    for (int g = t.lane; g < a.groups; g += LANES) {
      const S mine = rank[g];
      int before = 0;
      for (int f = 0; f < a.groups; ++f) {
        const S v = rank[f];
        before += v > mine || (v == mine && f < g);
        if constexpr (!kExact) {
          // the ranks around the border only matter, but ranks this near are rare enough
          if (by_value && f != g && v > -INFINITY && fabsf(v - mine) <= 2.f * near(mine, a.bias != nullptr)) unsure = true;
        }
      }
      if (before < a.kept) stays |= 1ull << g;
    }
    wave_sync();
    stays = fold<LANES>((int64_t)stays, [](int64_t p, int64_t q) { return p | q; });
    int g = t.base / size, left = (g + 1) * size - t.base;  // experts of group g from this one on
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (g < a.groups && !((uint64_t)stays >> g & 1)) k[i] = O::kGone;
      if (--left == 0) {
        ++g;
        left = size;
      }
    }
  }

  S last = 0;
  const bool margins = !kExact && a.bias != nullptr;
  const int rounds = a.topk + (margins ? 1 : 0);
  for (int j = 0; j < rounds; ++j) {
    key m = k[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < PER; ++i)
      if (k[i] > m) {
        m = k[i];
        at = i;
      }
    const key best = most<LANES>(m);
    if (margins) {
      const S v = O::value(best);
      if (best != O::kGone && v > -INFINITY && j > 0 && last - v <= (S)near((float)last, true)) unsure = true;
      last = v;
      if (j == a.topk) break;
    }
    const int e = least<LANES>(m == best ? t.base + at : 0x7fffffff);
#pragma unroll
    for (int q = 0; q < KEEP; ++q)
      if (j == t.lane + q * LANES) id[q] = e;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e == t.base + i) k[i] = O::kGone;
  }
  return unsure;
}

template <typename X, int LANES, int PER>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  constexpr int KEEP = LANES == 16 ? 2 : 1;  // choices a lane keeps: at most kMaxTopk in all
  constexpr int kTokens = 64 / LANES;        // a wave's
  // values and ranks of a token, in 64 bits
  extern __shared__ __align__(16) double lds[];
  const int lane = threadIdx.x % 64;
  Token<LANES, PER> t;
  t.lane = lane % LANES;
  t.base = t.lane * PER;
  const int64_t token = (int64_t)blockIdx.x * (4 * kTokens) + threadIdx.x / LANES;
  const bool real = token < a.tokens;
  // a wave's surplus lanes do the last token again, and do not write
  const char *row = a.logits + (real ? token : a.tokens - 1) * a.ld * (int64_t)sizeof(X);
  constexpr int kVec = 16 / (int)sizeof(X);
  if (PER % kVec == 0 && a.aligned && a.experts == LANES * PER) {
    if constexpr (PER % kVec == 0) {
#pragma unroll
      for (int i = 0; i < PER; i += kVec) {
        const u32x4 w = gload16(row + (int64_t)(t.base + i) * (int64_t)sizeof(X));
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          if constexpr (sizeof(X) == 2) t.x[i + v] = (v & 1) ? bf16_hi(w[v / 2]) : bf16_lo(w[v / 2]);
          else t.x[i + v] = __uint_as_float(w[v]);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) t.x[i] = t.base + i < a.experts ? logit_at<X>(row, t.base + i) : -INFINITY;
  }
  float top = -INFINITY;
  int nan = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    top = fmaxf(top, t.x[i]);
    nan |= t.x[i] != t.x[i];
  }
  t.top = most<LANES>(top);
  nan = fold<LANES>(nan, [](int p, int q) { return p | q; });

  double *mine = lds + (threadIdx.x / LANES) * (a.groups > 1 ? LANES * PER + kMaxGroups : 0);
  int id[KEEP];
#pragma unroll
  for (int q = 0; q < KEEP; ++q) id[q] = 0;
  const bool unsure = choose<float, LANES, PER, KEEP>(a, t, reinterpret_cast<float *>(mine), id);
  if (__any(unsure)) choose<double, LANES, PER, KEEP>(a, t, mine, id);

  // the chosen ones' scores, in 64 bits: a lane has one or two
  double s[KEEP], sum = 0;
#pragma unroll
  for (int q = 0; q < KEEP; ++q) {
    s[q] = 0;
    if (t.lane + q * LANES < a.topk) {
      const float x = logit_at<X>(row, id[q]);
      if (x > -INFINITY) s[q] = a.sigmoid ? 1. / (1. + exp(-(double)x)) : x == t.top ? 1. : exp((double)x - (double)t.top);
    }
    sum += s[q];
  }
  if (a.renorm) {
    sum = total<LANES>(sum);
  } else if (!a.sigmoid) {
    // the sum of all: 32 bits a lane (at most 16 of them), 64 across
    float part = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (t.x[i] > -INFINITY) part += t.x[i] == t.top ? 1.f : expf(t.x[i] - t.top);
    sum = total<LANES>((double)part);
  } else {
    sum = 1;
  }
#pragma unroll
  for (int q = 0; q < KEEP; ++q) {
    const int j = t.lane + q * LANES;
    if (real && j < a.topk) {
      float w = sum > 0 ? (float)(s[q] / sum * (double)a.scale) : 0.f;
      if (nan) w = __builtin_nanf("");
      a.ids[token * a.topk + j] = id[q];
      a.weights[token * a.topk + j] = w;
    }
  }
}

template <typename X, int LANES, int PER>
hipError_t launch_as(const RouteArgs &all, hipStream_t s) {
  constexpr int kTokens = 256 / LANES;
  constexpr int64_t kMost = (int64_t)1 << 22;  // workgroups of a launch
  const size_t lds = all.groups > 1 ? sizeof(double) * kTokens * (LANES * PER + kMaxGroups) : 0;
  for (int64_t t0 = 0; t0 < all.tokens; t0 += kMost * kTokens) {
    RouteArgs a = all;
    a.tokens = std::min(all.tokens - t0, kMost * kTokens);
    a.logits += t0 * a.ld * (int64_t)sizeof(X);
    a.ids += t0 * a.topk;
    a.weights += t0 * a.topk;
    route_kernel<X, LANES, PER><<<dim3((unsigned)((a.tokens + kTokens - 1) / kTokens)), dim3(256), lds, s>>>(a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <typename X>
hipError_t launch_for(const RouteArgs &a, hipStream_t s) {
  if (a.experts <= 16) return launch_as<X, 16, 1>(a, s);
  if (a.experts <= 64) return launch_as<X, 16, 4>(a, s);
  if (a.experts <= 128) return launch_as<X, 16, 8>(a, s);
  if (a.experts <= 256) return launch_as<X, 16, 16>(a, s);
  if (a.experts <= 512) return launch_as<X, 64, 8>(a, s);
  return launch_as<X, 64, 16>(a, s);
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? launch_for<uint16_t>(a, s) : launch_for<float>(a, s);
}

}  // namespace lora
