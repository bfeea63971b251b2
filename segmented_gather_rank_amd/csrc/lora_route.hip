// lora_route.hip -- expert choices from a router's logits.
//
// 16 lanes hold a token's values (a wave does, beyond 256 experts or 16 choices) as
// integers that order like them, PER consecutive experts a lane, so that equal values go
// to the lowest id by going to the lowest lane.
//
// 16 lanes: the topk-th largest of the maxima of the lanes' halves bounds the choices from
// below, and few values reach it (8 choices of 256: 10 or so).  They are laid out one a
// lane, and each counts how many come before it.  (Of whole lanes' maxima a grouped choice
// leaves too few: 17705 tokens 29 us for 25 then.)  A wave, or a token of whose values
// more than 16 reach the bound: topk rounds, each of which takes the largest that is left.
//
// What decides a choice is compared exactly.  Without bias (and where a group's rank is
// its largest value) the logits themselves are ordered.  With it c = s + bias is
// rounded, and two values that differ in 64 bits may agree or change places in 32: what
// comes within the error bound of its neighbour is compared again in 64 bits.  Choices
// that reached the bound are, one a lane; groups whose ranks leave the border open, the
// whole wave a token (all of it that way: 26.5 us for 20.8), and so are rounds.  Where all
// biases are equal and logits repeat (bf16) that may be all tokens.
//
// Bound: vector instructions, some 350 a token of 256 experts (scores and keys of 16 a
// lane, the groups' two largest, the bound), not its 1 KB.  17705 tokens x 256 experts
// fp32, 8 choices in 4 of 8 groups, with bias: 21.2 us a call, of which the tokens that are
// done again take 2; softmax without groups or bias: 10 us, 13 where weights are not
// renormalised; 4609 x 60 bf16, 4 choices: 4.7; one token of 256: 6.5, four dependent loads
// and the way through.  A wave a token: 4608 x 1024, 10 choices: 22 us, 17705 x 256, 32
// choices: 46, a chain of two folds a choice.
//
// Four waves a SIMD leave 128 registers, of which those of 256 experts spill 9 (bf16: 12), 40
// and 52 bytes a lane, since the pass in 64 bits is compiled into the kernel.  (Before it was,
// three waves measured as four, 21.1 us; five, 29.)
#include <algorithm>
#include <cmath>

#include "lora_base_host.h"

namespace lora {

namespace {

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

// In 32 bits the exponential and the quotient are the hardware's, a step off each: the
// choice allows for it, and the weights' quotients are taken in 64.
__device__ __forceinline__ float exp_of(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504f); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
__device__ __forceinline__ float inverse(float v) { return __builtin_amdgcn_rcpf(v); }
__device__ __forceinline__ double inverse(double v) { return 1. / v; }

template <typename X>
__device__ __forceinline__ float logit_at(const char *row, int e) {
  if constexpr (sizeof(X) == 2) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(row)[e] << 16);
  else return reinterpret_cast<const float *>(row)[e];
}

// ---------------------------------------------------------------- one token

template <int PER>
struct Token {
  float x[PER], bias[PER];       // of experts base .. base + PER - 1; -inf and 0 past the last
  int base, lane;                // lane of the token's
  float top;                     // largest logit (NaN aside)
};

// How near two values in 32 bits may be for their order to stand: twice a value's error.
// s is within 30 * 2^-24 of its size (the exponential, sums of 16 a lane and of the lanes,
// the quotient) and, by the exponent's argument z (its difference, its product with log2 e
// and that number's own rounding), 2.3 |z| * 2^-24.  2 (30 + 2.3 |z|) is below 400 up to |z|
// = 73; from there on s is below 2e-32, and what is missing up to |z| = 104, where the
// exponential ends (below 1e-38 it is 0), below the 1e-36.  With a bias, whose sum adds a
// rounding of c, the argument's part is at most 2.3 |z| e^-|z| < 0.9 steps of 1, and s at
// most 1.  `unit`: what v counts 1 as.
__device__ __forceinline__ float near(float v, bool biased, float unit = 1.f) {
  return biased ? 64.f * 0x1p-24f * (unit + fabsf(v)) : 400.f * 0x1p-24f * fabsf(v) + 1e-36f * unit;
}

template <typename S> __device__ __forceinline__ void two_largest(S v, S &first, S &second) {
  second = larger(second, smaller(first, v));
  first = larger(first, v);
}

// Whether 64 bits may have a rank of at most `out` in the place of one of at least `in`
// (each the farthest of the token's lanes).
template <int LANES, typename S> __device__ __forceinline__ bool may_change(S in, S out) {
  in = least<LANES>(in);
  out = most<LANES>(out);
  return out >= in && fabs(out) < INFINITY;
}

// The values' own order where nothing is added to them, and c where it is; kGone for
// experts past the last.  `stays`: a bit a group, of its own group at least in each lane.
// `unsure`: 32 bits could not tell which.  lds: LANES * PER values and kMaxGroups ranks, in 32 bits also
// how far off each may be.
template <typename S, int LANES, int PER>
__device__ __forceinline__ void keys_of(const RouteArgs &a, const Token<PER> &t, S *lds, typename Ordered<S>::key k[PER],
                                        uint64_t &stays, bool &unsure) {
  typedef Ordered<S> O;
  constexpr bool kExact = std::is_same<S, double>::value;
  const bool by_rank = a.groups > 1 && a.group_top > 1, biased = a.bias != nullptr;
  S c[PER];                      // what groups are ranked by
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] = t.x[i] == t.x[i] ? (S)t.x[i] : -(S)INFINITY;
    k[i] = O::of(c[i]);
  }
  if (biased || by_rank) {       // the order needs s
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = inverse((S)1 + exp_of(-(S)t.x[i]));
    } else {
      S sum = 0;
      const S top = (S)t.top;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const S x = (S)t.x[i];
        c[i] = x == top ? (S)1 : exp_of(x - top);
        sum += x == x ? c[i] : (S)0;
      }
      // one lane's sum for all: equal logits have equal scores
      const S by = __shfl(total<LANES>(sum), 0, LANES);
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = kExact ? c[i] / by : c[i] * inverse(by);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (biased) c[i] += (S)t.bias[i];
      if (!(t.x[i] > -INFINITY) || c[i] != c[i]) c[i] = -(S)INFINITY;  // masked, NaN
      if (biased) k[i] = O::of(c[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (t.base + i >= a.experts) k[i] = O::kGone;
  stays = ~0ull;
  if (a.groups == 1) return;

  const int size = a.experts / a.groups;
  // The group's rank; in 32 bits the 64-bit one is within `off` of it (c's own rounding
  // goes by the sizes of the two, which may cancel), and of scores a quarter is taken, so
  // that neither the sum nor the bounds leave float32 where c does not.
  S off = 0;
  const S unit = !kExact && (biased || by_rank) ? (S)0.25 : (S)1;
  auto rank_of = [&](S first, S second) {
    first *= unit;
    second *= unit;
    S v = a.group_top > 1 ? first + second : first;
    if (v != v) v = -(S)INFINITY;  // a bias of +inf beside masked experts alone
    if constexpr (!kExact) {
      const S of = fabsf(first) + (a.group_top > 1 ? fabsf(second) : 0.f);
      off = (biased || by_rank) && of < INFINITY ? near(of, biased, 0.25f) : 0.f;
    }
    return v;
  };
  // What the lowest rank that stays may be, and the highest that does not.
  S in = INFINITY, out = -INFINITY;
  auto border = [&](bool stays, S v) {
    if constexpr (!kExact) {
      if (stays) in = smaller(in, v - off);
      else out = larger(out, v + off);
    }
  };
  if (LANES == 16 && a.group_lanes) {
    // a group is `group_lanes` neighbouring lanes, a power of two
    S first = -(S)INFINITY, second = -(S)INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) two_largest(t.base + i < a.experts ? c[i] : -(S)INFINITY, first, second);
    auto join = [&](S f, S s) {
      second = larger(larger(second, s), smaller(first, f));
      first = larger(first, f);
    };
    if (a.group_lanes > 1) join(turned<0xB1>(first), turned<0xB1>(second));    // lane ^ 1
    if (a.group_lanes > 2) join(turned<0x4E>(first), turned<0x4E>(second));    // lane ^ 2
    if (a.group_lanes > 4) join(turned<0x141>(first), turned<0x141>(second));  // 7 - lane: the other four
    const S mine = rank_of(first, second);
    int before = 0;
    // lane l reads lane l - n of its 16: a group before its own where l >= n, n whole groups
    auto against = [&](S v, int n) { before += v > mine || (v == mine && t.lane >= n); };
    if (a.group_lanes == 1) {
      against(turned<0x121>(mine), 1);
      against(turned<0x123>(mine), 3);
      against(turned<0x125>(mine), 5);
      against(turned<0x127>(mine), 7);
      against(turned<0x129>(mine), 9);
      against(turned<0x12B>(mine), 11);
      against(turned<0x12D>(mine), 13);
      against(turned<0x12F>(mine), 15);
    }
    if (a.group_lanes <= 2) {
      against(turned<0x122>(mine), 2);
      against(turned<0x126>(mine), 6);
      against(turned<0x12A>(mine), 10);
      against(turned<0x12E>(mine), 14);
    }
    if (a.group_lanes <= 4) {
      against(turned<0x124>(mine), 4);
      against(turned<0x12C>(mine), 12);
    }
    against(turned<0x128>(mine), 8);
    border(before < a.kept, mine);
    if (!kExact && (biased || by_rank)) unsure = may_change<LANES>(in, out);
    stays = before < a.kept ? ~0ull : 0;
    return;
  }
  // groups of any size: the token's values in LDS, a group a lane
  S *rank = lds + LANES * PER, *spread = rank + kMaxGroups;
#pragma unroll
  for (int i = 0; i < PER; ++i) lds[t.base + i] = c[i];
  wave_sync();
  for (int g = t.lane; g < a.groups; g += LANES) {
    S first = -(S)INFINITY, second = -(S)INFINITY;
#pragma unroll 4
    for (int i = 0; i < size; ++i) two_largest(lds[g * size + i], first, second);
    rank[g] = rank_of(first, second);
    if (!kExact) spread[g] = off;
  }
  wave_sync();
  stays = 0;
  for (int g = t.lane; g < a.groups; g += LANES) {
    const S mine = rank[g];
    int before = 0;
    for (int f = 0; f < a.groups; ++f) {
      const S v = rank[f];
      before += v > mine || (v == mine && f < g);
    }
    if (!kExact) off = spread[g];
    border(before < a.kept, mine);
    if (before < a.kept) stays |= 1ull << g;
  }
  if (!kExact && (biased || by_rank)) unsure = may_change<LANES>(in, out);
  wave_sync();
  stays = (uint64_t)fold<LANES>((int64_t)stays, [](int64_t p, int64_t q) { return p | q; });
}

// kGone for the experts of groups that do not stay.
template <int PER, typename K>
__device__ __forceinline__ void drop(const RouteArgs &a, int base, uint64_t stays, K gone, K k[PER]) {
  if (a.groups == 1) return;
  const int size = a.experts / a.groups;
  int g = base / size;
  if (a.group_lanes) {           // a lane's are of one group
    if (!(stays >> g % 64 & 1)) {
#pragma unroll
      for (int i = 0; i < PER; ++i) k[i] = gone;
    }
    return;
  }
  int left = (g + 1) * size - base;  // experts of group g from this one on
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (g < a.groups && !(stays >> g & 1)) k[i] = gone;
    if (--left == 0) {
      ++g;
      left = size;
    }
  }
}

// The topk largest in rounds: choice j stays in lane j.
template <typename S, int LANES, int PER>
__device__ __forceinline__ void by_rounds(const RouteArgs &a, const Token<PER> &t, typename Ordered<S>::key k[PER], int &id,
                                          bool &unsure) {
  typedef Ordered<S> O;
  typedef typename O::key key;
  const bool margins = std::is_same<S, float>::value && a.bias != nullptr;
  S last = 0;
  for (int j = 0; j < a.topk + (margins ? 1 : 0); ++j) {
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
    if (j == t.lane) id = e;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e == t.base + i) k[i] = O::kGone;
  }
}

// How many of the 16 lanes' values come before this lane's: larger ones, and equal ones
// of lower lanes.
template <int N = 1, typename T>
__device__ __forceinline__ int before_me(T v, int lane) {
  if constexpr (N == 16) {
    return 0;
  } else {
    const T o = turned<0x120 + N>(v);  // lane - N's
    return (int)(lane >= N ? o >= v : o > v) + before_me<N + 1>(v, lane);
  }
}

// How many of 16 lanes' pairs of values are larger than this lane's two.
template <int N = 1>
__device__ __forceinline__ void larger_pairs(int32_t high, int32_t low, int &over_high, int &over_low) {
  if constexpr (N < 16) {
    const int32_t h = turned<0x120 + N>(high), l = turned<0x120 + N>(low);
    over_high += (int)(h > high) + (int)(l > high);
    over_low += (int)(h > low) + (int)(l > low);
    larger_pairs<N + 1>(high, low, over_high, over_low);
  }
}

// A value that reached the bound.
struct Reached {
  int32_t key, id;
};

// c of one expert a lane, in 64 bits.
template <typename X, int PER>
__device__ __forceinline__ double exact(const RouteArgs &a, const char *row, const Token<PER> &t, int e) {
  const double top = (double)t.top;
  auto term = [&](double x) { return x == top ? 1. : exp(x - top); };
  const double x = (double)logit_at<X>(row, e);
  double c;
  if (a.sigmoid) {
    c = 1. / (1. + exp(-x));
  } else {
    double sum = 0;
#pragma unroll 1
    for (int i = 0; i < PER && t.base + i < a.experts; ++i) {
      const double of = (double)logit_at<X>(row, t.base + i);
      if (of == of) sum += term(of);
    }
    c = term(x) / __shfl(total<16>(sum), 0, 16);
  }
  c += (double)a.bias[e];
  return x > -INFINITY && c == c ? c : -(double)INFINITY;
}

// The topk (at most 16) largest of 16 lanes' values; false where more than 16 reach the
// bound.  `box`: 16 places of this token's in LDS.
template <typename X, int PER>
__device__ __forceinline__ bool by_bound(const RouteArgs &a, const char *row, const Token<PER> &t, const int32_t k[PER], Reached *box,
                                         int &id) {
  typedef Ordered<float> O;
  const bool margins = a.bias != nullptr;
  // the bound: of the maxima of every lane's two halves (groups may have left few lanes), the topk-th largest
  int32_t high = k[0], low = PER > 1 ? k[PER / 2] : O::kGone;
#pragma unroll
  for (int i = 1; i < PER; ++i) {
    int32_t &m = i < (PER + 1) / 2 ? high : low;
    m = larger(m, k[i]);
  }
  int over_high = low > high, over_low = high > low;
  larger_pairs(high, low, over_high, over_low);
  int32_t bound = least<16>(smaller(over_high < a.topk ? high : INT32_MAX, over_low < a.topk ? low : INT32_MAX));
  // fewer halves than choices hold any value: all that are left
  bound = larger(bound, O::kGone + 1);
  if (margins) {
    // what 64 bits might put before the last choice reaches it too
    const float v = O::value(bound);
    if (fabsf(v) < INFINITY) bound = O::of(v - near(v, true));
  }
  int n = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) n += k[i] >= bound;
  int upto = n;
  upto += __builtin_amdgcn_update_dpp(0, upto, 0x111, 0xf, 0xf, false);  // row_shr:1
  upto += __builtin_amdgcn_update_dpp(0, upto, 0x112, 0xf, 0xf, false);
  upto += __builtin_amdgcn_update_dpp(0, upto, 0x114, 0xf, 0xf, false);
  upto += __builtin_amdgcn_update_dpp(0, upto, 0x118, 0xf, 0xf, false);
  const int all = __shfl(upto, 15, 16);
  if (__any(all > 16)) return false;
  int at = upto - n;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (k[i] >= bound) box[at++] = Reached{k[i], t.base + i};
  wave_sync();
  Reached mine{O::kGone, 0};
  if (t.lane < all) mine = box[t.lane];      // by ascending id: a lower lane has the lower one
  const int place = before_me(mine.key, t.lane);
  wave_sync();
  if (t.lane < all) box[place] = mine;
  wave_sync();
  Reached it{O::kGone, 0};
  if (t.lane < all) it = box[t.lane];
  id = it.id;
  if (margins) {
    const int32_t prior = __builtin_amdgcn_update_dpp(O::kGone, it.key, 0x111, 0xf, 0xf, false);
    const float v = O::value(it.key), p = O::value(prior);
    const bool near_by = t.lane > 0 && t.lane <= a.topk && t.lane < all && v > -INFINITY && p - v <= near(p, true);
    // 16 choices: the next one has no lane, and did not reach the bound, or there would be more than 16
    if (__any(near_by)) {
      const double c = exact<X>(a, row, t, mine.id);
      const int at64 = before_me(t.lane < all ? Ordered<double>::of(c) : Ordered<double>::kGone, t.lane);
      if (t.lane < all) box[at64].id = mine.id;
      wave_sync();
      if (t.lane < all) id = box[t.lane].id;
    }
  }
  wave_sync();
  return true;
}

// A token's logits and biases, over LANES lanes.
template <typename X, int LANES, int PER>
__device__ __forceinline__ Token<PER> token_at(const RouteArgs &a, const char *row) {
  Token<PER> t;
  t.lane = threadIdx.x % LANES;
  t.base = t.lane * PER;
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
#pragma unroll
      for (int i = 0; i < PER; ++i) t.bias[i] = a.bias ? a.bias[t.base + i] : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool in = t.base + i < a.experts;
      t.x[i] = in ? logit_at<X>(row, t.base + i) : -INFINITY;
      t.bias[i] = in && a.bias ? a.bias[t.base + i] : 0.f;
    }
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, t.x[i]);
  t.top = most<LANES>(top);
  return t;
}

template <typename X, int LANES, int PER>
__global__ __launch_bounds__(256, LANES == 64 && PER > 8 ? 2 : 4) void route_kernel(RouteArgs a) {
  constexpr int kTokens = 64 / LANES;             // a wave's
  constexpr int kExactPer = LANES * PER / 64 < 1 ? 1 : LANES * PER / 64;
  __shared__ Reached boxes[LANES == 16 ? 256 : 1];
  // a wave's: values and ranks of its tokens, or of one token in 64 bits
  constexpr int kShort = kTokens * (LANES * PER + 2 * kMaxGroups) * (int)sizeof(float);
  constexpr int kExact = (64 * kExactPer + kMaxGroups) * (int)sizeof(double);
  __shared__ __align__(16) char values[4][kShort > kExact ? kShort : kExact];
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const int64_t first = (int64_t)blockIdx.x * (4 * kTokens) + wave * kTokens;
  const int64_t token = first + lane / LANES;
  const bool real = token < a.tokens;
  // a wave's surplus lanes do the last token again, and do not write
  auto row_of = [&](int64_t i) { return a.logits + min(i, a.tokens - 1) * a.ld * (int64_t)sizeof(X); };
  const char *row = row_of(token);
  const Token<PER> t = token_at<X, LANES, PER>(a, row);
  bool nan = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) nan |= t.x[i] != t.x[i];
  nan = fold<LANES>((int)nan, [](int p, int q) { return p | q; });

  int id = 0;
  bool unsure = false, done = false;
  int32_t k[PER];
  uint64_t stays;
  keys_of<float, LANES, PER>(a, t, reinterpret_cast<float *>(values[wave]) + lane / LANES * (LANES * PER + 2 * kMaxGroups), k, stays,
                             unsure);
  // what 32 bits left open, in 64: the whole wave a token
  auto again = [&](uint64_t tokens, auto &&f) {
    while (tokens) {
      const int q = __builtin_ctzll(tokens) / LANES;
      tokens &= LANES == 64 ? 0 : ~(((1ull << LANES % 64) - 1) << q * LANES);
      const Token<kExactPer> u = token_at<X, 64, kExactPer>(a, row_of(first + q));
      int64_t v[kExactPer];
      uint64_t in;
      bool never = false;
      wave_sync();
      keys_of<double, 64, kExactPer>(a, u, reinterpret_cast<double *>(values[wave]), v, in, never);
      f(lane / LANES == q, u, v, in);
    }
  };
  again(__ballot(unsure), [&](bool own, const Token<kExactPer> &, const int64_t *, uint64_t in) {
    if (own) stays = in;
  });
  drop<PER>(a, t.base, stays, Ordered<float>::kGone, k);
  unsure = false;
  if constexpr (LANES == 16) done = by_bound<X, PER>(a, row, t, k, boxes + threadIdx.x / 16 * 16, id);
  if (!done) {
    by_rounds<float, LANES, PER>(a, t, k, id, unsure);
    again(__ballot(unsure), [&](bool own, const Token<kExactPer> &u, int64_t *v, uint64_t in) {
      int e = 0;
      bool never = false;
      drop<kExactPer>(a, u.base, in, Ordered<double>::kGone, v);
      by_rounds<double, 64, kExactPer>(a, u, v, e, never);
      e = __shfl(e, lane % LANES, 64);
      if (own) id = e;
    });
  }

  // the chosen one's score, in 64 bits
  double s = 0, sum = 1;
  if (t.lane < a.topk) {
    const float x = logit_at<X>(row, id);
    if (x > -INFINITY) s = a.sigmoid ? 1. / (1. + exp(-(double)x)) : x == t.top ? 1. : exp((double)x - (double)t.top);
  }
  if (a.renorm) {
    sum = total<LANES>(s);
  } else if (!a.sigmoid) {
    // the sum of all: its terms in 32 bits (a step, and |z| 2^-24 of an argument z that e^z makes small), added in 64
    double part = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (t.x[i] > -INFINITY) part += (double)(t.x[i] == t.top ? 1.f : expf(t.x[i] - t.top));
    sum = total<LANES>(part);
  }
  if (real && t.lane < a.topk) {
    float w = sum > 0 ? (float)(s / sum * (double)a.scale) : 0.f;
    if (nan) w = __builtin_nanf("");
    a.ids[token * a.topk + t.lane] = id;
    a.weights[token * a.topk + t.lane] = w;
  }
}

template <typename X, int LANES, int PER>
hipError_t launch_as(RouteArgs all, hipStream_t s) {
  constexpr int kTokens = 256 / LANES;
  // groups that are 1, 2, 4 or 8 whole lanes
  const int size = all.experts / all.groups, lanes = size / PER;
  const bool whole = LANES == 16 && all.groups > 1 && size % PER == 0 && lanes <= 8 && (lanes & (lanes - 1)) == 0;
  all.group_lanes = whole ? lanes : 0;
  constexpr int64_t kMost = (int64_t)1 << 22;  // workgroups of a launch
  for (int64_t t0 = 0; t0 < all.tokens; t0 += kMost * kTokens) {
    RouteArgs a = all;
    a.tokens = std::min(all.tokens - t0, kMost * kTokens);
    a.logits += t0 * a.ld * (int64_t)sizeof(X);
    a.ids += t0 * a.topk;
    a.weights += t0 * a.topk;
    route_kernel<X, LANES, PER><<<dim3((unsigned)((a.tokens + kTokens - 1) / kTokens)), dim3(256), 0, s>>>(a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <typename X>
hipError_t launch_for(const RouteArgs &a, hipStream_t s) {
  if (a.experts <= 256 && a.topk <= 16) {
    if (a.experts <= 16) return launch_as<X, 16, 1>(a, s);
    if (a.experts <= 64) return launch_as<X, 16, 4>(a, s);
    if (a.experts <= 128) return launch_as<X, 16, 8>(a, s);
    return launch_as<X, 16, 16>(a, s);
  }
  if (a.experts <= 256) return launch_as<X, 64, 4>(a, s);
  if (a.experts <= 512) return launch_as<X, 64, 8>(a, s);
  return launch_as<X, 64, 16>(a, s);
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? launch_for<uint16_t>(a, s) : launch_for<float>(a, s);
}

}  // namespace lora
