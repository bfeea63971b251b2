// lora_append.hip -- rotation of q and k, and k and v to their place in the
// paged cache, in one pass over the packed q | k | v rows.
//
// Bound: HBM; every element is read once and written once, a few operations
// each.  A workgroup takes one token: its cache place and positions are looked up
// once, and its row is cut into units of 8 pairs (two 16-byte pieces of bf16:
// elements j and j + half of a head, or 16 neighbours when pairs are interleaved)
// and 8 copied elements, one unit a thread and trip.
//
// Measured (32 + 2 x 8 heads of 128, bf16): 17705 tokens 83 us, 5.3 TB/s; 4608
// tokens 20 us, fp32 48 us; one token 3.2 us; 4097 tokens of 28 + 2 x 4 heads to e4m3
// 19.5 us, where 15 would be the copy rate's (320 units for 256 threads, so that a
// second trip runs one wave of four, and a division per stored value).  With a thread per unit (512 threads, no second
// trip) the long batch takes 118 us, with 128 threads 90.
#include <algorithm>

#include "lora_attn_dev.h"

namespace lora {

namespace {

template <typename T>
struct Vec8;
template <>
struct Vec8<uint16_t> {
  static __device__ __forceinline__ void load(const char *base, int64_t i, float v[8]) {
    load8(reinterpret_cast<const uint16_t *>(base) + i, v);
  }
  static __device__ __forceinline__ void store(char *base, int64_t i, const float v[8], float) {
    store8(reinterpret_cast<uint16_t *>(base) + i, v);
  }
};
template <>
struct Vec8<float> {
  static __device__ __forceinline__ void load(const char *base, int64_t i, float v[8]) {
    load8(reinterpret_cast<const float *>(base) + i, v);
  }
  static __device__ __forceinline__ void store(char *base, int64_t i, const float v[8], float) {
    store8(reinterpret_cast<float *>(base) + i, v);
  }
};
struct E4m3 {};
template <>
struct Vec8<E4m3> {
  // value / scale, beyond +-448 the largest value; NaN passes both comparisons
  static __device__ __forceinline__ void store(char *base, int64_t i, const float v[8], float scale) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = v[e] / scale;
      x[e] = y > 448.f ? 448.f : (y < -448.f ? -448.f : y);
    }
    int w0 = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    w0 = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w0, true);
    int w1 = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], 0, false);
    w1 = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], w1, true);
    typedef __attribute__((address_space(1))) u32x2 g_u32x2;
    *(g_u32x2 *)(base + i) = u32x2{(uint32_t)w0, (uint32_t)w1};
  }
};

template <typename X, typename C>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
  const int64_t t = blockIdx.x;
  const int64_t slot = a.slot[t];
  int32_t pos[4] = {0, 0, 0, 0};
  bool bad = slot < -1 || slot >= a.num_slots;
  if (a.table) {
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (x < a.axes) {
        pos[x] = a.pos[x * a.tokens + t];
        bad |= pos[x] < 0 || pos[x] >= a.num_pos;
      }
  }
  if (bad) {
    if (threadIdx.x == 0 && a.num_bad) atomicAdd(a.num_bad, 1);
    return;
  }
  const bool keep = slot >= 0;
  // small caches divide in 32 bits
  const int64_t page = !keep ? 0 : a.num_slots <= 0x7fffffff ? (int64_t)a.by_page.quotient((uint32_t)slot) : slot / a.page_size;
  const int64_t place = keep ? page * a.page_stride + (slot - page * a.page_size) * a.pos_stride : 0;
  const char *x = a.x + t * a.ldx * (int64_t)sizeof(X);
  const int both = a.q_heads + a.kv_heads, half = a.half, rot = 2 * half;
  const int rot_per = half / 8, copy_per = (a.dim - rot) / 8, v_per = a.dim / 8;
  const int n_rot = both * rot_per, n_copy = both * copy_per, n_v = a.kv_heads * v_per;

  // 8 elements of q or k head `head` (k heads follow the q heads) from element d
  auto source = [&](int head) -> int64_t {
    return head < a.q_heads ? a.off_q + (int64_t)head * a.dim : a.off_k + (int64_t)(head - a.q_heads) * a.dim;
  };
  auto put = [&](int head, int d, const float v[8]) {
    if (head < a.q_heads) {
      if (a.q) Vec8<X>::store(a.q, t * a.ldq + (int64_t)head * a.dim + d, v, 1.f);
    } else if (keep) {
      const int kh = head - a.q_heads;
      Vec8<C>::store(a.k, place + kh * a.head_stride + d, v, a.k_scale ? a.k_scale[kh] : 1.f);
    }
  };

  for (int u = threadIdx.x; u < n_rot + n_copy + n_v; u += 256) {
    if (u < n_rot) {
      const int head = (int)a.units[0].quotient(u), c = u - head * rot_per;
      const int d0 = a.interleaved ? 16 * c : 8 * c, d1 = a.interleaved ? d0 + 8 : d0 + half;
      float p[8], q[8], cs[8], sn[8];
      Vec8<X>::load(x, source(head) + d0, p);
      Vec8<X>::load(x, source(head) + d1, q);
      // this unit's pairs 8 c .. 8 c + 7: the axis of the first and of the last
      auto axis_of = [&](int j) {
        int ax = 0;
#pragma unroll
        for (int k = 0; k < 3; ++k) ax += j >= a.axis_end[k] && k + 1 < a.axes;
        return ax;
      };
      auto row_at = [&](int ax) -> int64_t {
        const int pp = ax == 0 ? pos[0] : ax == 1 ? pos[1] : ax == 2 ? pos[2] : pos[3];
        return (int64_t)pp * rot;
      };
      const int ax0 = axis_of(8 * c), ax1 = axis_of(8 * c + 7);
      if (ax0 == ax1) {
        const float *row = a.table + row_at(ax0) + 8 * c;
        load8(row, cs);
        load8(row + half, sn);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float *row = a.table + row_at(axis_of(8 * c + e)) + 8 * c + e;
          cs[e] = row[0];
          sn[e] = row[half];
        }
      }
      float o0[8], o1[8];
      if (a.interleaved) {
        // elements 16 c .. + 15: pairs (p[0], p[1]) ... (q[6], q[7])
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o0[2 * e] = p[2 * e] * cs[e] - p[2 * e + 1] * sn[e];
          o0[2 * e + 1] = p[2 * e + 1] * cs[e] + p[2 * e] * sn[e];
          o1[2 * e] = q[2 * e] * cs[4 + e] - q[2 * e + 1] * sn[4 + e];
          o1[2 * e + 1] = q[2 * e + 1] * cs[4 + e] + q[2 * e] * sn[4 + e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o0[e] = p[e] * cs[e] - q[e] * sn[e];
          o1[e] = q[e] * cs[e] + p[e] * sn[e];
        }
      }
      put(head, d0, o0);
      put(head, d1, o1);
    } else if (u < n_rot + n_copy) {
      const int w = u - n_rot, head = (int)a.units[1].quotient(w), d = rot + 8 * (w - head * copy_per);
      float v[8];
      Vec8<X>::load(x, source(head) + d, v);
      put(head, d, v);
    } else if (keep) {
      const int w = u - n_rot - n_copy, vh = (int)a.units[2].quotient(w), d = 8 * (w - vh * v_per);
      float v[8];
      Vec8<X>::load(x, a.off_v + (int64_t)vh * a.dim + d, v);
      Vec8<C>::store(a.v, place + vh * a.head_stride + d, v, a.v_scale ? a.v_scale[vh] : 1.f);
    }
  }
}

}  // namespace

hipError_t launch_append(const AppendArgs &all, AttnKind kind, hipStream_t s) {
  // a launch holds fewer than 2^32 threads; `tokens` stays the stride of the axes
  constexpr int64_t kMost = 1 << 23;
  const int64_t esize = kind == kAttnF32 ? 4 : 2;
  for (int64_t t0 = 0; t0 < all.tokens; t0 += kMost) {
    AppendArgs a = all;
    a.x += t0 * a.ldx * esize;
    if (a.q) a.q += t0 * a.ldq * esize;
    if (a.pos) a.pos += t0;
    a.slot += t0;
    const dim3 grid((unsigned)std::min(all.tokens - t0, kMost)), block(256);
    if (kind == kAttnF32) append_kernel<float, float><<<grid, block, 0, s>>>(a);
    else if (kind == kAttnE4m3) append_kernel<uint16_t, E4m3><<<grid, block, 0, s>>>(a);
    else append_kernel<uint16_t, uint16_t><<<grid, block, 0, s>>>(a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace lora
