// lora_attn.hip -- the attention kernels: the few-row and the tile work of a call
// in one launch, and the kernel that joins partial results.
//
// Few-row work is bound by HBM and tile work by the matrix cores, so a batch that
// has both runs them side by side: the slices' workgroups come first, one per CU,
// and the tile items' fill the CUs' second places.  Slices are alike by
// construction, so each has one wave.  Tile items are taken longest first,
// by as many workgroups as there are items, or in rounds beyond kMaxTileBlocks.
//
// Measured: 512 decode tokens (window 1024) and 4 prompts of 1024, 350 to 354 us (347
// before the slices took weights of two terms, alone 287 then, and the tiles alone 96); 8 and 8 workgroups of the two
// kinds in turn leave places empty where one kind has no work (a long prompt took
// 3268 instead of 2630 us), tiles first take 454 us on the mixed batch.
#include <algorithm>

#include "lora_attn_few.h"
#include "lora_attn_tile.h"

namespace lora {

namespace {

// Rows up to which the waves of a workgroup share a row's parts in the join.
constexpr int64_t kJoinShared = 1024;

__host__ __device__ inline int few_blocks(const AttnArgs &a) { return (a.few_waves + 3) / 4; }

// A wave's slice: f(item, head group) for each of its items.
template <typename F>
__device__ __forceinline__ void run_slice(const AttnArgs &a, F &&f) {
  const int w = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + threadIdx.x / kWave);
  if (w >= a.few_waves) return;
  const int slot = a.by_heads.quotient(w), h = w - slot * a.heads;
  const int32_t *p = a.slots + (int64_t)slot * kAttnSlotInts;
  const int first = p[0], end = p[1];
  AttnItem it{p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11]};
  for (int i = first; i < end; ++i) {
    if (i > first) it = load_item(a.few_items, i);
    f(it, h);
  }
}
template <int DP, bool FP8, bool GENERAL>
__device__ __forceinline__ void run_few_slice(const AttnArgs &a, uint16_t *v) {
  run_slice(a, [&](const AttnItem &it, int h) {
    if (run_few<DP, FP8, GENERAL, false>(a, it, h, v)) run_few<DP, FP8, GENERAL, true>(a, it, h, v);
  });
}

// Slices only (decode).
template <int DP, bool FP8, bool GENERAL>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void attn_few_kernel(AttnArgs a) {
  __shared__ __align__(16) uint16_t lds[4 * FewShape<DP, FP8>::REGION];
  run_few_slice<DP, FP8, GENERAL>(a, lds + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * FewShape<DP, FP8>::REGION);
}

template <int DP, bool GENERAL>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void attn_few_f32_kernel(AttnArgs a) {
  run_slice(a, [&](const AttnItem &it, int h) { run_few_f32<DP, GENERAL>(a, it, h); });
}

template <int DP, bool FP8, bool GENERAL>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void attn_both_kernel(AttnArgs a) {
  constexpr int kK = kKeys * TileShape<DP, FP8>::LDK, kV = kKeys * TileShape<DP, FP8>::LDV;
  static_assert(FewShape<DP, FP8>::REGION <= kK && kK <= kV, "a few-row wave's V rows fit one of these");
  __shared__ __align__(16) uint16_t k0[kK], k1[kK], v0[kV], v1[kV];
  __shared__ int good_lds[kKeys], flag_lds[1];
  const TileLds lds{k0, k1, v0, v1, good_lds, flag_lds};
  const int few_end = (few_blocks(a) + 7) / 8 * 8, index = (int)blockIdx.x - few_end;
  if (index < 0) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    run_few_slice<DP, FP8, GENERAL>(a, wave == 0 ? k0 : wave == 1 ? k1 : wave == 2 ? v0 : v1);
    return;
  }
  if (index >= a.tile_blocks) return;
  const int first = a.by_heads.quotient(index), h = index - first * a.heads, items = a.info[1];
  const int step = a.by_heads.quotient(a.tile_blocks);
  // the longest ranges of a causal prompt come last in the list and run first
  for (int i = first; i < items; i += step) {
    if (i != first) __syncthreads();
    const AttnItem it = load_item(a.tile_items, items - 1 - i);
    if (run_tile<DP, FP8, GENERAL, false>(a, it, h, lds)) run_tile<DP, FP8, GENERAL, true>(a, it, h, lds);
  }
}

// Rows whose result lies in parts: for each (token, query head) the parts of its
// group's shared keys and of its own, weighted by their sums, are added in the
// order of the keys.  Bound by latency (three dependent loads) for few rows and by
// L2 for many: lane p looks up part p, and the first parts' outputs, 64 / LANES
// side by side and 8 loads a lane, are on their way while the parts' maxima are
// reduced.  WAVES = 1: a wave per row; 4: the workgroup's waves share a row's
// parts, where rows are too few to fill the chip.
template <int LANES, int WAVES, typename OUT>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  constexpr int SIDE = kWave / LANES;  // parts read side by side
  constexpr int DEEP = 8;              // loads in flight a lane
  __shared__ float share[4][LANES * 4 + 2];
  const int lane = threadIdx.x % kWave, side = lane / LANES, d = 4 * (lane % LANES);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t step = gridDim.x * (4 / WAVES);
  uint32_t r = WAVES == 1 ? blockIdx.x * 4 + wave : blockIdx.x;
  // the first row's record is read before it is known whether there is one
  auto entry = [&](uint32_t row) {
    const int64_t j = min((int64_t)a.by_q_heads.quotient(row), a.tokens - 1);
    return reinterpret_cast<const int4 *>(a.join_list + kAttnJoinInts * j);
  };
  const int4 *e = entry(r);
  int t = e[0].x;
  int4 own = e[1], pre = e[2];
  const uint32_t rows = (uint32_t)a.info[4] * a.q_heads;
  for (; r < rows; r += step) {
    const int qh = r - a.by_q_heads.quotient(r) * a.q_heads, h = a.by_group.quotient(qh), of_group = qh - h * a.group;
    // this wave's parts: begin .. n - 1
    const int all = own.y + pre.y, per = (all + WAVES - 1) / WAVES;
    const int begin = WAVES == 1 ? 0 : min(wave * per, all), n = WAVES == 1 ? all : min(begin + per, all);
    float m = kNegInf, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int p0 = begin; p0 < n; p0 += kWave) {
      // lane p: where part p0 + p lies, its maximum and sum
      const int p = min(p0 + lane, n - 1), count = min(kWave, n - p0);
      const bool shared = p < pre.y;
      const int4 rec = shared ? pre : own;
      const int row = rec.w * a.group + of_group;
      const int64_t pr = part_row(a, rec.x + (int64_t)(shared ? p : p - pre.y) * rec.z + row / kUnitRows, h, row % kUnitRows);
      const float pm = p0 + lane < n ? a.part_ml[2 * pr] : kNegInf, pl = a.part_ml[2 * pr + 1];
      f32x4 v[DEEP];
      auto fetch = [&](int q) {
#pragma unroll
        for (int u = 0; u < DEEP; ++u)
          if (q + SIDE * u < count)
            v[u] = gload16f(a.part + __shfl(pr, min(q + SIDE * u + side, count - 1)) * a.dim + (d < a.dim ? d : 0));
      };
      fetch(0);
      float top = fmaxf(m, pm);
#pragma unroll
      for (int x = 1; x < 16; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
      top = max_rows(top);
      const float base = top == kNegInf ? 0.f : top;
      const float fade = exp2_fast(m - base);
      // a part in which no key is seen has -inf and 0
      const float f = p0 + lane < n ? exp2_fast(pm - base) : 0.f;
      m = top;
      float add = p0 + lane < n ? f * pl : 0.f;
#pragma unroll
      for (int x = 1; x < 16; x *= 2) add += __shfl_xor(add, x);
      l = l * fade + sum_rows(add);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] *= fade;
      for (int q = 0; q < count; q += DEEP * SIDE) {
        if (q) fetch(q);
#pragma unroll
        for (int u = 0; u < DEEP; ++u)
          if (q + SIDE * u < count) {
            const int from = q + SIDE * u + side;
            const float w = __shfl(f, min(from, count - 1));
            if (from < count) {
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] += w == 0.f ? 0.f : w * v[u][i];
            }
          }
      }
    }
#pragma unroll
    for (int x = LANES; x < kWave; x *= 2)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += __shfl_xor(o[i], x);
    if constexpr (WAVES > 1) {
      __syncthreads();  // the last row's shares are read
      if (side == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) share[wave][d + i] = o[i];
      }
      if (lane == 0) share[wave][LANES * 4] = m, share[wave][LANES * 4 + 1] = l;
      __syncthreads();
      float top = kNegInf;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) top = fmaxf(top, share[w][LANES * 4]);
      const float base = top == kNegInf ? 0.f : top;
      m = top, l = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const float f = exp2_fast(share[w][LANES * 4] - base);
        l += f * share[w][LANES * 4 + 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += f == 0.f ? 0.f : f * share[w][d + i];
      }
    }
    const float mul = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = mul == 0.f ? 0.f : o[i] * mul;
    const bool writes = WAVES == 1 || wave == 0;
    if (writes && side == 0 && d < a.dim) {
      const int64_t at = t * a.ldo + (int64_t)qh * a.dim + d;
      if constexpr (sizeof(OUT) == 4) {
        gstore16f(a.out + 4 * at, f32x4{o[0], o[1], o[2], o[3]});
      } else {
        typedef __attribute__((address_space(1))) u32x2 g_u32x2;
        *(g_u32x2 *)(a.out + 2 * at) = u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
      }
    }
    if (writes && lane == 0 && a.lse)
      a.lse[(int64_t)t * a.q_heads + qh] = l == 0.f ? kNegInf : (m + __log2f(l)) * kLn2;
    if (r + step < rows) {
      e = entry(r + step);
      t = e[0].x, own = e[1], pre = e[2];
    }
  }
}

template <int DP, bool FP8, bool GENERAL>
void start(const AttnArgs &a, hipStream_t s) {
  if (a.tile_blocks == 0) {
    attn_few_kernel<DP, FP8, GENERAL><<<dim3(few_blocks(a)), dim3(256), 0, s>>>(a);
  } else {
    const unsigned grid = 8 * ((few_blocks(a) + 7) / 8 + (a.tile_blocks + 7) / 8);
    attn_both_kernel<DP, FP8, GENERAL><<<dim3(grid), dim3(256), 0, s>>>(a);
  }
}

template <int DP>
void start(const AttnArgs &a, AttnKind kind, hipStream_t s) {
  // the plain form supposes a positive factor (hidden scores are -inf before it)
  const bool general = a.cap > 0.f || a.slopes || !(a.scale > 0.f);
  if (kind == kAttnF32) {
    if (general) attn_few_f32_kernel<DP, true><<<dim3(few_blocks(a)), dim3(256), 0, s>>>(a);
    else attn_few_f32_kernel<DP, false><<<dim3(few_blocks(a)), dim3(256), 0, s>>>(a);
  } else if (kind == kAttnE4m3) {
    general ? start<DP, true, true>(a, s) : start<DP, true, false>(a, s);
  } else {
    general ? start<DP, false, true>(a, s) : start<DP, false, false>(a, s);
  }
}

template <int WAVES, typename OUT>
void start_join(const AttnArgs &a, unsigned grid, hipStream_t s) {
  if (a.dim <= 64) attn_join_kernel<16, WAVES, OUT><<<dim3(grid), dim3(256), 0, s>>>(a);
  else if (a.dim <= 128) attn_join_kernel<32, WAVES, OUT><<<dim3(grid), dim3(256), 0, s>>>(a);
  else attn_join_kernel<64, WAVES, OUT><<<dim3(grid), dim3(256), 0, s>>>(a);
}
template <typename OUT>
void start_join(const AttnArgs &a, hipStream_t s) {
  // a row per workgroup where they fit the chip together
  const int64_t rows = a.tokens * a.q_heads;
  if (rows <= kJoinShared) start_join<4, OUT>(a, (unsigned)rows, s);
  else start_join<1, OUT>(a, (unsigned)std::min<int64_t>((rows + 3) / 4, 2048), s);
}

}  // namespace

hipError_t launch_attn(const AttnArgs &a, AttnKind kind, hipStream_t s) {
  if (a.dim <= 64) start<64>(a, kind, s);
  else if (a.dim <= 128) start<128>(a, kind, s);
  else start<256>(a, kind, s);
  return hipGetLastError();
}

hipError_t launch_attn_join(const AttnArgs &a, AttnKind kind, hipStream_t s) {
  if (kind == kAttnF32) start_join<float>(a, s);
  else start_join<uint16_t>(a, s);
  return hipGetLastError();
}

}  // namespace lora
