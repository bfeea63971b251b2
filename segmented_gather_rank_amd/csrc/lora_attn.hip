// lora_attn.hip -- the attention kernels: the few-row and the tile work of a call
// in one launch, and the kernel that joins partial results.
//
// Few-row work is bound by HBM and tile work by the matrix cores, so a batch that
// has both runs them side by side: the slices' workgroups come first, one per CU,
// and the tile items' fill the CUs' second places.  Slices are alike by
// construction, so each has one workgroup.  Tile items are taken longest first,
// by as many workgroups as there are items, or in rounds beyond kMaxTileBlocks.
#include "lora_attn_few.h"
#include "lora_attn_tile.h"

namespace lora {

namespace {

template <int DP, bool FP8, bool GENERAL>
__device__ __forceinline__ void run_slot(const AttnArgs &a, int index, char *lds, float (*ml_lds)[16][2]) {
  const int h = index % a.heads;
  const int32_t *p = a.slots + (int64_t)(index / a.heads) * kAttnSlotInts;
  const int first = p[0], end = p[1];
  AttnItem it{p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11]};
  for (int i = first; i < end; ++i) {
    if (i > first) {
      __syncthreads();  // the last item's results are read
      it = load_item(a.few_items, i);
    }
    if (run_few<DP, FP8, GENERAL, false>(a, it, h, lds, ml_lds)) run_few<DP, FP8, GENERAL, true>(a, it, h, lds, ml_lds);
  }
}

// Slices only (decode).
template <int DP, bool FP8, bool GENERAL>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void attn_few_kernel(AttnArgs a) {
  __shared__ __align__(16) char lds[4 * FewShape<DP, FP8>::REGION];
  __shared__ float ml_lds[4][16][2];
  run_slot<DP, FP8, GENERAL>(a, blockIdx.x, lds, ml_lds);
}

template <int DP, bool GENERAL>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void attn_few_f32_kernel(AttnArgs a) {
  __shared__ __align__(16) char lds[4 * 16 * (DP + 4) * 4];
  __shared__ float ml_lds[4][16][2];
  const int h = blockIdx.x % a.heads;
  const int32_t *p = a.slots + (int64_t)(blockIdx.x / a.heads) * kAttnSlotInts;
  const int first = p[0], end = p[1];
  for (int i = first; i < end; ++i) {
    if (i > first) __syncthreads();
    run_few_f32<DP, GENERAL>(a, load_item(a.few_items, i), h, lds, ml_lds);
  }
}

template <int DP, bool FP8, bool GENERAL>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void attn_both_kernel(AttnArgs a) {
  constexpr int kFewLds = 4 * FewShape<DP, FP8>::REGION, kTileLds = 4 * TileShape<DP, FP8>::BUF;
  __shared__ __align__(16) char lds[kFewLds > kTileLds ? kFewLds : kTileLds];
  __shared__ float ml_lds[4][16][2];
  __shared__ int flag_lds[4];
  const int few_end = (a.few_blocks + 7) / 8 * 8, index = (int)blockIdx.x - few_end;
  if (index < 0) {
    if ((int)blockIdx.x < a.few_blocks) run_slot<DP, FP8, GENERAL>(a, blockIdx.x, lds, ml_lds);
    return;
  }
  if (index >= a.tile_blocks) return;
  const int h = index % a.heads, items = a.info[1];
  // the longest ranges of a causal prompt come last in the list and run first
  for (int i = index / a.heads; i < items; i += a.tile_blocks / a.heads) {
    if (i != index / a.heads) __syncthreads();
    const AttnItem it = load_item(a.tile_items, items - 1 - i);
    uint16_t *buf = reinterpret_cast<uint16_t *>(lds);
    if (run_tile<DP, FP8, GENERAL, false>(a, it, h, buf, flag_lds)) run_tile<DP, FP8, GENERAL, true>(a, it, h, buf, flag_lds);
  }
}

// Rows whose result lies in parts: one wave per (token, query head) adds the
// parts of its group's shared keys and of its own, weighted by their sums, in
// the order of the keys.  Bound by latency (five dependent loads) for a few rows
// and by L2 for many: lane p looks up part p, then 64 / LANES parts' outputs are
// read at a time, four rounds in flight.
template <int LANES, typename OUT>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  constexpr int SIDE = kWave / LANES;  // parts read side by side
  const int lane = threadIdx.x % kWave, side = lane / LANES, d = 4 * (lane % LANES);
  const int64_t rows = (int64_t)a.info[4] * a.q_heads;
  for (int64_t r = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave; r < rows; r += (int64_t)gridDim.x * 4) {
    const int t = __builtin_amdgcn_readfirstlane(a.join_tokens[r / a.q_heads]);
    const int qh = __builtin_amdgcn_readfirstlane((int)(r % a.q_heads));
    const int h = qh / a.group;
    const int4 own = reinterpret_cast<const int4 *>(a.join)[2 * (int64_t)t];
    const int4 pre = reinterpret_cast<const int4 *>(a.join)[2 * (int64_t)t + 1];
    const int n = own.y + pre.y;
    float m = kNegInf, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int p0 = 0; p0 < n; p0 += kWave) {
      // lane p: where part p0 + p lies, its maximum and sum
      const int p = min(p0 + lane, n - 1);
      const bool shared = p < pre.y;
      const int4 rec = shared ? pre : own;
      const int row = rec.w * a.group + qh % a.group;
      const int64_t pr = part_row(a, rec.x + (int64_t)(shared ? p : p - pre.y) * rec.z + row / kUnitRows, h, row % kUnitRows);
      const float pm = p0 + lane < n ? a.part_ml[2 * pr] : kNegInf, pl = a.part_ml[2 * pr + 1];
      float top = fmaxf(m, pm);
#pragma unroll
      for (int x = 1; x < kWave; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
      const float base = top == kNegInf ? 0.f : top;
      const float fade = exp2_fast(m - base);
      // a part in which no key is seen has -inf and 0; with NaN it stays NaN
      const float f = p0 + lane < n ? exp2_fast(pm - base) : 0.f;
      m = top;
      float add = p0 + lane < n ? f * pl : 0.f;
#pragma unroll
      for (int x = 1; x < kWave; x *= 2) add += __shfl_xor(add, x);
      l = l * fade + add;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] *= fade;
      const int count = min(kWave, n - p0);
      for (int q = 0; q < count; q += 4 * SIDE) {
        f32x4 v[4];
        float w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int from = min(q + SIDE * u + side, count - 1);
          const int64_t at = __shfl(pr, from);
          w[u] = __shfl(f, from);
          if (q + SIDE * u + side >= count) w[u] = 0.f;
          v[u] = gload16f(a.part + at * a.dim + (d < a.dim ? d : 0));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] += w[u] == 0.f ? 0.f : w[u] * v[u][i];
      }
    }
#pragma unroll
    for (int x = LANES; x < kWave; x *= 2)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += __shfl_xor(o[i], x);
    const float mul = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = mul == 0.f ? 0.f : o[i] * mul;
    if (side == 0 && d < a.dim) {
      const int64_t at = t * a.ldo + (int64_t)qh * a.dim + d;
      if constexpr (sizeof(OUT) == 4) {
        gstore16f(a.out + 4 * at, f32x4{o[0], o[1], o[2], o[3]});
      } else {
        typedef __attribute__((address_space(1))) u32x2 g_u32x2;
        *(g_u32x2 *)(a.out + 2 * at) = u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
      }
    }
    if (lane == 0 && a.lse) a.lse[(int64_t)t * a.q_heads + qh] = l == 0.f ? kNegInf : (m + __log2f(l)) * kLn2;
  }
}

template <int DP, bool FP8, bool GENERAL>
void start(const AttnArgs &a, hipStream_t s) {
  if (a.tile_blocks == 0) {
    attn_few_kernel<DP, FP8, GENERAL><<<dim3(a.few_blocks), dim3(256), 0, s>>>(a);
  } else {
    const unsigned grid = 8 * ((a.few_blocks + 7) / 8 + (a.tile_blocks + 7) / 8);
    attn_both_kernel<DP, FP8, GENERAL><<<dim3(grid), dim3(256), 0, s>>>(a);
  }
}

template <int DP>
void start(const AttnArgs &a, AttnKind kind, hipStream_t s) {
  // the plain form supposes a positive factor (hidden scores are -inf before it)
  const bool general = a.cap > 0.f || a.slopes || !(a.scale > 0.f);
  if (kind == kAttnF32) {
    if (general) attn_few_f32_kernel<DP, true><<<dim3(a.few_blocks), dim3(256), 0, s>>>(a);
    else attn_few_f32_kernel<DP, false><<<dim3(a.few_blocks), dim3(256), 0, s>>>(a);
  } else if (kind == kAttnE4m3) {
    general ? start<DP, true, true>(a, s) : start<DP, true, false>(a, s);
  } else {
    general ? start<DP, false, true>(a, s) : start<DP, false, false>(a, s);
  }
}

template <typename OUT>
void start_join(const AttnArgs &a, hipStream_t s) {
  const int64_t blocks = (a.tokens * a.q_heads + 3) / 4;
  const dim3 grid((unsigned)(blocks < 2048 ? blocks : 2048));
  if (a.dim <= 64) attn_join_kernel<16, OUT><<<grid, dim3(256), 0, s>>>(a);
  else if (a.dim <= 128) attn_join_kernel<32, OUT><<<grid, dim3(256), 0, s>>>(a);
  else attn_join_kernel<64, OUT><<<grid, dim3(256), 0, s>>>(a);
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
