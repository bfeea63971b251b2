// lora_combine.hip -- the weighted sum of a token's expert outputs.
//
// Bound: HBM; the rows of a token's local choices are read once, its output written once.
// A thread takes 8 columns of a token; its choices are read eight at a time, so that a
// token's rows are all on their way at once.  The sum is in fp32, in ascending choice, then
// the row to add.  4608 tokens x 8 choices x 4096 columns bf16 and a row to add: 70 us, 5.4
// TB/s (71 with the eight waves a SIMD that its registers would allow); 256 tokens x 7168,
// an eighth of the choices local: 4.2 us, a launch and three dependent loads.
#include <algorithm>

#include "lora_base_host.h"

namespace lora {

namespace {

template <typename X>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 6))) void combine_kernel(CombineArgs a) {
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x % 64;
  // lane j of every wave looks choice j up
  bool here = false;
  float w = 0.f;
  if (lane < a.topk) {
    const int e = a.ids[t * a.topk + lane];
    w = a.weights[t * a.topk + lane];
    if (e >= 0 && e < a.experts) {
      const int l = a.map ? a.map[e] : e;
      here = l >= 0 && l < a.local;
    }
  }
  const uint64_t all = __ballot(here);
  // past the last column the last ones again, not stored: lanes hold weights that others read
  const int at = 8 * (blockIdx.y * 256 + threadIdx.x), c = min(at, a.width - 8);
  const X *y = reinterpret_cast<const X *>(a.y) + t * a.topk * a.ldy + c;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  // read along with the choices' rows, added last: the sum is rounded at its own size, not at this row's
  Raw8<X> base;
  base.zero();
  if (a.add) base.load(reinterpret_cast<const X *>(a.add) + t * a.ldadd + c);
  for (uint64_t left = all; left;) {
    Raw8<X> v[8];
    float by[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      by[q] = 0.f;
      if (left) {
        const int j = __builtin_ctzll(left);
        left &= left - 1;
        by[q] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), j));
        v[q].load(y + (int64_t)j * a.ldy);
      } else {
        v[q].zero();
      }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += by[q] * v[q][e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] += base[e];
  if (at < a.width) store8(reinterpret_cast<X *>(a.out) + t * a.ldout + c, sum);
}

}  // namespace

hipError_t launch_combine(const CombineArgs &all, bool bf16, hipStream_t s) {
  const int64_t esize = bf16 ? 2 : 4;
  const int cols = (all.width + 2047) / 2048;
  // workgroups of a launch, tokens times column blocks, stay below 2^23
  const int64_t most = std::max<int64_t>(1, ((int64_t)1 << 23) / cols);
  for (int64_t t0 = 0; t0 < all.tokens; t0 += most) {
    CombineArgs a = all;
    a.tokens = std::min(all.tokens - t0, most);
    a.y += t0 * a.topk * a.ldy * esize;
    a.ids += t0 * a.topk;
    a.weights += t0 * a.topk;
    if (a.add) a.add += t0 * a.ldadd * esize;
    a.out += t0 * a.ldout * esize;
    const dim3 grid((unsigned)a.tokens, (unsigned)cols);
    if (bf16) combine_kernel<uint16_t><<<grid, dim3(256), 0, s>>>(a);
    else combine_kernel<float><<<grid, dim3(256), 0, s>>>(a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace lora
