// lora_attn_meta.hip -- attention metadata of one step: which keys every query
// token sees, and the work lists of the attention kernels.  Two launches:
//
//   attn_limits_kernel  one thread per token: its sequence (binary search in
//                       q_start), its position and the interval [lo, hi) of keys
//                       it sees.  Causality, the window, the prefix and the
//                       document bounds all come down to this one interval, so
//                       the attention kernels know no mask but it.
//   attn_plan_kernel    one workgroup: cuts the sequences (and the groups) into
//                       tiles, lays the keys of the few-row tiles end to end and
//                       cuts that line into equal slices, cuts the other tiles
//                       where they are too few to fill the chip, and writes the
//                       items and, for tokens whose result comes in parts, where
//                       the parts lie.
//
// The algorithm is in lora_attn_plan.h.  Both are bound by latency and shared by the
// layers of a step: 2 and 17 us for one sequence of 1000 keys (a thread writes its
// slices), 5 and 12 us for 256 decode tokens, 6 and 20 us for those of 512 and 4
// prompts of 1024, 5 and 42 us for 512 tiles of 128 rows (a thread reads a tile's
// intervals).
#include "lora_attn_host.h"
#include "lora_attn_plan.h"
#include "lora_common.h"

namespace lora {

namespace {

constexpr int kPlanThreads = 1024;

__global__ __launch_bounds__(256) void attn_limits_kernel(AttnPlanArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t < a.tokens) reinterpret_cast<AttnLimit *>(a.limits)[t] = limit_of(a, t);
}

// The plan's team: a workgroup.
struct BlockTeam {
  int *lds;  // one int a wave
  TeamShared *common;
  __device__ __forceinline__ int id() const { return threadIdx.x; }
  __device__ __forceinline__ int size() const { return kPlanThreads; }
  __device__ __forceinline__ void sync() const { __syncthreads(); }
  __device__ __forceinline__ TeamShared &shared() const { return *common; }
  __device__ __forceinline__ bool any(bool x) const { return __syncthreads_or(x); }
  // (atomics pass by the CU's cache, and so does this)
  __device__ __forceinline__ int read(const int *p) const {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  template <typename T>
  __device__ __forceinline__ void add(T *p, T v) const { atomicAdd(p, v); }
  __device__ int before(int v, int &total) const {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int inc = wave_inclusive_scan(v);
    __syncthreads();
    if (lane == kWave - 1) lds[wave] = inc;
    __syncthreads();
    int base = 0, sum = 0;
    for (int w = 0; w < kPlanThreads / kWave; ++w) {
      if (w == wave) base = sum;
      sum += lds[w];
    }
    total = sum;
    return base + inc - v;
  }
  __device__ int most_before(int v, int &total) const {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    int inc = v;
    for (int x = 1; x < kWave; x *= 2) {
      const int other = __shfl_up(inc, x);
      if (lane >= x) inc = max(inc, other);
    }
    const int before_lane = __shfl_up(inc, 1);
    __syncthreads();
    if (lane == kWave - 1) lds[wave] = inc;
    __syncthreads();
    int base = 0, most = 0;
    for (int w = 0; w < kPlanThreads / kWave; ++w) {
      if (w == wave) base = most;
      most = max(most, lds[w]);
    }
    total = most;
    return lane > 0 ? max(base, before_lane) : base;
  }
};

__global__ __launch_bounds__(kPlanThreads) void attn_plan_kernel(AttnPlanArgs a) {
  __shared__ int scan_lds[kPlanThreads / kWave];
  __shared__ TeamShared common;
  BlockTeam team{scan_lds, &common};
  attn_plan(a, team);
}

}  // namespace

hipError_t launch_attn_plan(const AttnPlanArgs &a, hipStream_t s) {
  if (a.tokens > 0) attn_limits_kernel<<<dim3((unsigned)((a.tokens + 255) / 256)), dim3(256), 0, s>>>(a);
  attn_plan_kernel<<<dim3(1), dim3(kPlanThreads), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace lora
