// lora_attn_meta.hip -- attention metadata of one step: which keys every query
// token sees, and the work lists of the attention kernels.  Two launches:
//
//   attn_limits_kernel  one thread per token: its sequence (binary search in
//                       q_start), its position and the interval [lo, hi) of keys
//                       it sees.  Causality, the window, the prefix and the
//                       document bounds all come down to this one interval, so
//                       the attention kernels know no mask but it.
//   attn_plan_kernel    one workgroup: cuts the sequences (and the groups) into
//                       tiles, sums up their keys, cuts every tile's keys into
//                       ranges of one common length so that the items are alike
//                       whatever the lengths, and writes the items and, for
//                       tokens whose result comes in parts, where the parts lie.
//
// Both are latency-bound (a few microseconds) and shared by the layers of a step.
#include "lora_attn.h"
#include "lora_attn_host.h"
#include "lora_common.h"

namespace lora {

namespace {

constexpr int kPlanThreads = 1024;

// Query tokens of sequence n as [q0, q1), empty if the bounds are not in order.
__device__ __forceinline__ void seq_tokens(const AttnPlanArgs &a, int n, int64_t &q0, int64_t &q1) {
  q0 = a.q_start[n];
  q1 = a.q_start[n + 1];
  if (q0 < 0 || q1 < q0 || q1 > a.tokens) q0 = q1 = 0;
}

// Whether sequence n is usable (see lora_attn_batch).
__device__ __forceinline__ bool seq_ok(const AttnPlanArgs &a, int n) {
  const int64_t q0 = a.q_start[n], q1 = a.q_start[n + 1], kv = a.kv_len[n];
  return q0 >= 0 && q1 >= q0 && q1 <= a.tokens && q1 - q0 <= a.max_q_len && kv >= q1 - q0 &&
         kv <= a.table_stride * a.page_size;
}

__device__ __forceinline__ bool group_ok(const AttnPlanArgs &a, int g) {
  const int s0 = a.group_start[g], s1 = a.group_start[g + 1], len = a.group_len[g];
  if (s0 < 0 || s1 < s0 || s1 > a.seqs || len < 0) return false;
  return s0 == s1 || (seq_ok(a, s0) && len <= a.kv_len[s0]);
}

// Group of sequence n, or -1: the last group that starts at or before n.
__device__ __forceinline__ int group_of(const AttnPlanArgs &a, int n) {
  int lo = 0, hi = a.groups;  // first group that starts after n
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.group_start[mid] <= n) lo = mid + 1;
    else hi = mid;
  }
  const int g = lo - 1;
  if (g < 0 || n >= a.group_start[g + 1] || !group_ok(a, g) || a.group_len[g] == 0) return -1;
  return g;
}

__global__ __launch_bounds__(256) void attn_limits_kernel(AttnPlanArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= a.tokens) return;
  int lo = 0, hi = a.seqs;  // first sequence whose tokens start after t
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.q_start[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  const int n = lo - 1;
  int32_t key0 = 0, key1 = 0, p = 0;
  int32_t seq = -1;
  if (n >= 0 && t < a.q_start[n + 1]) {
    seq = n;
    if (seq_ok(a, n)) {
      const int kv = a.kv_len[n];
      p = (int)(kv - a.q_start[n + 1] + t);
      key1 = a.causal ? p + 1 : kv;
      if (a.prefix_len) key1 = max(key1, a.prefix_len[n]);
      if (a.window > 0) key0 = max(0, p + 1 - a.window);
      if (a.key_lo) key0 = max(key0, a.key_lo[t]);
      if (a.key_hi) key1 = min(key1, a.key_hi[t]);
      key1 = min(key1, kv);
      if (key1 <= key0) key0 = key1 = 0;
    }
  }
  int4 v = {key0, key1, p, seq};
  reinterpret_cast<int4 *>(a.limits)[t] = v;
}

// Exclusive prefix sum over the workgroup's threads, and the sum of all.
__device__ int block_scan(int v, int *lds, int &total) {
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

// Last entry of base[0 .. n] (non-decreasing) that is <= i, for base[0] <= i.
__device__ __forceinline__ int last_at_or_before(const int32_t *base, int n, int i) {
  int lo = 0, hi = n + 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (base[mid] <= i) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

__global__ __launch_bounds__(kPlanThreads) void attn_plan_kernel(AttnPlanArgs a) {
  __shared__ int scan_lds[kPlanThreads / kWave];
  __shared__ unsigned long long sum_lds[2];
  __shared__ int bad_lds[2];
  const int tid = threadIdx.x;
  if (tid < 2) sum_lds[tid] = 0, bad_lds[tid] = 0;
  __syncthreads();

  // ---- tiles per sequence, then per group
  const int few_tokens = kFewRows / a.group, tile_tokens = a.tile_rows / a.group;
  int own = 0;
  for (int n0 = 0; n0 < a.seqs; n0 += kPlanThreads) {
    const int n = n0 + tid;
    int count = 0;
    if (n < a.seqs) {
      int64_t q0, q1;
      seq_tokens(a, n, q0, q1);
      const int len = (int)(q1 - q0);
      count = len <= few_tokens ? (len > 0) : (len + tile_tokens - 1) / tile_tokens;
      if (!seq_ok(a, n)) atomicAdd(&bad_lds[0], 1);
    }
    int total;
    const int before = block_scan(count, scan_lds, total);
    if (n < a.seqs) a.seq_base[n] = min(own + before, a.max_tiles);
    own = min(own + total, a.max_tiles);
  }
  int tiles = own;
  for (int g0 = 0; g0 < a.groups; g0 += kPlanThreads) {
    const int g = g0 + tid;
    int count = 0;
    if (g < a.groups) {
      if (!group_ok(a, g)) {
        atomicAdd(&bad_lds[1], 1);
      } else if (a.group_len[g] > 0 && a.group_start[g] < a.group_start[g + 1]) {
        const int64_t q0 = a.q_start[a.group_start[g]], q1 = a.q_start[a.group_start[g + 1]];
        const int len = q0 >= 0 && q1 >= q0 && q1 <= a.tokens ? (int)(q1 - q0) : 0;
        count = len <= few_tokens ? (len > 0) : (len + tile_tokens - 1) / tile_tokens;
      }
    }
    int total;
    const int before = block_scan(count, scan_lds, total);
    if (g < a.groups) a.group_base[g] = min(tiles + before, a.max_tiles);
    tiles = min(tiles + total, a.max_tiles);
  }
  __syncthreads();  // the bases are written (one workgroup: its own stores)
  __threadfence_block();

  // ---- the tiles' tokens and keys
  unsigned long long keys[2] = {0, 0};
  for (int i = tid; i < tiles; i += kPlanThreads) {
    AttnTile r;
    int64_t q0, q1;
    int first = 0, shared_len = 0;
    r.shared = 0;
    if (i < own) {
      const int n = last_at_or_before(a.seq_base, a.seqs - 1, i);
      seq_tokens(a, n, q0, q1);
      first = a.seq_base[n];
      r.seq = n;
      const int g = a.groups ? group_of(a, n) : -1;
      if (g >= 0) {
        r.shared = 2;
        shared_len = a.group_len[g];
      }
    } else {
      const int g = last_at_or_before(a.group_base, a.groups - 1, i);
      first = a.group_base[g];
      r.seq = a.group_start[g];
      q0 = a.q_start[r.seq];
      q1 = a.q_start[a.group_start[g + 1]];
      r.shared = 1;
      shared_len = a.group_len[g];
    }
    const int len = (int)(q1 - q0), part = i - first;
    r.few = len <= few_tokens || a.tile_rows == kFewRows;
    const int per = r.few ? few_tokens : tile_tokens;
    r.tok0 = (int)q0 + part * per;
    r.ntok = max(0, min(per, len - part * per));
    int lo_min = 0x7fffffff, lo_max = 0, hi_min = 0x7fffffff, hi_max = 0;
    for (int t = 0; t < r.ntok; ++t) {
      const int4 v = reinterpret_cast<const int4 *>(a.limits)[r.tok0 + t];
      if (v.y > v.x) {
        lo_min = min(lo_min, v.x);
        hi_max = max(hi_max, v.y);
      }
      lo_max = max(lo_max, v.x);
      hi_min = min(hi_min, v.y);
    }
    r.key0 = r.shared == 2 ? max(lo_min, shared_len) : lo_min;
    r.key1 = r.shared == 1 ? min(hi_max, shared_len) : hi_max;
    if (r.key1 <= r.key0) r.key0 = r.key1 = 0;
    r.full0 = lo_max;
    r.full1 = hi_min;
    r.splits = r.unit0 = r.pad = 0;
    reinterpret_cast<AttnTile *>(a.tiles)[i] = r;
    keys[r.few ? 0 : 1] += (unsigned long long)(r.key1 - r.key0);
  }
  for (int c = 0; c < 2; ++c)
    if (keys[c]) atomicAdd(&sum_lds[c], keys[c]);
  __threadfence_block();
  __syncthreads();
  const int few_keys = keys_per_item((int64_t)sum_lds[0], a.heads, kFewTarget, kFewMinKeys);
  const int tile_keys = keys_per_item((int64_t)sum_lds[1], a.heads, kTileTarget, kTileMinKeys);

  // ---- items, partial-result units, tokens to join
  int few_items = 0, tile_items = 0, units = 0, joins = 0;
  for (int i0 = 0; i0 < tiles; i0 += kPlanThreads) {
    const int i = i0 + tid;
    AttnTile r;
    int splits = 0, per = 1, ups = 0;
    bool parts = false;
    if (i < tiles) {
      r = reinterpret_cast<const AttnTile *>(a.tiles)[i];
      per = r.few ? few_keys : tile_keys;
      splits = max(1, (r.key1 - r.key0 + per - 1) / per);
      parts = splits > 1 || r.shared;
      ups = (r.ntok * a.group + kUnitRows - 1) / kUnitRows;
    }
    const bool few = i < tiles && r.few;
    int nf, nt, nu, nj;
    int at_few = few_items + block_scan(few ? splits : 0, scan_lds, nf);
    int at_tile = tile_items + block_scan(few ? 0 : splits, scan_lds, nt);
    int unit = units + block_scan(parts ? splits * ups : 0, scan_lds, nu);
    int join = joins + block_scan(parts && r.shared != 1 ? r.ntok : 0, scan_lds, nj);
    if (i < tiles) {
      // never true for the sizes the capacities are derived from; with a
      // q_start that is out of order the surplus is dropped
      const bool fits = (few ? at_few + splits <= a.max_few_items : at_tile + splits <= a.max_tile_items) &&
                        unit + splits * ups <= a.max_units;
      AttnItem *items = reinterpret_cast<AttnItem *>(few ? a.few_items : a.tile_items);
      int at = few ? at_few : at_tile;
      const int cap = few ? a.max_few_items : a.max_tile_items;
      for (int s = 0; s < splits && at < cap; ++s, ++at) {
        const int k0 = r.key0 + s * per;
        items[at] = AttnItem{r.tok0, fits ? r.ntok : 0, r.seq, k0, min(r.key1, k0 + per), r.full0, r.full1,
                             parts ? unit + s * ups : -1};
      }
      if (parts) {
        for (int t = 0; t < r.ntok; ++t) {
          int4 *rec = reinterpret_cast<int4 *>(a.join) + 2 * (int64_t)(r.tok0 + t);
          rec[r.shared == 1] = int4{unit, fits ? splits : 0, ups, t};
          if (r.shared == 0) rec[1] = int4{0, 0, 0, 0};
          if (r.shared != 1 && join + t < a.tokens) a.join_tokens[join + t] = r.tok0 + t;
        }
      }
    }
    few_items += nf;
    tile_items += nt;
    units += nu;
    joins += nj;
  }
  if (tid == 0) {
    a.info[0] = min(few_items, a.max_few_items);
    a.info[1] = min(tile_items, a.max_tile_items);
    a.info[2] = bad_lds[0];
    a.info[3] = bad_lds[1];
    a.info[4] = (int)min((int64_t)joins, a.tokens);
    a.info[5] = min(units, a.max_units);
    a.info[6] = few_keys;
    a.info[7] = tile_keys;
    for (int k = 8; k < kAttnInfoInts; ++k) a.info[k] = 0;
  }
}

}  // namespace

hipError_t launch_attn_plan(const AttnPlanArgs &a, hipStream_t s) {
  if (a.tokens > 0) attn_limits_kernel<<<dim3((unsigned)((a.tokens + 255) / 256)), dim3(256), 0, s>>>(a);
  attn_plan_kernel<<<dim3(1), dim3(kPlanThreads), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace lora
