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
// Both are bound by latency and shared by the layers of a step: 4 and 9 us for one
// sequence, 6 and 21 us for 512 decode tokens and 4 prompts of 1024, 5 and 33 us
// for 67 tiles of 128 tokens (a thread reads a tile's intervals).
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

__global__ __launch_bounds__(kPlanThreads) void attn_plan_kernel(AttnPlanArgs a) {
  __shared__ int scan_lds[kPlanThreads / kWave];
  __shared__ unsigned long long sum_lds;
  __shared__ int bad_lds[2];
  const int tid = threadIdx.x;
  if (tid == 0) sum_lds = 0;
  if (tid < 2) bad_lds[tid] = 0;
  __syncthreads();

  // ---- tiles per sequence, then per group: which one, and which of its tiles
  const int few_tokens = kFewRows / a.group, tile_tokens = a.tile_rows / a.group;
  AttnTile *tile_list = reinterpret_cast<AttnTile *>(a.tiles);
  int own = 0, tiles = 0;
  for (int pass = 0; pass < 2; ++pass) {
    const int count_all = pass ? a.groups : a.seqs;
    for (int n0 = 0; n0 < count_all; n0 += kPlanThreads) {
      const int n = n0 + tid;
      int count = 0;
      if (n < count_all) {
        int64_t q0 = 0, q1 = 0;
        if (pass == 0) {
          seq_tokens(a, n, q0, q1);
          if (!seq_ok(a, n)) atomicAdd(&bad_lds[0], 1);
        } else if (!group_ok(a, n)) {
          atomicAdd(&bad_lds[1], 1);
        } else if (a.group_len[n] > 0 && a.group_start[n] < a.group_start[n + 1]) {
          q0 = a.q_start[a.group_start[n]];
          q1 = a.q_start[a.group_start[n + 1]];
          if (q0 < 0 || q1 < q0 || q1 > a.tokens) q0 = q1 = 0;
        }
        const int len = (int)(q1 - q0);
        count = len <= few_tokens ? (len > 0) : (len + tile_tokens - 1) / tile_tokens;
      }
      int total;
      const int before = tiles + block_scan(count, scan_lds, total);
      for (int i = 0; i < count && before + i < a.max_tiles; ++i) {
        tile_list[before + i].seq = n;
        tile_list[before + i].part = i;
      }
      tiles = min(tiles + total, a.max_tiles);
    }
    if (pass == 0) own = tiles;
  }
  __syncthreads();  // the list is written and read by this workgroup alone

  // ---- the tiles' tokens and keys; few-row tiles take their place on the line
  long long line = 0;
  unsigned long long keys = 0;
  for (int i0 = 0; i0 < tiles; i0 += kPlanThreads) {
    const int i = i0 + tid;
    AttnTile r;
    r.few = 0;
    int width = 0;
    if (i < tiles) {
      const int n = tile_list[i].seq, part = tile_list[i].part;
      int64_t q0, q1;
      int shared_len = 0;
      r.shared = 0;
      r.seq = n;
      if (i < own) {
        seq_tokens(a, n, q0, q1);
        const int g = a.groups ? group_of(a, n) : -1;
        if (g >= 0) {
          r.shared = 2;
          shared_len = a.group_len[g];
        }
      } else {
        r.seq = a.group_start[n];
        q0 = a.q_start[r.seq];
        q1 = a.q_start[a.group_start[n + 1]];
        r.shared = 1;
        shared_len = a.group_len[n];
      }
      const int len = (int)(q1 - q0);
      r.few = len <= few_tokens || a.tile_rows == kFewRows;
      const int per = r.few ? few_tokens : tile_tokens;
      r.tok0 = (int)q0 + part * per;
      r.ntok = max(0, min(per, len - part * per));
      int lo_min = 0x7fffffff, lo_max = 0, hi_min = 0x7fffffff, hi_max = 0;
      const int4 *lim = reinterpret_cast<const int4 *>(a.limits) + r.tok0;
      for (int t0 = 0; t0 < r.ntok; t0 += 8) {
        int4 v[8];  // past the end the last token again
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = lim[min(t0 + t, r.ntok - 1)];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          if (v[t].y > v[t].x) {
            lo_min = min(lo_min, v[t].x);
            hi_max = max(hi_max, v[t].y);
          }
          lo_max = max(lo_max, v[t].x);
          hi_min = min(hi_min, v[t].y);
        }
      }
      r.key0 = r.shared == 2 ? max(lo_min, shared_len) : lo_min;
      r.key1 = r.shared == 1 ? min(hi_max, shared_len) : hi_max;
      if (r.key1 <= r.key0) r.key0 = r.key1 = 0;
      r.full0 = lo_max;
      r.full1 = hi_min;
      r.part = part;
      if (r.few) width = line_keys(r.key1 - r.key0) / kCutKeys;
      else keys += (unsigned long long)(r.key1 - r.key0);
    }
    int total;
    const int before = block_scan(width, scan_lds, total);
    if (i < tiles) {
      r.at = line + before;
      tile_list[i] = r;
    }
    line += total;
  }
  if (keys) atomicAdd(&sum_lds, keys);
  __syncthreads();
  const int slice = share_of(line * kCutKeys, a.heads, a.few_slots, kFewMinKeys, kCutKeys);
  const int share = share_of((int64_t)sum_lds, a.heads, kTileSlots, kTileMinKeys, kPartKeys);
  const int cuts = slice / kCutKeys;  // of a slice
  const int slots = (int)min((line + cuts - 1) / cuts, (long long)a.max_slots - 1);

  // ---- items, slices, partial-result units, tokens to join
  int few_items = 0, tile_items = 0, units = 0, joins = 0;
  AttnSlot *slot_list = reinterpret_cast<AttnSlot *>(a.slots);
  for (int i0 = 0; i0 < tiles; i0 += kPlanThreads) {
    const int i = i0 + tid;
    AttnTile r;
    int parts = 0, per = 1, ups = 0;
    bool join = false;
    if (i < tiles) {
      r = tile_list[i];
      const int n = r.key1 - r.key0;
      if (r.few) {
        const int64_t last = r.at + line_keys(n) / kCutKeys - 1;
        parts = (int)(last / cuts - r.at / cuts) + 1;
      } else {
        per = part_keys(n, share);
        parts = max(1, (n + per - 1) / per);
      }
      join = parts > 1 || r.shared;
      ups = (r.ntok * a.group + kUnitRows - 1) / kUnitRows;
    }
    const bool few = i < tiles && r.few;
    int nf, nt, nu, nj;
    const int at_few = few_items + block_scan(few ? parts : 0, scan_lds, nf);
    const int at_tile = tile_items + block_scan(few ? 0 : parts, scan_lds, nt);
    const int unit = units + block_scan(join ? parts * ups : 0, scan_lds, nu);
    const int at_join = joins + block_scan(join && r.shared != 1 ? r.ntok : 0, scan_lds, nj);
    if (i < tiles) {
      // true for every batch in order, by the capacities' derivation; with a
      // q_start out of order the surplus is dropped
      const bool fits = (few ? at_few + parts <= a.max_few_items : at_tile + parts <= a.max_tile_items) &&
                        unit + parts * ups <= a.max_units;
      AttnItem item{r.tok0, fits ? r.ntok : 0, r.seq, r.key0, r.key1, r.full0, r.full1, -1};
      for (int s = 0; s < parts; ++s) {
        const int at = (few ? at_few : at_tile) + s;
        if (at >= (few ? a.max_few_items : a.max_tile_items)) break;
        if (join) item.unit = unit + s * ups;
        if (few) {
          // the piece of the tile on slice k: the line from `from` on
          const int64_t k = r.at / cuts + s, from = max(r.at, k * cuts);
          item.key0 = r.key0 + (int)(from - r.at) * kCutKeys;
          item.key1 = (int)min((int64_t)r.key1, r.key0 + ((k + 1) * cuts - r.at) * kCutKeys);
          reinterpret_cast<AttnItem *>(a.few_items)[at] = item;
          if (from == k * cuts && k < a.max_slots) {
            slot_list[k].first = at;
            slot_list[k].item = item;
            if (k > 0) slot_list[k - 1].end = at;
          }
        } else {
          item.key0 = r.key0 + s * per;
          item.key1 = min(r.key1, item.key0 + per);
          reinterpret_cast<AttnItem *>(a.tile_items)[at] = item;
        }
      }
      if (join) {
        for (int t = 0; t < r.ntok; ++t) {
          int4 *rec = reinterpret_cast<int4 *>(a.join) + 2 * (int64_t)(r.tok0 + t);
          rec[r.shared == 1] = int4{unit, fits ? parts : 0, ups, t};
          if (r.shared == 0) rec[1] = int4{0, 0, 0, 0};
          if (r.shared != 1 && at_join + t < a.tokens) a.join_list[kAttnJoinInts * (int64_t)(at_join + t)] = r.tok0 + t;
        }
      }
    }
    few_items += nf;
    tile_items += nt;
    units += nu;
    joins += nj;
  }
  few_items = min(few_items, a.max_few_items);
  if (tid == 0) {
    if (slots > 0) slot_list[slots - 1].end = few_items;
    a.info[0] = slots;
    a.info[1] = min(tile_items, a.max_tile_items);
    a.info[2] = bad_lds[0];
    a.info[3] = bad_lds[1];
    a.info[4] = (int)min((int64_t)joins, a.tokens);
    a.info[5] = min(units, a.max_units);
    a.info[6] = slice;
    a.info[7] = share;
    a.info[8] = few_items;
    for (int k = 9; k < kAttnInfoInts; ++k) a.info[k] = 0;
  }
  // the list of tokens to join takes their records along
  __syncthreads();
  for (int j = tid; j < min((int64_t)joins, a.tokens); j += kPlanThreads) {
    int4 *e = reinterpret_cast<int4 *>(a.join_list + kAttnJoinInts * (int64_t)j);
    const int4 *rec = reinterpret_cast<const int4 *>(a.join) + 2 * (int64_t)e[0].x;
    e[1] = rec[0];
    e[2] = rec[1];
  }
  // slices without work
  for (int k = slots + tid; k < a.max_slots; k += kPlanThreads) slot_list[k].first = slot_list[k].end = 0;
}

}  // namespace

hipError_t launch_attn_plan(const AttnPlanArgs &a, hipStream_t s) {
  if (a.tokens > 0) attn_limits_kernel<<<dim3((unsigned)((a.tokens + 255) / 256)), dim3(256), 0, s>>>(a);
  attn_plan_kernel<<<dim3(1), dim3(kPlanThreads), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace lora
