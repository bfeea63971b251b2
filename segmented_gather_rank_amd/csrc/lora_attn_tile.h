// lora_attn_tile.h -- attention of up to 128 rows (query token x query head of
// one key head) over a range of cached keys: prompts, and the shared keys of a
// group of sequences.
//
// The products are those of the few-row kernel, with 32 rows as the columns of
// a wave's matrix tiles: S^T = K Q^T for 64 keys (two 32 x 32 tiles) and O^T +=
// V^T P^T.  A lane holds 32 of its row's 64 scores, the lane 32 further the
// others, so a row's maximum takes one exchange between the two halves; its sum
// stays per lane until the end, and the weights, packed to bf16 where they are,
// are the next product's operand.  Q and O stay in registers.
//
// The weights are rounded to bf16 (their sum is not): a second term, as the few-row
// kernel takes, would be half as many products again where they are the bound.  The
// error of a bf16 result is then 1.9e-3 to 2.2e-3 of its size, where fp32 weights
// leave the 1.7e-3 of its own rounding.
//
// Bound: 4 dim operations per row and key on the matrix cores against one
// exponential and about six vector operations per score, which cost about as many
// cycles; so the loop is written to keep both busy.  128 rows share each 64-key
// tile of K and V through LDS, in two buffers each.  With a bf16 cache the next
// tile goes from global memory straight to LDS (no registers in between) while a
// tile is computed; an e4m3 cache is widened on the way, through registers.  Operand
// reads run six matrix instructions ahead in the first product, and in the second
// every matrix instruction is followed by its share of the exponentials.
//
// Measured (16384-token prompt, 32 / 8 heads of 128, causal): 2230 to 2290 us, 960 to
// 990 TFLOP/s, where a library product of 8192^3 reaches 1200; through registers 2419
// us, but an e4m3 cache 2209.  At
// this rate the chip lowers its clock (2.0 GHz): with the scores of tile t + 1
// computed beside the weights of tile t the matrix cores were busy 45 % of the
// cycles instead of 37 %, for 2290 us in all, and short ranges lost a quarter.
//
// Workgroups of one key head follow each other at the distance of the number of
// head groups: with the usual 8 key heads, on one XCD, whose L2 then holds that
// head's keys.
#pragma once

#include "lora_attn_dev.h"

namespace lora {

namespace {

constexpr int kKeys = 64;  // keys per tile

template <int DP, bool FP8>
struct TileShape {
  static constexpr int KS = DP / 16;                  // k-steps of a score product
  static constexpr int DT = DP / 32;                  // 32-row tiles of O^T
  // LDS rows (elements).  Tiles that pass through registers are padded so that
  // the operand reads have no bank conflicts; those loaded straight to LDS are
  // packed, with the 16-byte pieces of a row permuted instead (k_swap, v_swap).
  static constexpr int LDK = FP8 ? DP + 8 : DP, LDV = FP8 ? DP + 16 : DP;
  static constexpr int CPR = FP8 ? DP / 16 : DP / 8;  // 16-byte pieces of a cached row
  static constexpr int ROWS = 256 / CPR;              // rows per load of the workgroup
  static constexpr int NL = kKeys / ROWS;             // loads per thread, K and V each
  // Piece p of row r is kept in place p ^ swap(r).  K: 16 lanes read one piece of
  // 16 consecutive rows (8 where a row holds more than the 64 banks); V: 32 lanes
  // read four neighbouring pieces of 4 consecutive rows.
  static __device__ __forceinline__ int k_swap(int r) {
    return FP8 ? 0 : DP == 64 ? (r >> 1) & 7 : DP == 128 ? r & 15 : r & 7;
  }
  static __device__ __forceinline__ int v_swap(int r) { return FP8 ? 0 : DP == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2; }
};

// A workgroup's LDS.  Separate arrays, so that the compiler sees that reads of one
// buffer need not wait for the loads into another.
struct TileLds {
  uint16_t *k0, *k1, *v0, *v1;
  int *good, *flag;  // CAREFUL: which keys are keys; whether V holds infinities or NaN
};

// One item.  CAREFUL = false supposes that every key of the range lies in a page
// of the cache and that no tile with hidden keys holds an infinite or NaN value;
// it returns true, with nothing written, when it met either, and the item is
// then done again with CAREFUL = true, which supposes nothing.  (One loop with
// both costs the usual case a third of its registers.)
template <int DP, bool FP8, bool GENERAL, bool CAREFUL>
__device__ __forceinline__ bool run_tile(const AttnArgs &a, const AttnItem &it, int h, const TileLds lds) {
  using S = TileShape<DP, FP8>;
  const int tid = thread_of_item(), lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int g = lane / 32, c = lane % 32;
  const int kvh = a.by_kv_parts.quotient(h);
  const int row = 32 * wave + c, rows = it.ntok * a.group;
  const bool row_ok = row < rows;
  const int nth = row_ok ? a.by_group.quotient(row) : 0;
  const int tok = it.tok0 + nth, qh = h * a.group + (row_ok ? row - nth * a.group : 0);
  const bool wave_ok = 32 * wave < rows;

  const int32_t *table = a.cache.table + it.seq * a.cache.table_stride;
  const int ntiles = (it.key1 - it.key0 + kKeys - 1) / kKeys;
  const char *k_head = a.cache.k + kvh * a.cache.head_bytes, *v_head = a.cache.v + kvh * a.cache.head_bytes;
  bool odd = false;  // met what CAREFUL = false does not handle

  // lane j of every wave looks up key j of a tile; beyond the range the last key
  // again, never seen
  auto fetch_page = [&](int tile) -> int32_t {
    const int key = min(it.key0 + tile * kKeys + lane, it.key1 - 1);
    return table[a.cache.page_size.quotient(key)];
  };
  uint64_t good = 0;  // CAREFUL: keys of the located tile in a good page
  auto offset_of = [&](int tile, int32_t page) -> int64_t {
    const int key = it.key0 + tile * kKeys + lane;
    const int64_t off = key_offset(a.cache, min(key, it.key1 - 1), page);
    if constexpr (CAREFUL) good = __ballot(off >= 0 && key < it.key1);
    else odd |= off < 0;
    return max((int64_t)0, off);
  };
  auto is_masked = [&](int tile) {
    const int k0 = it.key0 + tile * kKeys;
    return k0 < it.full0 || k0 + kKeys > min(it.full1, it.key1);
  };

  // the first tiles' pages are on their way while Q is read
  int32_t page = 0, page1 = 0, page2 = 0;
  if (ntiles > 0) {
    page = fetch_page(0);
    page1 = fetch_page(1);
    page2 = fetch_page(2);
  }
  bf16x8 q[S::KS];
#pragma unroll
  for (int s = 0; s < S::KS; ++s) {
    const int d = 16 * s + 8 * g;
    u32x4 w = {0, 0, 0, 0};
    if (row_ok && d < a.dim) w = gload16(a.q + 2 * (tok * a.ldq + (int64_t)qh * a.dim + d));
    q[s] = __builtin_bit_cast(bf16x8, w);
  }
  int lo = 0, hi = 0, pos = 0;
  if (row_ok) {
    const int4 v = reinterpret_cast<const int4 *>(a.limits)[tok];
    lo = max(v.x, it.key0), hi = min(v.y, it.key1), pos = v.z;
  }
  const uint32_t span = (uint32_t)max(hi - lo, 0);
  const ScoreArgs sc = score_args<GENERAL>(a, kvh, qh);
  const float mul = GENERAL ? 1.f : sc.mul;  // score registers * mul: base-2 logits

  float base = kNegInf, l = 0.f;
  f32x16 o[S::DT];
#pragma unroll
  for (int d = 0; d < S::DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;

  // ---- pieces of the loops.  Register i of score tile t is key 32 t + 8 (i / 4) +
  // 4 g + i % 4; step s of the second product takes keys 16 s + 8 (e / 4) + 4 g + e % 4.
  const int k_at = c * S::LDK, k_x = S::k_swap(c);
  auto k_operand = [&](const uint16_t *kl, int t, int s) {
    return *reinterpret_cast<const bf16x8 *>(kl + 32 * t * S::LDK + k_at + 8 * ((2 * s + g) ^ k_x));
  };
  const int v_r = 4 * g + (lane % 16) / 4, v_x = S::v_swap(v_r), v_p = 2 * ((lane / 16) % 2) + (lane % 4) / 2;
  auto v_operand = [&](const uint16_t *vl, int d, int s) {
    const uint16_t *b = vl + (16 * s + v_r) * S::LDV + 8 * ((4 * d + v_p) ^ v_x) + 4 * (lane % 2);
    const u32x2 v0 = lds_read_tr(b), v1 = lds_read_tr(b + 8 * S::LDV);
    return u32x4{v0.x, v0.y, v1.x, v1.y};
  };
  auto zero = [&](f32x16 (&st)[2]) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) st[t][i] = 0.f;
  };
  // Scores of a tile, kAhead operand reads in flight before the first product and
  // between the others.
  constexpr int kAhead = 6;
  auto scores = [&](const uint16_t *kl, f32x16 (&st)[2]) {
    bf16x8 k[2 * S::KS];
#pragma unroll
    for (int i = 0; i < 2 * S::KS; ++i) k[i] = k_operand(kl, i % 2, i / 2);
    zero(st);
#pragma unroll
    for (int i = 0; i < 2 * S::KS; ++i)
      st[i % 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[i], q[i / 2], st[i % 2], 0, 0, 0);
    __builtin_amdgcn_sched_group_barrier(kSchedDsRead, kAhead, 0);
#pragma unroll
    for (int i = 0; i < 2 * S::KS - kAhead; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedDsRead, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kSchedMfma, kAhead, 0);
  };
  auto logits = [&](int tile, f32x16 (&st)[2]) {
    const int away = pos - (it.key0 + tile * kKeys + 4 * g);
#pragma unroll
    for (int t = 0; t < 2; ++t) general_logits<16>(sc, st[t], [&](int i) { return away - (32 * t + 8 * (i / 4) + i % 4); });
  };
  auto hide = [&](int tile, f32x16 (&st)[2]) {
    const int from = it.key0 + tile * kKeys + 4 * g - lo;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if ((uint32_t)(from + 32 * t + 8 * (i / 4) + i % 4) >= span) st[t][i] = kNegInf;
  };
  // Raises the base of the weights if a score exceeds it by more than the slack.
  auto raise = [&](const f32x16 (&st)[2]) {
    float top0 = kNegInf, top1 = kNegInf;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      top0 = max3(top0, st[0][i], st[0][i + 1]);
      top1 = max3(top1, st[1][i], st[1][i + 1]);
    }
    const float top = max_halves(fmaxf(top0, top1)) * mul;
    // (a NaN score makes its weight NaN below; it may not steer the branch)
    if (__any(!(top <= base + kSlack) && top > kNegInf)) {
      const float next = fmaxf(base, top);
      const float fade = next > kNegInf ? exp2_fast(base - next) : 1.f;
      base = next;
      l *= fade;
#pragma unroll
      for (int d = 0; d < S::DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= fade;
    }
  };
  u32x4 p[4];
  float even = 0.f, minus = 0.f;  // the first weight of a pair; -base
  auto weights = [&](const f32x16 (&st)[2], int e0, int e1) {  // weights e0 .. e1 - 1 of this lane's 32
#pragma unroll
    for (int e = e0; e < e1; ++e) {
      const float x = exp2_fast(__builtin_fmaf(st[e / 16][e % 16], mul, minus));
      l += x;
      if (e % 2 == 0) even = x;
      else p[e / 8][(e % 8) / 2] = pack_bf16x2(even, x);
    }
  };
  auto product = [&](f32x16 &od, u32x4 v, u32x4 w) {
    od = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, w), od, 0, 0, 0);
  };
  // O^T += V^T P^T with the weights from `first` on still to be computed: each
  // product goes out with its share of what the next steps need, two reads of V
  // and some weights, which run beside it.
  auto outputs = [&](const uint16_t *vl, const f32x16 (&st)[2], int first) {
    u32x4 v[2][S::DT];
#pragma unroll
    for (int d = 0; d < S::DT; ++d) v[0][d] = v_operand(vl, d, 0);
    if (first < 8) {
      weights(st, first, 8);
      first = 8;
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int d = 0; d < S::DT; ++d) {
        product(o[d], v[s % 2][d], p[s]);
        if (s < 3) {
          v[(s + 1) % 2][d] = v_operand(vl, d, s + 1);
          // weights of step s + 1, where they are not there yet
          const int e0 = 8 * (s + 1) + 8 * d / S::DT, e1 = 8 * (s + 1) + 8 * (d + 1) / S::DT;
          if (e0 >= first) weights(st, e0, e1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
  };

  if constexpr (CAREFUL) {
    // ---- one tile at a time, in the first buffers
    for (int tile = 0; tile < ntiles; ++tile) {
      const int k0 = it.key0 + tile * kKeys;
      const int64_t off = offset_of(tile, fetch_page(tile));
      __syncthreads();  // the previous tile is read
      if (tid < kKeys) lds.good[tid] = (good >> tid) & 1;
      if (tid == 0) lds.flag[0] = 0;
      __syncthreads();
      const int piece = tid % S::CPR;
      const int col = piece * (FP8 ? 16 : 8) < a.dim ? 16 * piece : 0;
      bool poison = false;
#pragma unroll 1
      for (int i = 0; i < S::NL; ++i) {
        const int r = S::ROWS * i + tid / S::CPR;
        const int64_t at = __shfl(off, r) + col;
        u32x4 k = gload16(k_head + at), v = gload16(v_head + at);
        if (!((good >> r) & 1)) k = v = u32x4{0, 0, 0, 0};
        uint16_t *kp = lds.k0 + r * S::LDK, *vp = lds.v0 + r * S::LDV;
        if constexpr (FP8) {
          const u32x4 v0 = e4m3x8_to_bf16(v[0], v[1]), v1 = e4m3x8_to_bf16(v[2], v[3]);
          poison |= any_nonfinite(v0) || any_nonfinite(v1);
          *reinterpret_cast<u32x4 *>(kp + 16 * piece) = e4m3x8_to_bf16(k[0], k[1]);
          *reinterpret_cast<u32x4 *>(kp + 16 * piece + 8) = e4m3x8_to_bf16(k[2], k[3]);
          *reinterpret_cast<u32x4 *>(vp + 16 * piece) = v0;
          *reinterpret_cast<u32x4 *>(vp + 16 * piece + 8) = v1;
        } else {
          poison |= any_nonfinite(v);
          *reinterpret_cast<u32x4 *>(kp + 8 * (piece ^ S::k_swap(r))) = k;
          *reinterpret_cast<u32x4 *>(vp + 8 * (piece ^ S::v_swap(r))) = v;
        }
      }
      if (poison) atomicOr(lds.flag, 1);
      __syncthreads();
      if (!wave_ok) continue;
      f32x16 st[2];
      scores(lds.k0, st);
      if constexpr (GENERAL) logits(tile, st);
      uint32_t see = 0;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = 32 * t + 8 * (i / 4) + 4 * g + i % 4;
          if ((uint32_t)(k0 + j - lo) < span && lds.good[j]) see |= 1u << (16 * t + i);
          else st[t][i] = kNegInf;
        }
      raise(st);
      minus = base == kNegInf ? 0.f : -base;
      weights(st, 0, 32);
      const bool bad = lds.flag[0];
#pragma unroll
      for (int d = 0; d < S::DT; ++d) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          u32x4 v = v_operand(lds.v0, d, s);
          if (bad) v = v_part(v, kVFinite);
          product(o[d], v, p[s]);
        }
        if (!bad) continue;
#pragma unroll 1
        for (int part = kVPosInf; part <= kVNegInf; ++part) {
          f32x16 n;
#pragma unroll
          for (int i = 0; i < 16; ++i) n[i] = 0.f;
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            u32x4 seen;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int b = 8 * s + 2 * i;
              seen[i] = ((see >> b) & 1 ? 0x3f80u : 0u) | ((see >> (b + 1)) & 1 ? 0x3f800000u : 0u);
            }
            product(n, v_part(v_operand(lds.v0, d, s), part), seen);
          }
          const float inf = part == kVPosInf ? __builtin_inff() : kNegInf;
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][i] = n[i] > 0.f ? o[d][i] + inf : o[d][i];
        }
      }
    }
    __syncthreads();  // the buffers may be reused
  } else if constexpr (FP8) {
    // ---- through registers, one tile ahead
    const int piece = tid % S::CPR, lrow = tid / S::CPR;
    // past the head dimension the first piece again: Q is zero there, and O^T's
    // rows there are not stored
    const char *k_piece = k_head + (piece * 16 < a.dim ? 16 * piece : 0);
    const int64_t k_to_v = v_head - k_head;
    u32x4 kr[S::NL], vr[S::NL];
    const char *at[S::NL];
    auto locate = [&](int tile, int32_t pid) {
      const int64_t off = offset_of(tile, pid);
#pragma unroll
      for (int i = 0; i < S::NL; ++i) at[i] = k_piece + __shfl(off, S::ROWS * i + lrow);
    };
    auto issue = [&]() {
#pragma unroll
      for (int i = 0; i < S::NL; ++i) {
        kr[i] = gload16(at[i]);
        vr[i] = gload16(at[i] + k_to_v);
      }
    };
    auto stage = [&](int tile, auto masked_tag) {
      constexpr bool MASKED = decltype(masked_tag)::value;
      uint16_t *kl = tile & 1 ? lds.k1 : lds.k0, *vl = tile & 1 ? lds.v1 : lds.v0;
#pragma unroll
      for (int i = 0; i < S::NL; ++i) {
        const int r = S::ROWS * i + lrow;
        uint16_t *kp = kl + r * S::LDK + piece * 16, *vp = vl + r * S::LDV + piece * 16;
        const u32x4 v0 = e4m3x8_to_bf16(vr[i][0], vr[i][1]), v1 = e4m3x8_to_bf16(vr[i][2], vr[i][3]);
        if (MASKED) odd |= any_nonfinite(v0) || any_nonfinite(v1);
        *reinterpret_cast<u32x4 *>(kp) = e4m3x8_to_bf16(kr[i][0], kr[i][1]);
        *reinterpret_cast<u32x4 *>(kp + 8) = e4m3x8_to_bf16(kr[i][2], kr[i][3]);
        *reinterpret_cast<u32x4 *>(vp) = v0;
        *reinterpret_cast<u32x4 *>(vp + 8) = v1;
      }
    };
    auto put = [&](int tile) {
      if (is_masked(tile)) stage(tile, std::true_type{});
      else stage(tile, std::false_type{});
    };
    if (ntiles > 0) {
      locate(0, page);
      issue();
      if (ntiles > 1) {
        locate(1, page1);
        page = page2;
      }
      put(0);
    }
    __syncthreads();
    for (int tile = 0; tile < ntiles; ++tile) {
      if (tile + 1 < ntiles) issue();
      if (wave_ok) {
        f32x16 st[2];
        scores(tile & 1 ? lds.k1 : lds.k0, st);
        if constexpr (GENERAL) logits(tile, st);
        if (is_masked(tile)) hide(tile, st);
        raise(st);
        minus = base == kNegInf ? 0.f : -base;
        outputs(tile & 1 ? lds.v1 : lds.v0, st, 0);
      }
      if (tile + 1 < ntiles) {
        if (tile + 2 < ntiles) {
          locate(tile + 2, page);
          if (tile + 3 < ntiles) page = fetch_page(tile + 3);
        }
        // the other buffers were last read before the previous barrier
        put(tile + 1);
        __syncthreads();
      }
    }
  } else {
    // ---- straight to LDS.  Load i of wave w fills rows (4 i + w) * PER .. in
    // order; a lane's piece is the one whose place is the lane's, which for all
    // of its rows is the same (the swaps repeat every 4 * PER rows or less).
    constexpr int PER = kWave / S::CPR;  // rows per load of a wave
    const int in_row = lane % S::CPR, in_load = lane / S::CPR, r0 = wave * PER + in_load;
    static_assert(4 * PER % (DP == 256 ? 8 : 16) == 0, "the swaps repeat");
    // past the head dimension the first piece again: Q is zero there, and O^T's
    // rows there are not stored
    auto column = [&](int p) { return 8 * p < a.dim ? 16 * p : 0; };
    const char *k_lane = k_head + column(in_row ^ S::k_swap(r0));
    const char *v_lane = v_head + column(in_row ^ S::v_swap(r0));
    int64_t at[S::NL];  // rows of the next tile to load
    auto locate = [&](int tile, int32_t pid) {
      const int64_t off = offset_of(tile, pid);
#pragma unroll
      for (int i = 0; i < S::NL; ++i) at[i] = __shfl(off, 4 * PER * i + r0);
    };
    auto load = [&](const char *from, uint16_t *to) {
#pragma unroll
      for (int i = 0; i < S::NL; ++i)
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(from + at[i]),
                                         (__attribute__((address_space(3))) void *)(to + (4 * i + wave) * 64 * 8), 16, 0, 0);
    };
    // A tile with hidden keys: whether its values hold what a weight of zero does
    // not hide.
    auto inspect = [&](const uint16_t *vl) {
#pragma unroll
      for (int i = 0; i < S::NL; ++i) odd |= any_nonfinite(*reinterpret_cast<const u32x4 *>(vl + (256 * i + tid) * 8));
    };
    // The other buffers were last read before the last barrier: they take the next
    // tile, which is waited for at the end.
    auto iterate = [&](int t, uint16_t *k_now, uint16_t *v_now, uint16_t *k_next, uint16_t *v_next) {
      if (t + 1 < ntiles) {
        load(k_lane, k_next);
        load(v_lane, v_next);
      }
      const bool masked = is_masked(t);
      if (wave_ok) {
        f32x16 st[2];
        scores(k_now, st);
        if constexpr (GENERAL) logits(t, st);
        if (masked) hide(t, st);
        raise(st);
        minus = base == kNegInf ? 0.f : -base;
        outputs(v_now, st, 0);
      }
      if (masked) inspect(v_now);
      if (t + 2 < ntiles) {
        locate(t + 2, page);
        if (t + 3 < ntiles) page = fetch_page(t + 3);
      }
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
    };
    if (ntiles > 0) {
      locate(0, page);
      load(k_lane, lds.k0);
      load(v_lane, lds.v0);
      locate(1, page1);
      page = page2;
      __builtin_amdgcn_s_waitcnt(0);
    }
    __syncthreads();
    for (int t = 0; t < ntiles; t += 2) {
      iterate(t, lds.k0, lds.v0, lds.k1, lds.v1);
      if (t + 1 < ntiles) iterate(t + 1, lds.k1, lds.v1, lds.k0, lds.v0);
    }
  }
  if constexpr (!CAREFUL) {
    if (__syncthreads_or(odd)) return true;
  }

  if (!row_ok) return false;
  l = sum_halves(l);
  const float vs = a.cache.v_scale ? a.cache.v_scale[kvh] : 1.f;
  const float f = it.unit >= 0 ? vs : (l > 0.f ? vs / l : (l == 0.f ? 0.f : l));
  const int64_t pr = it.unit >= 0 ? part_row(a, it.unit + row / kUnitRows, h, row % kUnitRows) : 0;
#pragma unroll
  for (int d = 0; d < S::DT; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = 32 * d + 8 * i + 4 * g;
      if (at >= a.dim) continue;
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = f == 0.f ? 0.f : o[d][4 * i + e] * f;
      if (it.unit >= 0) {
        gstore16f(a.part + pr * a.dim + at, f32x4{x[0], x[1], x[2], x[3]});
      } else {
        typedef __attribute__((address_space(1))) u32x2 g_u32x2;
        *(g_u32x2 *)(a.out + 2 * (tok * a.ldo + (int64_t)qh * a.dim + at)) =
            u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
      }
    }
  if (g == 0) {
    if (it.unit >= 0) {
      a.part_ml[2 * pr] = base;
      a.part_ml[2 * pr + 1] = l;
    } else if (a.lse) {
      a.lse[(int64_t)tok * a.q_heads + qh] = l == 0.f ? kNegInf : (base + __log2f(l)) * kLn2;
    }
  }
  return false;
}

}  // namespace

}  // namespace lora
