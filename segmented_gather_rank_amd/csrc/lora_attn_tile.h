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
// Bound: 4 dim operations per row and key on the matrix cores against one
// exponential and about ten vector operations per score.  128 rows share each
// 64-key tile of K and V through LDS (two buffers; the next tile's global loads
// are in flight while a tile is computed), so a key read once from L2 serves 128
// rows.  Workgroups of one key head follow each other at the distance of the
// number of head groups, with the usual 8 key heads on one XCD, whose L2 then
// holds that head's keys.
#pragma once

#include "lora_attn_dev.h"

namespace lora {

namespace {

constexpr int kKeys = 64;  // keys per tile
template <int DP, bool FP8>
struct TileShape {
  static constexpr int KS = DP / 16;                  // k-steps of a score product
  static constexpr int DT = DP / 32;                  // 32-row tiles of O^T
  static constexpr int LDK = DP + 8, LDV = DP + 16;   // LDS rows (elements): no bank conflicts
  static constexpr int CPR = FP8 ? DP / 16 : DP / 8;  // 16-byte pieces of a cached row
  static constexpr int ROWS = 256 / CPR;              // rows per load of the workgroup
  static constexpr int NL = kKeys / ROWS;             // loads per thread, K and V each
  static constexpr int BUF = kKeys * (LDK + LDV);
};

// One item.  CAREFUL = false supposes that every key of the range lies in a page
// of the cache and that no tile with hidden keys holds an infinite or NaN value;
// it returns true, with nothing written, when it met either, and the item is
// then done again with CAREFUL = true, which supposes nothing.  (One loop with
// both costs the usual case a third of its registers.)
template <int DP, bool FP8, bool GENERAL, bool CAREFUL>
__device__ __forceinline__ bool run_tile(const AttnArgs &a, const AttnItem &it, int h, uint16_t *lds, int *flag_lds) {
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
  const int piece = tid % S::CPR, lrow = tid / S::CPR;
  // past the head dimension the first piece again: Q is zero there, and O^T's
  // rows there are not stored
  const bool piece_ok = piece * (FP8 ? 16 : 8) < a.dim;
  const char *k_piece = a.cache.k + kvh * a.cache.head_bytes + (piece_ok ? 16 * piece : 0);

  // lane j of every wave looks up key j of a tile
  auto fetch_page = [&](int tile) -> int32_t {
    const int key = min(it.key0 + tile * kKeys + lane, it.key1 - 1);
    return table[a.cache.page_size.quotient(key)];
  };
  u32x4 kr[S::NL], vr[S::NL];
  uint64_t good = 0;  // keys of the issued tile in a good page
  bool odd = false;   // met what CAREFUL = false does not handle
  const char *at[S::NL];   // this thread's pieces of K of the next tile to issue
  const int64_t k_to_v = a.cache.v - a.cache.k;
  uint64_t good_next = 0;  // and which of its keys lie in a good page
  auto locate = [&](int tile, int32_t page) {
    // beyond the range the last key is loaded again, and never seen
    const int key = it.key0 + tile * kKeys + lane;
    const int64_t off = key_offset(a.cache, min(key, it.key1 - 1), page);
    if constexpr (CAREFUL) good_next = __ballot(off >= 0 && key < it.key1);
    else odd |= off < 0;
    const int64_t o = max((int64_t)0, off);
#pragma unroll
    for (int i = 0; i < S::NL; ++i) at[i] = k_piece + __shfl(o, S::ROWS * i + lrow);
  };
  auto issue = [&]() {
    good = good_next;
#pragma unroll
    for (int i = 0; i < S::NL; ++i) {
      kr[i] = gload16(at[i]);
      vr[i] = gload16(at[i] + k_to_v);
    }
  };
  auto is_masked = [&](int tile) {
    const int k0 = it.key0 + tile * kKeys;
    return k0 < it.full0 || k0 + kKeys > min(it.full1, it.key1);
  };
  // Registers to LDS.  In K the 8 spare elements of a row tell whether it is a
  // key (CAREFUL).  Returns whether V holds what a weight of zero does not hide.
  auto stage_as = [&](int tile, auto plain_tag) -> bool {
    constexpr bool PLAIN = decltype(plain_tag)::value;  // all keys seen
    uint16_t *kl = lds + (tile & 1) * S::BUF, *vl = kl + kKeys * S::LDK;
    bool poison = false;
#pragma unroll
    for (int i = 0; i < S::NL; ++i) {
      const int r = S::ROWS * i + lrow;
      u32x4 k = kr[i], v = vr[i];
      if constexpr (!PLAIN) {
        if constexpr (CAREFUL) {
          if (!((good >> r) & 1)) k = v = u32x4{0, 0, 0, 0};
          if (piece == 0) kl[r * S::LDK + DP] = (good >> r) & 1;
        } else {
          if (it.key0 + tile * kKeys + r >= it.key1) v = u32x4{0, 0, 0, 0};
        }
      }
      uint16_t *kp = kl + r * S::LDK + piece * (FP8 ? 16 : 8), *vp = vl + r * S::LDV + piece * (FP8 ? 16 : 8);
      if constexpr (FP8) {
        const u32x4 v0 = e4m3x8_to_bf16(v[0], v[1]), v1 = e4m3x8_to_bf16(v[2], v[3]);
        if (!PLAIN) poison |= any_nonfinite(v0) || any_nonfinite(v1);
        *reinterpret_cast<u32x4 *>(kp) = e4m3x8_to_bf16(k[0], k[1]);
        *reinterpret_cast<u32x4 *>(kp + 8) = e4m3x8_to_bf16(k[2], k[3]);
        *reinterpret_cast<u32x4 *>(vp) = v0;
        *reinterpret_cast<u32x4 *>(vp + 8) = v1;
      } else {
        if (!PLAIN) poison |= any_nonfinite(v);
        *reinterpret_cast<u32x4 *>(kp) = k;
        *reinterpret_cast<u32x4 *>(vp) = v;
      }
    }
    return poison;
  };
  // CAREFUL: a tile's word says that its values hold infinities or NaN.  Four
  // words in turn: one is cleared after the barrier that ends its tile and next
  // written two barriers later.
  auto put = [&](int tile) {
    if constexpr (CAREFUL) {
      if (stage_as(tile, std::false_type{})) atomicOr(&flag_lds[tile & 3], 1);
    } else if (is_masked(tile)) {
      odd |= stage_as(tile, std::false_type{});
    } else {
      stage_as(tile, std::true_type{});
    }
  };

  int32_t page = ntiles > 0 ? fetch_page(0) : 0;
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
  const float mul = GENERAL ? 1.f : sc.mul;  // st * mul: base-2 logits

  float base = kNegInf, l = 0.f;
  f32x16 o[S::DT];
#pragma unroll
  for (int d = 0; d < S::DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;

  if (CAREFUL && tid < 4) flag_lds[tid] = 0;
  if (ntiles > 0) {
    locate(0, page);
    issue();
    if (ntiles > 1) {
      locate(1, fetch_page(1));
      if (ntiles > 2) page = fetch_page(2);
    }
  }
  if constexpr (CAREFUL) __syncthreads();
  if (ntiles > 0) put(0);
  __syncthreads();

  for (int tile = 0; tile < ntiles; ++tile) {
    const int k0 = it.key0 + tile * kKeys;
    if (tile + 1 < ntiles) issue();
    if (wave_ok) {
      const uint16_t *kl = lds + (tile & 1) * S::BUF, *vl = kl + kKeys * S::LDK;
      // ---- scores of 64 keys
      f32x16 st[2];
      {
        bf16x8 k[2 * S::KS];
#pragma unroll
        for (int s = 0; s < S::KS; ++s)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            k[2 * s + t] = *reinterpret_cast<const bf16x8 *>(kl + (32 * t + c) * S::LDK + 16 * s + 8 * g);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) st[t][i] = 0.f;
#pragma unroll
        for (int s = 0; s < S::KS; ++s)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            st[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[2 * s + t], q[s], st[t], 0, 0, 0);
        // kAhead reads in flight before the first product and between the others
        constexpr int kAhead = 6;
        __builtin_amdgcn_sched_group_barrier(kSchedDsRead, kAhead, 0);
#pragma unroll
        for (int s = 0; s < 2 * S::KS - kAhead; ++s) {
          __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
          __builtin_amdgcn_sched_group_barrier(kSchedDsRead, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(kSchedMfma, kAhead, 0);
      }
      // ---- softmax; register i of tile t is key 32 t + 8 (i / 4) + 4 g + i % 4
      if constexpr (GENERAL) {
        const int away = pos - (k0 + 4 * g);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) st[t][i] = logit2<true>(sc, st[t][i], away - (32 * t + 8 * (i / 4) + i % 4));
      }
      uint32_t see = 0xffffffffu;
      if constexpr (CAREFUL) {
        see = 0;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = 32 * t + 8 * (i / 4) + 4 * g + i % 4;
            if ((uint32_t)(k0 + j - lo) < span && kl[j * S::LDK + DP]) see |= 1u << (16 * t + i);
            else st[t][i] = kNegInf;
          }
      } else if (is_masked(tile)) {
        const int from = k0 + 4 * g - lo;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if ((uint32_t)(from + 32 * t + 8 * (i / 4) + i % 4) >= span) st[t][i] = kNegInf;
      }
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
      const float minus = base == kNegInf ? 0.f : -base;
      // ---- weights, and O^T += V^T P^T; step s: keys 16 s + 8 (e / 4) + 4 g + e % 4
      u32x4 p[4];
      float even;  // the first of a pair
      auto weights = [&](int s, int e0, int e1) {
#pragma unroll
        for (int e = e0; e < e1; ++e) {
          const float x = exp2_fast(__builtin_fmaf(st[s / 2][8 * (s % 2) + e], mul, minus));
          l += x;
          if (e % 2 == 0) even = x;
          else p[s][e / 2] = pack_bf16x2(even, x);
        }
      };
      auto v_operand = [&](int d, int s) {
        const uint16_t *b = vl + (16 * s + 4 * g + (lane % 16) / 4) * S::LDV + 32 * d + 16 * ((lane / 16) % 2) + 4 * (lane % 4);
        const u32x2 v0 = lds_read_tr(b), v1 = lds_read_tr(b + 8 * S::LDV);
        return u32x4{v0.x, v0.y, v1.x, v1.y};
      };
      const bool poison = CAREFUL && flag_lds[tile & 3];
      if constexpr (CAREFUL) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          weights(s, 0, 8);
#pragma unroll
          for (int d = 0; d < S::DT; ++d) {
            u32x4 v = v_operand(d, s);
            if (poison) v = v_part(v, kVFinite);
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, p[s]),
                                                           o[d], 0, 0, 0);
          }
        }
      } else {
        // Each product of step s goes out with its share of what step s + 1 needs:
        // two reads of V and 8 / DT weights, which run beside it.
        u32x4 v[2][S::DT];
#pragma unroll
        for (int d = 0; d < S::DT; ++d) v[0][d] = v_operand(d, 0);
        weights(0, 0, 8);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int d = 0; d < S::DT; ++d) {
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v[s % 2][d]),
                                                           __builtin_bit_cast(bf16x8, p[s]), o[d], 0, 0, 0);
            if (s < 3) {
              v[(s + 1) % 2][d] = v_operand(d, s + 1);
              weights(s + 1, 8 * d / S::DT, 8 * (d + 1) / S::DT);
              __builtin_amdgcn_sched_barrier(0);
            }
          }
      }
      if (CAREFUL && poison) {
#pragma unroll
        for (int d = 0; d < S::DT; ++d)
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
              n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v_part(v_operand(d, s), part)),
                                                          __builtin_bit_cast(bf16x8, seen), n, 0, 0, 0);
            }
            const float inf = part == kVPosInf ? __builtin_inff() : kNegInf;
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = n[i] > 0.f ? o[d][i] + inf : o[d][i];
          }
      }
    }
    if (tile + 1 < ntiles) {
      if (tile + 2 < ntiles) {
        locate(tile + 2, page);
        if (tile + 3 < ntiles) page = fetch_page(tile + 3);
      }
      // the other buffer was last read before the previous barrier
      put(tile + 1);
      __syncthreads();
      if (CAREFUL && tid == 0) flag_lds[tile & 3] = 0;
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
