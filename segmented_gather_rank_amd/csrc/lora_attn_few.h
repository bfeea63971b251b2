// lora_attn_few.h -- attention of up to 16 rows (query token x query head of
// one key head) over a range of cached keys: decode, short extensions, and every
// fp32 call.  Device code of lora_attn.hip.
//
// With the rows of one key head as the columns of a matrix product, the scores
// of 16 keys are S^T = K Q^T (16 x 16, contracted over the head dimension) and
// the output is O^T += V^T P^T (dim x 16, contracted over the keys).  A lane's
// column is then one row from beginning to end: its running maximum and sum, its
// weights and its part of O stay in that lane, and the scores that a product
// leaves in a lane (keys 4g .. 4g + 3 of each 16, g the lane's group of 16) are
// the operand of the next product if V is taken in the same key order, which the
// transposing LDS read does.  No weight ever leaves its lane.
//
// The matrix cores take bf16, so a weight goes in as two terms, its rounding and
// what that leaves out (2^-16 of it is lost), and the products with V run twice.  The
// kernel waits for memory anyway: 537 us with one term and with two on the decode
// batch below, 349 and 354 on 512 decode tokens beside 4 prompts of 1024.  (The tile
// kernel, which the matrix cores bound, takes one term.)
//
// Bound: the keys and values are read once and used by at most 16 rows, 16 / 2
// operations per byte, so HBM bounds it.  Hence no sharing: every wave is a
// worker of its own with a slice of the keys (lora_attn.h), 32 keys a step, and
// never waits for another.  K goes from global memory straight into operand
// registers, V through LDS that only its wave touches (for the transposition),
// the next step's 16 loads of 16 bytes a lane are in flight while a step is
// computed, and page ids are fetched two steps ahead.
//
// Measured (32 / 8 heads of 128): 256 decode sequences of 64 to 6000 keys, bf16
// pages of 16, 530 us, 5.9 TB/s; 24 of 30 to 65 thousand keys, e4m3, capped, 367
// us, 5.8 TB/s; 64 of 64 to 3000 keys, fp32, 204 us, 3.8 TB/s.  Twice as many waves read no faster (544 us).
#pragma once

#include "lora_attn_dev.h"

namespace lora {

namespace {

constexpr int kStep = 32;  // keys per wave and step

// A wave's result, final or partial: lane (g, c) holds row c, dimensions
// 16 d + 4 g .. + 3, and its row's maximum and sum.
template <int DP, typename OUT>
__device__ __forceinline__ void finish_few(const AttnArgs &a, const AttnItem &it, int h, int lane, const f32x4 (&o)[DP / 16],
                                           float base, float l) {
  const int g = lane / 16, row = lane % 16;
  if (row >= it.ntok * a.group) return;
  const int nth = a.by_group.quotient(row), t = it.tok0 + nth, qh = h * a.group + row - nth * a.group;
  const float vs = a.cache.v_scale ? a.cache.v_scale[a.by_kv_parts.quotient(h)] : 1.f;
  const float mul = it.unit >= 0 ? vs : (l > 0.f ? vs / l : (l == 0.f ? 0.f : l));
  const int64_t pr = it.unit >= 0 ? part_row(a, it.unit, h, row) : 0;
#pragma unroll
  for (int d = 0; d < DP / 16; ++d) {
    const int at = 16 * d + 4 * g;
    if (at >= a.dim) break;
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = mul == 0.f ? 0.f : o[d][i] * mul;
    if (it.unit >= 0) {
      gstore16f(a.part + pr * a.dim + at, f32x4{x[0], x[1], x[2], x[3]});
    } else if constexpr (sizeof(OUT) == 4) {
      gstore16f(a.out + 4 * (t * a.ldo + (int64_t)qh * a.dim + at), f32x4{x[0], x[1], x[2], x[3]});
    } else {
      typedef __attribute__((address_space(1))) u32x2 g_u32x2;
      *(g_u32x2 *)(a.out + 2 * (t * a.ldo + (int64_t)qh * a.dim + at)) =
          u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
    }
  }
  if (g == 0) {
    if (it.unit >= 0) {
      a.part_ml[2 * pr] = base;
      a.part_ml[2 * pr + 1] = l;
    } else if (a.lse) {
      a.lse[(int64_t)t * a.q_heads + qh] = l == 0.f ? kNegInf : (base + __log2f(l)) * kLn2;
    }
  }
}

// One item.  DP: head dimension rounded up to 64, 128 or 256 (the
// dimensions past a.dim are computed and dropped).  FP8: e4m3 cache, widened to bf16 (exactly) on the way in.
// CAREFUL as in run_tile.
template <int DP, bool FP8>
struct FewShape {
  static constexpr int KS = DP / 32;                   // k-steps of a score product
  static constexpr int LDV = DP + 16;                  // V row in LDS: 8 consecutive rows cover all 64 banks
  static constexpr int CPR = FP8 ? DP / 16 : DP / 8;   // 16-byte pieces of a V row
  static constexpr int VROWS = 64 / CPR;               // V rows per load of the wave
  static constexpr int NV = kStep / VROWS;
  static constexpr int KL = FP8 ? KS / 2 : KS;         // 16-byte loads of one key's share of a lane
  static constexpr int REGION = kStep * LDV;           // LDS elements of a wave
};

template <int DP, bool FP8, bool GENERAL, bool CAREFUL>
__device__ __forceinline__ bool run_few(const AttnArgs &a, const AttnItem &it, int h, uint16_t *vl) {
  using S = FewShape<DP, FP8>;
  const int lane = thread_of_item() % kWave, g = lane / 16, c = lane % 16;
  const int kvh = a.by_kv_parts.quotient(h);
  const bool row_ok = c < it.ntok * a.group;
  const int nth = row_ok ? a.by_group.quotient(c) : 0;
  const int tok = it.tok0 + nth, qh = h * a.group + (row_ok ? c - nth * a.group : 0);

  // lane j looks up key j of a step (both halves of the wave alike); beyond the
  // range the last key again, never seen
  const int32_t *table = a.cache.table + it.seq * a.cache.table_stride;
  auto page_of = [&](int step) -> int32_t {
    const int key = min(it.key0 + step * kStep + lane % kStep, it.key1 - 1);
    return table[a.cache.page_size.quotient(key)];
  };
  const char *k_head = a.cache.k + kvh * a.cache.head_bytes, *v_head = a.cache.v + kvh * a.cache.head_bytes;
  const int nsteps = (it.key1 - it.key0 + kStep - 1) / kStep;

  int32_t page = 0, page_next = 0;
  if (nsteps > 0) {
    page = page_of(0);
    page_next = page_of(1);
  }

  // Q: this row's share of the dimensions, in the order the K loads deliver them
  bf16x8 q[S::KS];
#pragma unroll
  for (int s = 0; s < S::KS; ++s) {
    const int d = FP8 ? 64 * (s / 2) + 16 * g + 8 * (s % 2) : 32 * s + 8 * g;
    u32x4 w = {0, 0, 0, 0};
    if (row_ok && d < a.dim) w = gload16(a.q + 2 * (tok * a.ldq + (int64_t)qh * a.dim + d));
    q[s] = __builtin_bit_cast(bf16x8, w);
  }
  // past the head dimension the first piece again: Q is zero there, and O^T's
  // rows there are not stored
  auto k_ok = [&](int s) { return (FP8 ? 64 * s + 16 * g : 32 * s + 8 * g) < a.dim; };
  int lo = 0, hi = 0, pos = 0;
  if (row_ok) {
    const int4 v = reinterpret_cast<const int4 *>(a.limits)[tok];
    lo = max(v.x, it.key0), hi = min(v.y, it.key1), pos = v.z;
  }
  const uint32_t span = (uint32_t)max(hi - lo, 0);
  const ScoreArgs sc = score_args<GENERAL>(a, kvh, qh);
  const float mul = GENERAL ? 1.f : sc.mul;  // st * mul: base-2 logits

  u32x4 kr[2][S::KL], vr[S::NV];
  uint32_t good = 0;  // CAREFUL: keys of the issued step in a good page
  bool odd = false;   // met what CAREFUL = false does not handle
  auto issue = [&](int step, int32_t pid) {
    const int key = it.key0 + step * kStep + lane % kStep;
    const int64_t off = key_offset(a.cache, min(key, it.key1 - 1), pid);
    if constexpr (CAREFUL) good = (uint32_t)__ballot(off >= 0 && key < it.key1);
    else odd |= off < 0;
    const int64_t at = max((int64_t)0, off);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t o = __shfl(at, 16 * t + c);
#pragma unroll
      for (int s = 0; s < S::KL; ++s)
        kr[t][s] = gload16(k_head + o + (k_ok(s) ? (FP8 ? 64 * s + 16 * g : 2 * (32 * s + 8 * g)) : 0));
    }
    const int vc = lane % S::CPR;
    const int vcol = 16 * vc < a.dim * (FP8 ? 1 : 2) ? 16 * vc : 0;
#pragma unroll
    for (int i = 0; i < S::NV; ++i) vr[i] = gload16(v_head + __shfl(at, S::VROWS * i + lane / S::CPR) + vcol);
  };

  float base = kNegInf, l = 0.f;
  f32x4 o[DP / 16];
#pragma unroll
  for (int d = 0; d < DP / 16; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (nsteps > 0) issue(0, page);
  for (int step = 0; step < nsteps; ++step) {
    const int k0 = it.key0 + step * kStep;
    const bool masked = CAREFUL || k0 < it.full0 || k0 + kStep > min(it.full1, it.key1);
    // ---- scores
    f32x4 st[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      st[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < S::KL; ++s) {
        const u32x4 w = kr[t][s];
        if constexpr (FP8) {
          st[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, e4m3x8_to_bf16(w[0], w[1])),
                                                          q[2 * s], st[t], 0, 0, 0);
          st[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, e4m3x8_to_bf16(w[2], w[3])),
                                                          q[2 * s + 1], st[t], 0, 0, 0);
        } else {
          st[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), q[s], st[t], 0, 0, 0);
        }
      }
    }
    // ---- V to LDS; rows that are no keys as zeros
    bool poison = false;
#pragma unroll
    for (int i = 0; i < S::NV; ++i) {
      const int r = S::VROWS * i + lane / S::CPR;
      u32x4 w = vr[i];
      if (CAREFUL ? !((good >> r) & 1) : masked && k0 + r >= it.key1) w = u32x4{0, 0, 0, 0};
      uint16_t *p = vl + r * S::LDV + (lane % S::CPR) * (FP8 ? 16 : 8);
      if constexpr (FP8) {
        const u32x4 w0 = e4m3x8_to_bf16(w[0], w[1]), w1 = e4m3x8_to_bf16(w[2], w[3]);
        if (masked) poison |= any_nonfinite(w0) || any_nonfinite(w1);
        *reinterpret_cast<u32x4 *>(p) = w0;
        *reinterpret_cast<u32x4 *>(p + 8) = w1;
      } else {
        if (masked) poison |= any_nonfinite(w);
        *reinterpret_cast<u32x4 *>(p) = w;
      }
    }
    if (!CAREFUL) odd |= poison;
    poison = CAREFUL && __any(poison);
    const uint32_t good_now = good;
    // ---- the next step's loads
    if (step + 1 < nsteps) {
      issue(step + 1, page_next);
      page_next = page_of(step + 2);
    }
    // ---- softmax
    if constexpr (GENERAL) {
      const int away = pos - (k0 + 4 * g);
#pragma unroll
      for (int t = 0; t < 2; ++t) general_logits<4>(sc, st[t], [&](int i) { return away - (16 * t + i); });
    }
    uint32_t see = 0xff;  // of this lane's keys (bit 4 t + i)
    if (masked) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = 16 * t + 4 * g + i;
          const bool hide = (uint32_t)(k0 + j - lo) >= span || (CAREFUL && !((good_now >> j) & 1));
          if (hide) {
            st[t][i] = kNegInf;
            see &= ~(1u << (4 * t + i));
          }
        }
    }
    float top = max3(st[0][0], st[0][1], st[0][2]);
    top = max3(top, st[0][3], st[1][0]);
    top = max3(top, st[1][1], st[1][2]);
    top = max_rows(max3(top, top, st[1][3])) * mul;
    if (__any(!(top <= base + kSlack) && top > kNegInf)) {
      const float next = fmaxf(base, top);
      const float fade = next > kNegInf ? exp2_fast(base - next) : 1.f;
      base = next;
      l *= fade;
#pragma unroll
      for (int d = 0; d < DP / 16; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][i] *= fade;
    }
    const float minus = base == kNegInf ? 0.f : -base;
    u32x4 pw, rest;  // the weights in bf16; what that leaves out
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        st[t][i] = exp2_fast(__builtin_fmaf(st[t][i], mul, minus));
        l += st[t][i];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w = pack_bf16x2(st[t][2 * i], st[t][2 * i + 1]);
        pw[2 * t + i] = w;
        rest[2 * t + i] = pack_bf16x2(st[t][2 * i] - __uint_as_float(w << 16), st[t][2 * i + 1] - __uint_as_float(w & 0xffff0000u));
      }
    }
    const bf16x8 p = __builtin_bit_cast(bf16x8, pw), p_rest = __builtin_bit_cast(bf16x8, rest);
    // ---- O^T += V^T P^T
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) {
      const uint16_t *b = vl + (4 * g + c / 4) * S::LDV + 16 * d + 4 * (c % 4);
      const u32x2 v0 = lds_read_tr(b), v1 = lds_read_tr(b + 16 * S::LDV);
      u32x4 v = {v0.x, v0.y, v1.x, v1.y};
      if (CAREFUL && poison) {
        u32x4 seen;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          seen[i] = ((see >> (2 * i)) & 1 ? 0x3f80u : 0u) | ((see >> (2 * i + 1)) & 1 ? 0x3f800000u : 0u);
        const bf16x8 sb = __builtin_bit_cast(bf16x8, seen);
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        const f32x4 pi = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v_part(v, kVPosInf)), sb, zero, 0, 0, 0);
        const f32x4 ni = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v_part(v, kVNegInf)), sb, zero, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][i] = add_counted_infs(o[d][i], pi[i], ni[i]);
        v = v_part(v, kVFinite);
      }
      o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v), p_rest, o[d], 0, 0, 0);
      o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v), p, o[d], 0, 0, 0);
    }
  }

  if (!CAREFUL && __any(odd)) return true;
  finish_few<DP, uint16_t>(a, it, h, lane, o, base, sum_rows(l));
  return false;
}

// fp32 queries and cache: the same products with v_mfma_f32_16x16x4_f32 (one
// value of each operand a lane), 16 keys per wave and step.  Every call with an
// fp32 cache comes here, in tiles of 16 rows.
template <int DP, bool GENERAL>
__device__ __forceinline__ void run_few_f32(const AttnArgs &a, const AttnItem &it, int h) {
  constexpr int NC = DP / 16;  // 16-byte loads of one key's share of a lane
  const int lane = thread_of_item() % kWave, g = lane / 16, c = lane % 16;
  const int kvh = a.by_kv_parts.quotient(h);
  const bool row_ok = c < it.ntok * a.group;
  const int nth = row_ok ? a.by_group.quotient(c) : 0;
  const int tok = it.tok0 + nth, qh = h * a.group + (row_ok ? c - nth * a.group : 0);
  const int32_t *table = a.cache.table + it.seq * a.cache.table_stride;
  const char *k_head = a.cache.k + kvh * a.cache.head_bytes, *v_head = a.cache.v + kvh * a.cache.head_bytes;
  const int nsteps = (it.key1 - it.key0 + 15) / 16;

  f32x4 q[NC];
#pragma unroll
  for (int s = 0; s < NC; ++s) {
    const int d = 16 * s + 4 * g;
    q[s] = row_ok && d < a.dim ? gload16f(a.q + 4 * (tok * a.ldq + (int64_t)qh * a.dim + d)) : f32x4{0.f, 0.f, 0.f, 0.f};
  }
  int lo = 0, hi = 0, pos = 0;
  if (row_ok) {
    const int4 v = reinterpret_cast<const int4 *>(a.limits)[tok];
    lo = v.x, hi = v.y, pos = v.z;
  }
  const ScoreArgs sc = score_args<GENERAL>(a, kvh, qh);

  auto page_of = [&](int step) -> int32_t {
    const int key = it.key0 + step * 16 + c;
    return key < it.key1 ? table[a.cache.page_size.quotient(key)] : -1;
  };
  int32_t page = page_of(0);
  float m = kNegInf, l = 0.f;
  f32x4 o[NC];
#pragma unroll
  for (int d = 0; d < NC; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int step = 0; step < nsteps; ++step) {
    const int k0 = it.key0 + step * 16;
    const int key_c = k0 + c;
    const int64_t off = key_offset(a.cache, key_c, page);
    page = page_of(step + 1);
    const uint64_t good = __ballot(off >= 0);
    f32x4 kr[NC];
#pragma unroll
    for (int s = 0; s < NC; ++s) {
      const int d = 16 * s + 4 * g;
      kr[s] = d < a.dim ? gload16f(k_head + max((int64_t)0, off) + 4 * d) : f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // V of keys 4g + i: column c of every 16 dimensions
    float vr[4][NC];
    bool poison = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t ov = __shfl(off, 4 * g + i);
#pragma unroll
      for (int d = 0; d < NC; ++d) {
        vr[i][d] = ov >= 0 && 16 * d + c < a.dim
                       ? *(const __attribute__((address_space(1))) float *)(v_head + ov + 4 * (16 * d + c))
                       : 0.f;
        poison |= !(fabsf(vr[i][d]) < __builtin_inff());
      }
    }
    f32x4 st = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < NC; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) st = __builtin_amdgcn_mfma_f32_16x16x4f32(kr[s][e], q[s][e], st, 0, 0, 0);
    float top = m, seen[4];
    if constexpr (GENERAL) general_logits<4>(sc, st, [&](int i) { return pos - (k0 + 4 * g + i); });
    else st *= sc.mul;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 4 * g + i, key = k0 + j;
      const bool see = key >= lo && key < hi && key < it.key1 && ((good >> j) & 1);
      seen[i] = see ? 1.f : 0.f;
      st[i] = see ? st[i] : kNegInf;
      top = fmaxf(top, st[i]);
    }
    top = max_rows(top);
    const float base = top == kNegInf ? 0.f : top;
    const float fade = exp2_fast(m - base);
    m = top;
    l *= fade;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      st[i] = exp2_fast(st[i] - base);
      l += st[i];
    }
    const bool bad = __any(poison);
#pragma unroll
    for (int d = 0; d < NC; ++d) {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[d][i] *= fade;
      if (__builtin_expect(!bad, 1)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d] = __builtin_amdgcn_mfma_f32_16x16x4f32(vr[i][d], st[i], o[d], 0, 0, 0);
      } else {
        f32x4 pi = {0.f, 0.f, 0.f, 0.f}, ni = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = vr[i][d], inf = __builtin_inff();
          const bool nan = v != v;
          o[d] = __builtin_amdgcn_mfma_f32_16x16x4f32(nan || fabsf(v) == inf ? 0.f : v, st[i], o[d], 0, 0, 0);
          pi = __builtin_amdgcn_mfma_f32_16x16x4f32(nan || v == inf ? 1.f : 0.f, seen[i], pi, 0, 0, 0);
          ni = __builtin_amdgcn_mfma_f32_16x16x4f32(nan || v == -inf ? 1.f : 0.f, seen[i], ni, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][i] = add_counted_infs(o[d][i], pi[i], ni[i]);
      }
    }
  }
  finish_few<DP, float>(a, it, h, lane, o, m, sum_rows(l));
}

}  // namespace

}  // namespace lora
