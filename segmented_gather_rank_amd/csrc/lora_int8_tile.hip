// lora_int8_tile.hip -- 8-bit products of many rows: tiles of rows and columns, whose
// operands go through LDS.
//
// Bound, for a large dense batch: power.  17705 rows x 4096 x 28672 take 1.61 to 1.67 ms,
// 2490 to 2580 TOP/s at a clock of some 1.8 GHz, with the matrix cores busy 76 % of the
// cycles (a library product of 8192^3 in 8 bits: 2134 TOP/s).  Tiles of 256 x 256 on
// eight waves of 128 x 64: a byte from LDS feeds as many products as registers allow.
// Two stages alternate; transfers go straight to LDS and have a stage's products to
// arrive in.  16x16x64 products are faster than 32x32x32 with the same operands (1690 and
// 1870 us), four waves of 128 x 128 slower than eight (2340 and 1870 then), transfers by
// address slower than by buffer (1670 and 1620), and stages without the placement of
// pieces below meet in LDS banks (2030 and 1890).
//
// By expert, tiles are 128 x 128 unless segments are long (lora_base_host.h): 4609 tokens
// x 8 choices, an eighth of the experts here, x 2048 x 7168: 137 us of the call's 156, 3.9
// TB/s, with the matrix cores busy 28 %.  Neither bytes nor products bound it alone (a third
// of the tiles' rows are past their segments; with nothing to load it still takes 100),
// but a tile's 16 stages with a barrier each, its start and its results' way out, beside
// the weights' stream.  Longer segments take tiles of 256: 17705 tokens, 521 rows a segment,
// 347 us (products alone would take 229), and x 7168 x 4096 544 us (459).  Other tiles
// for the mixed step: 128 x 256 159 us, 128 x 192 173, 64 x 256 194, 64 x 128 211; two stages
// on their way, through registers: 154.
#include <algorithm>

#include "lora_int8_tile.h"

namespace lora {

namespace {

template <typename Y, bool GROUPED, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void tile_kernel(Int8Args a) {
  constexpr int kWaves = WM * WN;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;          // blocks of 16 of a wave
  constexpr int XQ = BM / 8 / kWaves, WQ = BN / 8 / kWaves;    // transfers of 8 rows of a wave and stage
  __shared__ u32x4 buf0[(BM + BN) * kPieces], buf1[(BM + BN) * kPieces];
  __shared__ __align__(16) float columns[kWaves][2 * TN * 16];
  extern __shared__ __align__(16) char table[];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane % 16, quarter = lane / 16;
  const TileList<GROUPED, BM, BN> list(a, table);
  int index = list.index;
  if (index >= list.last) return;

  // ---- transfers of the tile that `aim` was called for
  rsrc_t xb, wb;                                  // from where its rows of either operand are counted
  uint32_t xo[XQ], wo[WQ];                        // bytes from there to the piece of its row that a lane transfers
  // A row's piece p lies at place p ^ (row / 2 % 8) of its 8: the same piece of 16 neighbouring rows fills the 64 banks.
  // A transfer takes 8 rows, 8 (wave + kWaves q) and on.
  static_assert(kWaves % 2 == 0, "the place of a lane's piece is the same in all transfers");
  auto piece_of = [&](int lane) { return (lane % 8) ^ (4 * (wave % 2) + lane / 16); };
  int32_t row_of[XQ];                             // rows that this lane will transfer, of the tile that was looked up
  auto look_up = [&](const Tile &t) {
#pragma unroll
    for (int q = 0; q < XQ; ++q) {
      const int r = min(t.m0 + (q * kWaves + wave) * 8 + lane / 8, t.count - 1);
      if constexpr (GROUPED) row_of[q] = a.meta.sorted[t.start + r];
      else row_of[q] = r - t.m0;
    }
  };
  auto aim = [&](const Tile &t) {
    int lane = threadIdx.x % 64;  // hidden, as in `store_tile`
    asm volatile("" : "+v"(lane));
    const int piece = piece_of(lane);
    xb = make_rsrc(GROUPED ? a.x : a.x + (int64_t)t.m0 * a.ldx, kNowhere - 1);
#pragma unroll
    for (int q = 0; q < XQ; ++q) {
      uint32_t row = (uint32_t)row_of[q];
      if (GROUPED && a.meta.x_row_div != 1) row /= (uint32_t)a.meta.x_row_div;
      xo[q] = row * (uint32_t)a.ldx + 16 * piece;
    }
    wb = make_rsrc(a.w + t.expert * a.expert_stride + t.n0 * a.row_stride, kNowhere - 1);
#pragma unroll
    for (int q = 0; q < WQ; ++q)
      wo[q] = (uint32_t)min((q * kWaves + wave) * 8 + lane / 8, a.d_out - 1 - t.n0) * (uint32_t)a.row_stride + 16 * piece;
  };
  // a stage's transfers where d_in may end
  auto transfer_end = [&](u32x4 *buf, int k) {
    const bool in = k + 16 * piece_of(lane) < a.d_in;
#pragma unroll
    for (int q = 0; q < XQ; ++q) to_lds(xb, in ? xo[q] : kNowhere, k, buf + (q * kWaves + wave) * 64);
#pragma unroll
    for (int q = 0; q < WQ; ++q) to_lds(wb, in ? wo[q] : kNowhere, k, buf + BM * kPieces + (q * kWaves + wave) * 64);
  };

  // ---- products: a stage is two phases of 64 bytes.  A block of x's operands is overwritten
  // with the next phase's as soon as its products are on their way; w's have two sets.
  static_assert(TM >= TN, "w's operands are read along with x's");
  i32x4 sum[TM][TN];
  i32x4 xv[TM], wv[2][TN];
  const int xr = (wm * TM * 16 + l16) * kPieces + (quarter ^ (l16 / 2));
  const int wr = (BM + wn * TN * 16 + l16) * kPieces + (quarter ^ (l16 / 2));
  auto read_x = [&](const u32x4 *buf, int phase, int m) {
    xv[m] = __builtin_bit_cast(i32x4, buf[(xr ^ (4 * phase)) + m * 16 * kPieces]);
  };
  auto read_w = [&](const u32x4 *buf, int phase, int n) {
    wv[phase][n] = __builtin_bit_cast(i32x4, buf[(wr ^ (4 * phase)) + n * 16 * kPieces]);
  };
  auto multiply = [&](int phase, int m) {
#pragma unroll
    for (int n = 0; n < TN; ++n)
      sum[m][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[phase][n], xv[m], sum[m][n], 0, 0, 0);
  };
  // the next phase's operands that are read behind block m's products
  auto refill = [&](const u32x4 *buf, int phase, int m) {
    if (m < TN) read_w(buf, phase, m);
    read_x(buf, phase, m);
  };
  constexpr int kEarly = 2;      // blocks of the second phase that are multiplied before the barrier
  auto first_phase = [&](const u32x4 *here) {
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      multiply(0, m);
      refill(here, 1, m);
      __builtin_amdgcn_sched_barrier(0);  // in this order: a read that is moved back is waited for too early
    }
  };
  // the second phase's operands are in registers by the barrier, so that the transfers of the
  // stage after the next may overwrite this one's place
  auto stage = [&](u32x4 *here, const u32x4 *next, int k) {
    first_phase(here);
#pragma unroll
    for (int m = 0; m < kEarly; ++m) multiply(1, m);
    __builtin_amdgcn_sched_barrier(0);
    settle();
    k += 2 * kDepth;
#pragma unroll
    for (int m = 0; m < kEarly; ++m) refill(next, 0, m);
#pragma unroll
    for (int m = kEarly; m < TM; ++m) {
      multiply(1, m);
      refill(next, 0, m);
#pragma unroll
      for (int q = 0; q < XQ; ++q)
        if (kEarly + q * (TM - kEarly) / (XQ + WQ) == m) to_lds(xb, xo[q], k, here + (q * kWaves + wave) * 64);
#pragma unroll
      for (int q = 0; q < WQ; ++q)
        if (kEarly + (XQ + q) * (TM - kEarly) / (XQ + WQ) == m)
          to_lds(wb, wo[q], k, here + BM * kPieces + (q * kWaves + wave) * 64);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const int stages = (a.d_in + kDepth - 1) / kDepth, whole = a.d_in / kDepth;
  // a stage that may be among a tile's last ones
  auto stage_end = [&](u32x4 *here, const u32x4 *next, int s) {
    first_phase(here);
    const bool goes_on = s + 1 < stages;
    if (goes_on) {
      settle();
      if (s + 2 < stages) transfer_end(here, (s + 2) * kDepth);
    }
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      multiply(1, m);
      if (goes_on) refill(next, 0, m);
    }
  };

  Tile now = list.at(index), then;
  look_up(now);
  aim(now);
  transfer_end(buf0, 0);
  while (true) {
    const bool follows = index + list.per < list.last;
    if (follows) {
      then = list.at(index + list.per);
      look_up(then);
    }
    settle();         // the first stage is there, and the last tile's scratch is free
    if (stages > 1) transfer_end(buf1, kDepth);
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int n = 0; n < TN; ++n) sum[m][n] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int m = 0; m < TM; ++m) refill(buf0, 0, m);
    int s = 0;
    for (; s + 3 < whole; s += 2) {
      stage(buf0, buf1, s * kDepth);
      stage(buf1, buf0, (s + 1) * kDepth);
    }
    while (true) {
      stage_end(buf0, buf1, s);
      if (++s == stages) break;
      stage_end(buf1, buf0, s);
      if (++s == stages) break;
    }
    __syncthreads();  // every wave has read its last stage
    // the next tile's first stage arrives while this one's results leave
    if (follows) {
      aim(then);
      transfer_end(buf0, 0);
    }
    constexpr int kRowPieces = TN * 16 * (int)sizeof(Y) / 16;
    static_assert(kWaves * 32 * kRowPieces <= (BM + BN) * kPieces, "the waves' rows fit the stage");
    store_tile<Y, GROUPED, TM, TN>(a, now, sum, wm * TM * 16, now.n0 + wn * TN * 16, buf1 + wave * 32 * kRowPieces,
                                   columns[wave]);
    if (!follows) return;
    now = then;
    index += list.per;
  }
}

template <typename Y, bool GROUPED, int BM, int BN, int WM, int WN>
hipError_t launch_as(const Int8Args &a, hipStream_t s) {
  static std::atomic<int> cache[2][kMaxDevices];
  // workgroups that fit a CU go by the length of the table of segments
  const bool wide = a.experts > 256;
  const size_t lds = GROUPED ? seg_table_bytes(wide ? kMaxSlots : 256) : 0;
  const void *f = reinterpret_cast<const void *>(&tile_kernel<Y, GROUPED, BM, BN, WM, WN>);
  const int64_t cols = (a.d_out + BN - 1) / BN;
  const int64_t bound = ((a.rows + BM - 1) / BM + (GROUPED ? std::min<int64_t>(a.experts, a.rows) : 0)) * cols;
  const int grid = xcd_grid(bound, resident_groups(cache[wide], f, 64 * WM * WN, lds));
  tile_kernel<Y, GROUPED, BM, BN, WM, WN><<<dim3((unsigned)grid), dim3(64 * WM * WN), lds, s>>>(a);
  return hipGetLastError();
}

template <typename Y>
hipError_t launch_for(const Int8Args &a, hipStream_t s) {
  if (!a.meta.sorted) {
    // tiles of 256 from half a chip of them on (4096 x 6144: 1500 rows 45 us; below, four times as many of 128)
    const int64_t tiles = (a.rows + 255) / 256 * ((a.d_out + 255) / 256);
    return tiles > 128 ? launch_as<Y, false, 256, 256, 2, 4>(a, s) : launch_as<Y, false, 128, 128, 2, 2>(a, s);
  }
  const hipError_t err = launch_as<Y, true, 128, 128, 2, 2>(a, s);
  // (no average reaches 160 rows where there are fewer)
  return err != hipSuccess || a.rows <= 160 ? err : launch_as<Y, true, 256, 256, 2, 4>(a, s);
}

}  // namespace

hipError_t launch_int8_tile(const Int8Args &a, bool bf16, hipStream_t s) {
  return bf16 ? launch_for<uint16_t>(a, s) : launch_for<float>(a, s);
}

}  // namespace lora
