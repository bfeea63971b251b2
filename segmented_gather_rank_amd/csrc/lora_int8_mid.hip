// lora_int8_mid.hip -- 8-bit products of dense batches that large tiles would not spread
// over the chip: tiles of 64 x 64, whose operands wait in registers for their place in LDS.
//
// Neither bytes nor the matrix cores (busy a sixth of the time) bound such a product, but
// the way of a stage: from memory, to LDS, past a barrier, to the products.  Tiles are
// small, so that every CU has some, two workgroups share a CU, and a workgroup keeps two
// stages of its operands on their way at all times, across the ends of its tiles.  (They
// go through registers: the compiler waits for those one by one, while it cannot tell
// transfers to a ring in LDS apart.)  256 rows x 4096 x 6144: 16.4 us, 790 TOP/s; in
// tiles of 64 x 128 17.7, of 128 x 128 25, with four stages on their way 17, six 19, with
// stages of 256 bytes 18.
#include <algorithm>

#include "lora_int8_tile.h"

namespace lora {

namespace {

template <typename Y, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void mid_kernel(Int8Args a) {
  constexpr int kWaves = WM * WN;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;          // blocks of 16 of a wave
  constexpr int XQ = BM / 8 / kWaves, WQ = BN / 8 / kWaves;    // transfers of 8 rows of a wave and stage
  static_assert(kWaves % 2 == 0, "a lane's piece is the same in all transfers");
  __shared__ u32x4 buf0[(BM + BN) * kPieces], buf1[(BM + BN) * kPieces];
  __shared__ __align__(16) float columns[kWaves][2 * TN * 16];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane % 16, quarter = lane / 16;
  const TileList<false, BM, BN> list(a, nullptr);
  if (list.index >= list.last) return;

  // ---- what is loaded: a tile at byte `lk` of d_in, then the next one of the list
  int loads = list.index, lk = 0;
  rsrc_t xb, wb;                              // from where the loaded tile's rows of either operand are counted
  uint32_t xo[XQ], wo[WQ];                    // bytes from there to the piece of its row that a lane loads
  const int piece = (lane % 8) ^ (4 * (wave % 2) + lane / 16);
  auto aim = [&](const Tile &t) {
    xb = make_rsrc(a.x + (int64_t)t.m0 * a.ldx, kNowhere - 1);
#pragma unroll
    for (int q = 0; q < XQ; ++q)
      xo[q] = (uint32_t)min((q * kWaves + wave) * 8 + lane / 8, t.count - 1 - t.m0) * (uint32_t)a.ldx + 16 * piece;
    wb = make_rsrc(a.w + t.n0 * a.row_stride, kNowhere - 1);
#pragma unroll
    for (int q = 0; q < WQ; ++q)
      wo[q] = (uint32_t)min((q * kWaves + wave) * 8 + lane / 8, a.d_out - 1 - t.n0) * (uint32_t)a.row_stride + 16 * piece;
  };
  // a stage's operands into a set of registers; zeros past the end of d_in, and of the list (no branch: a wait counts
  // the loads that came after what it waits for)
  u32x4 xs[2][XQ], ws[2][WQ];
  auto fetch = [&](int set) {
    const bool in = loads < list.last && lk + 16 * piece < a.d_in;
#pragma unroll
    for (int q = 0; q < XQ; ++q)
      xs[set][q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xb, (int)(in ? xo[q] : kNowhere), lk, 0));
#pragma unroll
    for (int q = 0; q < WQ; ++q)
      ws[set][q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wb, (int)(in ? wo[q] : kNowhere), lk, 0));
  };
  auto put = [&](int set, u32x4 *buf) {
#pragma unroll
    for (int q = 0; q < XQ; ++q) buf[(q * kWaves + wave) * 64 + lane] = xs[set][q];
#pragma unroll
    for (int q = 0; q < WQ; ++q) buf[BM * kPieces + (q * kWaves + wave) * 64 + lane] = ws[set][q];
  };
  // on to the stage after the one that was fetched
  auto advance = [&]() {
    lk += kDepth;
    if (lk < a.d_in || loads >= list.last) return;
    lk = 0;
    loads += list.per;
    if (loads < list.last) aim(list.at(loads));
  };

  // ---- products, as in the large tiles
  static_assert(TM >= TN, "w's operands are read along with x's");
  i32x4 sum[TM][TN];
  i32x4 xv[TM], wv[2][TN];
  const int xr = (wm * TM * 16 + l16) * kPieces + (quarter ^ (l16 / 2));
  const int wr = (BM + wn * TN * 16 + l16) * kPieces + (quarter ^ (l16 / 2));
  auto refill = [&](const u32x4 *buf, int phase, int m) {
    if (m < TN) wv[phase][m] = __builtin_bit_cast(i32x4, buf[(wr ^ (4 * phase)) + m * 16 * kPieces]);
    xv[m] = __builtin_bit_cast(i32x4, buf[(xr ^ (4 * phase)) + m * 16 * kPieces]);
  };
  auto multiply = [&](int phase, int m) {
#pragma unroll
    for (int n = 0; n < TN; ++n)
      sum[m][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[phase][n], xv[m], sum[m][n], 0, 0, 0);
  };
  auto clear = [&]() {
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int n = 0; n < TN; ++n) sum[m][n] = i32x4{0, 0, 0, 0};
  };

  Tile now = list.at(list.index);
  int index = list.index, left = a.d_in;
  // A stage, whose following one is in registers.
  auto stage = [&](u32x4 *here, u32x4 *following, int set) {
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      multiply(0, m);
      refill(here, 1, m);
    }
    put(set, following);
    fetch(set);
    advance();
    __syncthreads();
    left -= kDepth;
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      multiply(1, m);
      refill(following, 0, m);
    }
    if (left > 0 || index >= list.last) return;
    constexpr int kRowPieces = TN * 16 * (int)sizeof(Y) / 16;
    static_assert(kWaves * 32 * kRowPieces <= (BM + BN) * kPieces, "the waves' rows fit the stage");
    store_tile<Y, false, TM, TN>(a, now, sum, wm * TM * 16, now.n0 + wn * TN * 16, here + wave * 32 * kRowPieces,
                                   columns[wave]);
    __syncthreads();  // the waves' scratch is free
    index += list.per;
    if (index >= list.last) return;
    clear();
    now = list.at(index);
    left = a.d_in;
  };

  aim(now);
  fetch(0);
  advance();
  fetch(1);
  advance();
  put(0, buf0);
  __syncthreads();
  fetch(0);
  advance();
  clear();
#pragma unroll
  for (int m = 0; m < TM; ++m) refill(buf0, 0, m);
  // All stages of all tiles, two at a time, one more than there are if need be: a way out between the two would look to
  // the compiler like a way back as well, on which the first one's loads are the latest.
  const int stages = (list.last - list.index + list.per - 1) / list.per * ((a.d_in + kDepth - 1) / kDepth);
  for (int s = 0; s < stages; s += 2) {
    stage(buf0, buf1, 1);
    stage(buf1, buf0, 0);
  }
}

template <typename Y>
hipError_t launch_for(const Int8Args &a, hipStream_t s) {
  constexpr int BM = 64, BN = 64, WM = 2, WN = 4 / WM;
  static std::atomic<int> cache[kMaxDevices];
  const void *f = reinterpret_cast<const void *>(&mid_kernel<Y, BM, BN, WM, WN>);
  const int64_t tiles = ((a.rows + BM - 1) / BM) * ((a.d_out + BN - 1) / BN);
  const int grid = xcd_grid(tiles, resident_groups(cache, f, 64 * WM * WN, 0));
  mid_kernel<Y, BM, BN, WM, WN><<<dim3((unsigned)grid), dim3(64 * WM * WN), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_mid(const Int8Args &a, bool bf16, hipStream_t s) {
  return bf16 ? launch_for<uint16_t>(a, s) : launch_for<float>(a, s);
}

}  // namespace lora
