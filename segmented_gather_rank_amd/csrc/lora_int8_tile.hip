// lora_int8_tile.hip -- 8-bit products of many rows: tiles of rows and columns, whose
// operands go through LDS.
#include <algorithm>

#include "lora_base_host.h"

namespace lora {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kDepth = 128;  // bytes of d_in a stage holds of every row
constexpr int kPieces = kDepth / 16;

// An offset past the end of every buffer: a lane that transfers from there gets zeros.
constexpr uint32_t kNowhere = 0xffffffffu;

struct Tile {
  int expert, n0, m0, count, start;  // rows m0 .. of a segment of `count` rows from `start` in `sorted`
};

// Tile i of a rows x cols grid, taken `kBand` row tiles at a time, so that what is in
// work at once reads few different rows of either operand.
constexpr int kBand = 4;
__device__ __forceinline__ void place(int i, int row_tiles, int col_tiles, int &m, int &n) {
  const int band = i / (kBand * col_tiles), in = i - band * kBand * col_tiles;
  const int high = min(kBand, row_tiles - band * kBand);
  n = in / high;
  m = band * kBand + in - n * high;
}

// 16 bytes a lane from `at` + k of the buffer; `to` is the wave's.  (A transfer by address
// would count as an LDS operation too, and every wait for LDS would be one for all of them.)
__device__ __forceinline__ void to_lds(rsrc_t from, uint32_t at, int k, u32x4 *to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 16, (int)at, k, 0, 0);
}

// Every wave's transfers to LDS have arrived, and its reads have left.  (A barrier alone
// waits for LDS operations, not for transfers that memory still holds.)
__device__ __forceinline__ void settle() {
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
}

// LDS written by this wave is read by this wave.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <typename Y, bool GROUPED, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void tile_kernel(Int8Args a, int fewest) {
  constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;          // blocks of 16 of a wave
  constexpr int XQ = BM / 8 / kWaves, WQ = BN / 8 / kWaves;    // transfers of 8 rows of a wave and stage
  __shared__ u32x4 buf0[(BM + BN) * kPieces], buf1[(BM + BN) * kPieces];
  __shared__ int32_t ids[2][GROUPED ? BM : 1];
  __shared__ __align__(16) float columns[kWaves][2][TN * 16];
  extern __shared__ __align__(16) char table[];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane % 16, quarter = lane / 16;
  const int col_tiles = (a.d_out + BN - 1) / BN;
  const SegTable tb = seg_table_at(table, a.experts);
  int tiles;
  if constexpr (GROUPED) {
    build_items(a.meta, tb, true, [&](int count, int) { return count >= fewest ? (count + BM - 1) / BM * col_tiles : 0; });
    tiles = uniform_value(tb.scal[2]);
  } else {
    tiles = (int)((a.rows + BM - 1) / BM) * col_tiles;
  }
  // every XCD takes a run of neighbouring tiles
  const int share = (tiles + 7) / 8, per = gridDim.x / 8;
  const int last = min(tiles, (int)(blockIdx.x % 8 + 1) * share);
  int index = blockIdx.x % 8 * share + blockIdx.x / 8;
  if (index >= last) return;

  auto tile_at = [&](int i) {
    Tile t;
    int m, n;
    if constexpr (GROUPED) {
      const int s = find_item_segment(tb, i), at = tb.scal[1] + s;
      t.expert = uniform_value(tb.slot[at]);
      t.count = uniform_value(tb.count[at]);
      t.start = uniform_value(tb.start[at]);
      const int from = s ? tb.item_end[s - 1] : 0;
      place(uniform_value(i - from), (t.count + BM - 1) / BM, col_tiles, m, n);
    } else {
      t.expert = t.start = 0;
      t.count = (int)a.rows;
      place(i, (t.count + BM - 1) / BM, col_tiles, m, n);
    }
    t.m0 = m * BM;
    t.n0 = n * BN;
    return t;
  };

  // ---- transfers of the tile that `aim` was called for
  rsrc_t xb, wb;                                  // from where its rows of either operand are counted
  uint32_t xo[XQ], wo[WQ];                        // bytes from there to the piece of its row that a lane transfers
  // A row's piece p lies at place p ^ (row / 2 % 8) of its 8: the same piece of 16 neighbouring rows fills the 64 banks.
  // A transfer takes 8 rows, 8 (wave + kWaves q) and on.
  static_assert(kWaves % 2 == 0, "the place of a lane's piece is the same in all transfers");
  auto piece_of = [&](int lane) { return (lane % 8) ^ (4 * (wave % 2) + lane / 16); };
  constexpr int kIds = (BM + kThreads - 1) / kThreads;
  int32_t pending[kIds];
  auto fetch_ids = [&](const Tile &t) {
    if constexpr (GROUPED) {
#pragma unroll
      for (int q = 0; q < kIds; ++q)
        pending[q] = a.meta.sorted[t.start + min(t.m0 + q * kThreads + (int)threadIdx.x, t.count - 1)];
    }
  };
  auto keep_ids = [&](int slot) {
    if constexpr (GROUPED) {
#pragma unroll
      for (int q = 0; q < kIds; ++q)
        if (q * kThreads + (int)threadIdx.x < BM) ids[slot][q * kThreads + threadIdx.x] = pending[q];
    }
  };
  auto aim = [&](const Tile &t, int slot) {
    int lane = threadIdx.x % 64;  // hidden, as in `finish` below
    asm volatile("" : "+v"(lane));
    const int piece = piece_of(lane);
    xb = make_rsrc(GROUPED ? a.x : a.x + (int64_t)t.m0 * a.ldx, kNowhere - 1);
#pragma unroll
    for (int q = 0; q < XQ; ++q) {
      const int r = (q * kWaves + wave) * 8 + lane / 8;
      uint32_t row;
      if constexpr (GROUPED) {
        row = (uint32_t)ids[slot][r];
        if (a.meta.x_row_div != 1) row /= (uint32_t)a.meta.x_row_div;
      } else {
        row = (uint32_t)min(r, t.count - 1 - t.m0);
      }
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

  // ---- y of the finished tile, through LDS so that whole lines are stored: 32 rows at a time
  auto finish = [&](const Tile &t, int slot, u32x4 *scratch) {
    constexpr int kRowPieces = TN * 16 * (int)sizeof(Y) / 16;
    u32x4 *mine = scratch + wave * 32 * kRowPieces;
    // hidden from the optimiser, which would keep what follows from it in registers all through the products
    int lane = threadIdx.x % 64;
    asm volatile("" : "+v"(lane));
    const int l16 = lane % 16, quarter = lane / 16;
    // the pieces of a row change places by its number, so that neither the writes nor the reads meet in a bank
    auto turn = [&](int row) { return kRowPieces >= 16 ? row % kRowPieces : row * kRowPieces / 16 % kRowPieces; };
    const int c0 = t.n0 + wn * TN * 16;
    // the wave's columns' scales and bias: fetched once, read from LDS as they are needed
    float *ws = columns[wave][0], *bs = columns[wave][1];
    for (int c = lane; c < TN * 16; c += 64) {
      const int64_t at = (int64_t)t.expert * a.d_out + min(c0 + c, a.d_out - 1);
      ws[c] = a.w_scale[at];
      bs[c] = a.bias ? a.bias[at] : 0.f;
    }
    wave_sync();
#pragma unroll
    for (int m = 0; m < TM; m += 2) {
      const int r = (wm * TM + m) * 16;           // of the tile
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t row = (uint32_t)min(t.m0 + r + 16 * b + l16, t.count - 1);
        if constexpr (GROUPED) {
          row = (uint32_t)ids[slot][r + 16 * b + l16];
          if (a.meta.x_row_div != 1) row /= (uint32_t)a.meta.x_row_div;
        }
        const float xs = a.x_scale[row];
        u32x4 *line = mine + (16 * b + l16) * kRowPieces;
        const int places = turn(16 * b + l16);
#pragma unroll
        for (int n = 0; n < TN; ++n) {
          // columns 16 n + 4 quarter .. + 3 of the row
          const f32x4 w4 = *reinterpret_cast<const f32x4 *>(ws + 16 * n + 4 * quarter);
          const f32x4 b4 = *reinterpret_cast<const f32x4 *>(bs + 16 * n + 4 * quarter);
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = (float)sum[m + b][n][e] * (xs * w4[e]) + b4[e];
          if constexpr (sizeof(Y) == 2) {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            u32x2 *to = reinterpret_cast<u32x2 *>(line + ((2 * n + quarter / 2) ^ places));
            to[quarter % 2] = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
          } else {
            line[(4 * n + quarter) ^ places] = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
          }
        }
      }
      wave_sync();
      constexpr int kRowsAtOnce = 64 / kRowPieces;
#pragma unroll
      for (int q = 0; q < 32 / kRowsAtOnce; ++q) {
        const int lr = q * kRowsAtOnce + lane / kRowPieces, p = lane % kRowPieces;
        const u32x4 v = mine[lr * kRowPieces + (p ^ turn(lr))];
        const int c = c0 + p * (16 / (int)sizeof(Y));
        if (t.m0 + r + lr < t.count && c < a.d_out) {
          int64_t to = t.m0 + r + lr;
          if constexpr (GROUPED) to = (uint32_t)ids[slot][r + lr];
          gstore16(a.y + (to * a.ldy + c) * (int64_t)sizeof(Y), v);
        }
      }
      wave_sync();
    }
  };

  Tile now = tile_at(index), then;
  int slot = 0;
  if constexpr (GROUPED) {
    fetch_ids(now);
    keep_ids(0);
    __syncthreads();
  }
  aim(now, 0);
  transfer_end(buf0, 0);
  while (true) {
    const bool follows = index + per < last;
    if (follows) {
      then = tile_at(index + per);
      fetch_ids(then);
    }
    settle();         // the first stage is there, and the last tile's scratch is free
    if (follows) keep_ids(slot ^ 1);
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
      aim(then, slot ^ 1);
      transfer_end(buf0, 0);
    }
    finish(now, slot, buf1);
    if (!follows) return;
    now = then;
    slot ^= 1;
    index += per;
  }
}

template <typename Y, bool GROUPED, int BM, int BN, int WM, int WN>
hipError_t launch_as(const Int8Args &a, int fewest, hipStream_t s) {
  static std::atomic<int> cache[kMaxDevices];
  // the table's size only matters where it costs a workgroup its place: sized for the most
  const size_t lds = GROUPED ? seg_table_bytes(a.experts) : 0;
  const void *f = reinterpret_cast<const void *>(&tile_kernel<Y, GROUPED, BM, BN, WM, WN>);
  const int64_t cols = (a.d_out + BN - 1) / BN;
  const int64_t bound = ((a.rows + BM - 1) / BM + (GROUPED ? std::min<int64_t>(a.experts, a.rows) : 0)) * cols;
  const int grid = xcd_grid(bound, resident_groups(cache, f, 64 * WM * WN, lds));
  tile_kernel<Y, GROUPED, BM, BN, WM, WN><<<dim3((unsigned)grid), dim3(64 * WM * WN), lds, s>>>(a, fewest);
  return hipGetLastError();
}

template <typename Y>
hipError_t launch_for(const Int8Args &a, int fewest, hipStream_t s) {
  if (a.meta.sorted) return launch_as<Y, true, 256, 256, 2, 4>(a, fewest, s);
  return launch_as<Y, false, 256, 256, 2, 4>(a, fewest, s);
}

}  // namespace

hipError_t launch_int8_tile(const Int8Args &a, bool bf16, int fewest, hipStream_t s) {
  return bf16 ? launch_for<uint16_t>(a, fewest, s) : launch_for<float>(a, fewest, s);
}

}  // namespace lora
