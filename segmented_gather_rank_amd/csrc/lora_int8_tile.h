// lora_int8_tile.h -- what the tile kernels of the 8-bit products share: the order of
// tiles, transfers to LDS, the way back from sums to rows of y.
#pragma once

#include "lora_base_host.h"

namespace lora {

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

// The list of tiles of BM rows and BN columns that a persistent grid walks: all of a dense
// batch, or of the segments that are not few_kernel's where the rule says tiles of BM.  Every
// XCD takes a run of neighbours.
template <bool GROUPED, int BM, int BN>
struct TileList {
  SegTable tb;
  int col_tiles, rows, index, last, per;  // this workgroup's tiles: index, index + per, ... below last
  __device__ __forceinline__ TileList(const Int8Args &a, char *table)
      : tb(seg_table_at(table, a.experts)), col_tiles((a.d_out + BN - 1) / BN), rows((int)a.rows) {
    int tiles;
    if constexpr (GROUPED) {
      const ExpertRule rule(a.meta, a.d_out);
      tiles = 0;
      if (rule.large == (BM > 128)) {
        build_items(a.meta, tb, true, [&](int count, int) { return count > rule.few ? (count + BM - 1) / BM * col_tiles : 0; });
        tiles = uniform_value(tb.scal[2]);
      }
    } else {
      tiles = (rows + BM - 1) / BM * col_tiles;
    }
    const int share = (tiles + 7) / 8;
    per = gridDim.x / 8;
    last = min(tiles, (int)(blockIdx.x % 8 + 1) * share);
    index = blockIdx.x % 8 * share + blockIdx.x / 8;
  }
  __device__ __forceinline__ Tile at(int i) const {
    Tile t;
    int m, n;
    if constexpr (GROUPED) {
      const int s = find_item_segment(tb, i), seg = tb.scal[1] + s;
      t.expert = uniform_value(tb.slot[seg]);
      t.count = uniform_value(tb.count[seg]);
      t.start = uniform_value(tb.start[seg]);
      const int from = s ? tb.item_end[s - 1] : 0;
      place(uniform_value(i - from), (t.count + BM - 1) / BM, col_tiles, m, n);
    } else {
      t.expert = t.start = 0;
      t.count = rows;
      place(i, (t.count + BM - 1) / BM, col_tiles, m, n);
    }
    t.m0 = m * BM;
    t.n0 = n * BN;
    return t;
  }
};

// y of a wave's TM x TN blocks of a finished tile, rows r0 and columns c0 on, through LDS so
// that whole lines are stored: 32 rows at a time.  `mine`: 32 rows in LDS, `columns`: 2 x 16 TN
// floats, both the wave's own.
template <typename Y, bool GROUPED, int TM, int TN>
__device__ __forceinline__ void store_tile(const Int8Args &a, const Tile &t, const i32x4 (&sum)[TM][TN], int r0, int c0,
                                           u32x4 *mine, float *columns) {
  constexpr int kRowPieces = TN * 16 * (int)sizeof(Y) / 16;
  // hidden from the optimiser, which would keep what follows from it in registers all through the products
  int lane = threadIdx.x % 64;
  asm volatile("" : "+v"(lane));
  const int l16 = lane % 16, quarter = lane / 16;
  // the pieces of a row change places by its number, so that neither the writes nor the reads meet in a bank
  auto turn = [&](int row) { return kRowPieces >= 16 ? row % kRowPieces : row * kRowPieces / 16 % kRowPieces; };
  // y's row of row r of the tile; past the last one the last one again
  auto row_id = [&](int r) -> uint32_t {
    const int i = min(t.m0 + r, t.count - 1);
    if constexpr (GROUPED) return (uint32_t)a.meta.sorted[t.start + i];
    else return (uint32_t)i;
  };
  // the wave's columns' scales and bias: fetched once, read from LDS as they are needed
  float *ws = columns, *bs = columns + TN * 16;
  for (int c = lane; c < TN * 16; c += 64) {
    const int64_t at = (int64_t)t.expert * a.d_out + min(c0 + c, a.d_out - 1);
    ws[c] = a.w_scale[at];
    bs[c] = a.bias ? a.bias[at] : 0.f;
  }
  wave_sync();
#pragma unroll
  for (int m = 0; m < TM; m += 2) {
    const int r = r0 + m * 16;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t row = row_id(r + 16 * b + l16);
      if (GROUPED && a.meta.x_row_div != 1) row /= (uint32_t)a.meta.x_row_div;
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
        gstore16(a.y + ((int64_t)row_id(r + lr) * a.ldy + c) * (int64_t)sizeof(Y), v);
      }
    }
    wave_sync();
  }
}

}  // namespace lora
