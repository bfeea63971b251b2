// lora_attn.h -- plan arithmetic and argument blocks of the paged attention
// kernels and of the cache append.  Internal to the library (not part of the
// ABI).  Everything marked LORA_HD is plain integer arithmetic that also
// compiles for the host alone, where the CPU tests check it against the sizes
// of the buffers it indexes.
#pragma once

#include <stdint.h>

#if defined(__HIP__)
#include <hip/hip_runtime.h>
#define LORA_HD __host__ __device__ __forceinline__
#else
#define LORA_HD inline
#endif

namespace lora {

// Rows (query token x query head) of one work item: the few-row kernel takes up
// to 16 (one 16-wide matrix tile, the keys split over its waves), the tile
// kernel up to 128 (32 per wave, the keys shared by the waves).
constexpr int kFewRows = 16;
constexpr int kTileQRows = 128;
// A partial-result unit: 16 rows of one head group.
constexpr int kUnitRows = 16;
// Workers that the work is cut for.  The few-row kernel's keys are laid end to end
// and cut into one slice per wave.  A tile's keys are cut only where it has more
// than its share of them for three quarters of the CUs: every part costs a start,
// partial results and the join.  Measured with 192, 256 and 512 places: 4 prompts
// of 512 tokens 32, 32, 46 us; one of 1000, 34, 36, 40; one of 4096 with 16 key
// heads 113, 113, 135; 4 groups of 32 requests 117, 128, 127; one group of 64
// requests 35, 34, 42.
constexpr int kFewSlots = 1024;
// Where a key is at most 128 bytes and nothing else is in the launch: twice as
// many, since a wave then has less under way.
constexpr int kFewSlotsSmall = 2048;
constexpr int kSmallKeyBytes = 128;
constexpr int kTileSlots = 192;
// Shortest slice and shortest part of a tile, in keys: one step; four tiles.
constexpr int kFewMinKeys = 32;
constexpr int kTileMinKeys = 256;
// Workgroups that the tile items of a call are spread over at most.
constexpr int kMaxTileBlocks = 4096;
// Granularity of slices and of parts: a step of either kernel.
constexpr int kCutKeys = 32;
constexpr int kPartKeys = 64;

constexpr int kAttnTileInts = 12;  // see AttnTile
constexpr int kAttnItemInts = 8;   // see AttnItem
constexpr int kAttnSlotInts = 12;  // see AttnSlot
constexpr int kAttnJoinInts = 12;  // a token to join: token, 3 unused, its own parts, its group's parts
constexpr int kAttnInfoInts = 16;

LORA_HD int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Query heads of a work item: the query heads of one key head, cut into equal
// parts of at most 16 so that one token's rows always fit a few-row item.
LORA_HD int heads_per_item(int per_kv) {
  for (int parts = 1; parts < per_kv; ++parts)
    if (per_kv % parts == 0 && per_kv / parts <= kFewRows) return per_kv / parts;
  return 1;
}

LORA_HD int64_t round_to(int64_t keys, int step) { return (keys + step - 1) & ~(int64_t)(step - 1); }

// Length of a slice (few-row kernel) or most keys of a part (tile kernel): an
// equal share of all keys for each of the `slots` workers, heads of which
// work on the same keys, and at least `least`, in whole steps.  (Few workers a head
// and long sequences: beyond 32 bits.)
LORA_HD int slots_per_head(int heads, int slots) { return slots / heads > 0 ? slots / heads : 1; }
LORA_HD int64_t share_of(int64_t total, int heads, int slots, int least, int step) {
  const int64_t c = ceil_div64(total, slots_per_head(heads, slots));
  return round_to(c < least ? least : c, step);
}

// Keys that a few-row tile occupies on the line that is cut into slices (a sequence
// has at most 2^31 - 2^16).
LORA_HD int line_keys(int keys) { return keys > 0 ? (int)round_to(keys, kCutKeys) : kCutKeys; }

// Parts of a tile-kernel tile: equal parts of at most `share` keys.
LORA_HD int part_keys(int keys, int64_t share) {
  if (keys <= share) return keys > 0 ? keys : 1;
  return (int)round_to(ceil_div64(keys, ceil_div64(keys, share)), kPartKeys);
}

// Capacities of the work lists, from sizes the host knows.
struct AttnCaps {
  int64_t tiles;      // tiles of both kernels, groups' included
  int64_t few_items;  // pieces of few-row tiles
  int64_t slots;      // slices of the few-row kernel
  int64_t tile_items;
  int64_t units;      // partial-result units
};

// heads: head groups (items per tile and key range); group: query heads of an
// item; tile_rows: rows of the larger tile (16 where only the few-row kernel
// runs).  A sequence of q tokens makes ceil(q / tokens) tiles, a single one
// where they are few rows.  Every cut between two slices adds one piece; parts
// of at most share_of keys number at most twice the slots in all tiles that are
// cut.  With groups every tile may need partial results.
LORA_HD AttnCaps attn_caps(int64_t tokens, int64_t seqs, int64_t groups, int heads, int group, int tile_rows, int few_slots) {
  const int64_t per = tile_rows / group;
  const int64_t own = seqs + tokens / per, shared = groups ? groups + tokens / per : 0;
  const int64_t few = slots_per_head(heads, few_slots) + 1, big = slots_per_head(heads, kTileSlots) + 1;
  const bool wide = tile_rows > kFewRows;
  AttnCaps c;
  c.tiles = own + shared;
  c.slots = few;
  c.few_items = (wide ? seqs + groups : c.tiles) + few;
  c.tile_items = wide ? c.tiles + big : 0;
  const int64_t ups = wide ? kTileQRows / kUnitRows : 0;
  if (groups)
    c.units = 2 * (ceil_div64(tokens * group, kUnitRows) + c.tiles) + few + ups * big;
  else
    c.units = 2 * (few + ups * big);
  return c;
}

// What follows from the heads, the cache's type and the longest sequence.
struct AttnShape {
  int group, heads;  // query heads of an item, items per tile and key range
  int tile_rows, few_slots;
  bool few_only;     // sequences of at most 16 rows and no groups: nothing for the tile kernel
};
LORA_HD AttnShape attn_shape(int q_heads, int kv_heads, int64_t key_bytes, bool f32, int groups, int max_q_len) {
  AttnShape s;
  s.group = heads_per_item(q_heads / kv_heads);
  s.heads = q_heads / s.group;
  s.tile_rows = f32 ? kFewRows : kTileQRows;
  s.few_only = f32 || (!groups && (int64_t)max_q_len * s.group <= kFewRows);
  s.few_slots = s.few_only && key_bytes <= kSmallKeyBytes ? kFewSlotsSmall : kFewSlots;
  return s;
}

// One tile: rows [tok0 * group, (tok0 + ntok) * group) of every head group.
struct AttnTile {
  int32_t tok0, ntok, seq;    // seq: row of the page table
  int32_t key0, key1;         // keys any of its tokens sees
  int32_t full0, full1;       // keys all of its tokens see (full0 >= full1: none)
  int32_t few;                // 1: few-row kernel
  int32_t shared;             // 1: a group's shared keys; 2: the own keys of a member of a group
  int32_t part;               // which of its sequence's (group's) tiles
  int64_t at;                 // few: start on the line of keys, in cuts
};

// One item: a tile's rows on a part of its keys (a piece of a slice, or a part of
// a tile-kernel tile).  unit < 0: the result is final
// and goes to the output; else to partial-result units unit, unit + 1, ...
struct AttnItem {
  int32_t tok0, ntok, seq, key0, key1, full0, full1, unit;
};
// One slice of the few-row kernel: its items [first, end), and the first of them.
struct AttnSlot {
  int32_t first, end, pad[2];
  AttnItem item;
};
static_assert(sizeof(AttnSlot) == 4 * kAttnSlotInts, "record size");
static_assert(sizeof(AttnTile) == 4 * kAttnTileInts && sizeof(AttnItem) == 4 * kAttnItemInts, "record sizes");

// x / d for 0 <= x < 2^31 and 1 <= d <= 65536.  With m = 2^32 / d rounded up,
// x * m / 2^32 exceeds x / d by less than x / 2^32 < 1/2, so its integer part is
// right or one too large, which one comparison mends.
LORA_HD uint32_t div_magic(uint32_t d) { return (uint32_t)(((1ull << 32) + d - 1) / d); }
LORA_HD uint32_t div_by(uint32_t x, uint32_t d, uint32_t m) {
  if (d == 1) return x;
  uint32_t q = (uint32_t)(((uint64_t)x * m) >> 32);
  return q - (q * d > x ? 1u : 0u);
}

// A divisor that the host knows, with its magic number.
struct Divisor {
  uint32_t d, m;
  LORA_HD uint32_t quotient(uint32_t x) const { return div_by(x, d, m); }
};
LORA_HD Divisor divisor(uint32_t d) { return Divisor{d, div_magic(d)}; }

// What the attention kernels know of the cache.
struct CacheView {
  const char *k, *v;
  int64_t page_bytes, head_bytes, pos_bytes;
  uint32_t num_pages;
  Divisor page_size;
  const int32_t *table;
  int64_t table_stride;
  const float *k_scale, *v_scale;
};

// Byte offset of position `key` of a sequence inside a head's plane, given the
// page id its table holds; ids outside [0, num_pages) give -1.
LORA_HD int64_t key_offset(const CacheView &c, uint32_t key, int32_t page) {
  if ((uint32_t)page >= c.num_pages) return -1;
  const uint32_t at = key - c.page_size.quotient(key) * c.page_size.d;
  return (int64_t)page * c.page_bytes + (int64_t)at * c.pos_bytes;
}

}  // namespace lora
