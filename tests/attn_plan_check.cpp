// attn_plan_check.cpp -- the attention plan's arithmetic on the CPU, built with
// sanitizers by tests/test_attention_cpu.py from the header the kernels use:
// division by magic numbers, key addresses (pages out of range, pages that end
// anywhere) against the cache's size, and the work lists of random batches
// against the capacities that the workspaces are sized by.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../segmented_gather_rank_amd/csrc/lora_attn.h"

using namespace lora;

static uint64_t state = 88172645463325252ull;
static uint32_t rnd() {
  state ^= state << 13, state ^= state >> 7, state ^= state << 17;
  return (uint32_t)(state >> 16);
}
static int64_t upto(int64_t n) { return n > 0 ? (int64_t)(rnd() % (uint64_t)(n + 1)) : 0; }
#define CHECK(c)                                                    \
  do {                                                              \
    if (!(c)) {                                                     \
      std::fprintf(stderr, "line %d: %s\n", __LINE__, #c);          \
      std::exit(1);                                                 \
    }                                                               \
  } while (0)

static void division() {
  for (uint32_t d = 1; d <= 65536; d = d < 300 ? d + 1 : d + 1 + rnd() % 97) {
    const uint32_t m = div_magic(d);
    const uint32_t top = 0x7fffffffu;
    for (uint32_t x : {0u, 1u, d - 1, d, d + 1, top, top - 1, top / d * d, top / d * d - 1}) CHECK(x > top || div_by(x, d, m) == x / d);
    for (int i = 0; i < 200; ++i) {
      const uint32_t x = rnd() & top;
      CHECK(div_by(x, d, m) == x / d);
    }
  }
}

// Every address lies inside the cache, whatever the page table holds.
static void addresses() {
  for (int trial = 0; trial < 3000; ++trial) {
    const int page = 1 + (int)upto(trial % 3 ? 70 : 5), heads = 1 + (int)upto(4), dim = 16 * (1 + (int)upto(4));
    const int64_t pages = 1 + upto(9);
    CacheView c = {};
    const bool tokens = rnd() & 1;
    c.pos_bytes = (tokens ? heads : 1) * dim;
    c.head_bytes = (tokens ? 1 : page) * dim;
    c.page_bytes = (int64_t)page * heads * dim;
    c.num_pages = (uint32_t)pages;
    c.page_size = divisor((uint32_t)page);
    const int64_t size = pages * c.page_bytes;
    std::vector<int32_t> table(8);
    for (auto &p : table) p = rnd() % 4 ? (int32_t)upto(pages - 1) : (int32_t)rnd();
    for (uint32_t key = 0; key < 8u * page; ++key) {
      const int32_t id = table[c.page_size.quotient(key)];
      const int64_t off = key_offset(c, key, id);
      if (id < 0 || id >= pages) {
        CHECK(off == -1);
        continue;
      }
      CHECK(off >= 0);
      for (int h = 0; h < heads; ++h) CHECK(off + h * c.head_bytes + dim <= size);
      CHECK(off == id * c.page_bytes + (int64_t)(key % page) * c.pos_bytes);
    }
  }
}

static void groups_of_heads() {
  for (int per = 1; per <= 1024; ++per) {
    const int g = heads_per_item(per);
    CHECK(g >= 1 && g <= kFewRows && per % g == 0);
  }
}

// The plan kernel's counting over a batch in order: never more items, tiles or
// units than attn_caps allows.
static void capacities() {
  for (int trial = 0; trial < 20000; ++trial) {
    const int group = 1 + (int)upto(15), heads = 1 + (int)upto(trial % 5 ? 40 : 1000), rows = rnd() & 1 ? kTileQRows : kFewRows;
    const int seqs = (int)upto(trial % 7 ? 40 : 600);
    std::vector<int64_t> q(seqs), kv(seqs);
    int64_t tokens = 0;
    for (int n = 0; n < seqs; ++n) {
      q[n] = rnd() % 3 ? upto(3) : upto(rnd() % 4 ? 60 : 700);
      kv[n] = q[n] + (rnd() % 3 ? upto(200) : upto(100000));
      tokens += q[n];
    }
    const int groups = seqs && rnd() % 2 ? 1 + (int)upto(seqs < 5 ? 0 : 3) : 0;
    const int few_slots = rnd() & 1 ? kFewSlots : kFewSlotsSmall;
    const AttnCaps cap = attn_caps(tokens, seqs, groups, heads, group, rows, few_slots);
    struct Tile { int64_t ntok, len; bool few, parts; };
    std::vector<Tile> tiles;
    const int few = kFewRows / group, per = rows / group;
    auto cut = [&](int64_t len, int64_t keys, bool parts) {
      const bool is_few = len <= few || rows == kFewRows;
      const int64_t step = is_few ? few : per;
      for (int64_t t = 0; t < len; t += step) tiles.push_back({len - t < step ? len - t : step, upto(3) ? keys : upto(keys), is_few, parts});
    };
    for (int n = 0; n < seqs; ++n) cut(q[n], kv[n], groups && rnd() % 8);
    for (int g = 0; g < groups; ++g) {
      int64_t len = 0;
      for (int n = seqs * g / groups; n < seqs * (g + 1) / groups; ++n) len += q[n];
      cut(len, upto(50000), true);
    }
    // the few-row tiles' keys on one line, cut into slices; the others in parts
    int64_t line = 0, total = 0;
    for (auto &t : tiles) (t.few ? line : total) += t.few ? line_keys((int)t.len) : t.len;
    const int slice = share_of(line, heads, few_slots, kFewMinKeys, kCutKeys), share = share_of(total, heads, kTileSlots, kTileMinKeys, kPartKeys);
    CHECK(slice % kCutKeys == 0 && (int64_t)slice * (cap.slots - 1) >= line);
    int64_t items[2] = {0, 0}, units = 0, at = 0;
    for (auto &t : tiles) {
      CHECK(t.ntok * group <= (t.few ? kFewRows : kTileQRows));
      int64_t parts;
      if (t.few) {
        const int64_t last = at + line_keys((int)t.len) - 1;
        parts = last / slice - at / slice + 1;
        CHECK(last / slice < cap.slots - 1);
        at = last + 1;
      } else {
        const int per = part_keys((int)t.len, share);
        CHECK(per >= 1 && per <= share && (per == t.len || per % kPartKeys == 0 || t.len == 0));
        parts = t.len ? ceil_div64(t.len, per) : 1;
      }
      items[!t.few] += parts;
      if (t.parts || parts > 1) units += parts * ceil_div64(t.ntok * group, kUnitRows);
    }
    CHECK((int64_t)tiles.size() <= cap.tiles);
    CHECK(items[0] <= cap.few_items);
    CHECK(items[1] <= cap.tile_items);
    CHECK(units <= cap.units);
  }
}

int main() {
  division();
  addresses();
  groups_of_heads();
  capacities();
  std::puts("all checks passed");
  return 0;
}
