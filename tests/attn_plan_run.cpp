// attn_plan_run.cpp -- the attention plan itself on the CPU, built with sanitizers by
// tests/test_attention_plan_cpu.py: the code that the device's workgroup runs, by a
// team of one thread, on buffers of exactly the workspace's sizes whose first contents
// are garbage.  Every plan is then followed as the attention kernels follow it, and
// every key that a token sees has to be computed once, through the right page table,
// and reach the output by one writer.  argv: kind of batches, how many, and "records" to
// follow the records alone, without asking what they compute.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <set>
#include <string>
#include <vector>

#include "../segmented_gather_rank_amd/csrc/lora_attn_plan.h"

using namespace lora;

static uint64_t state = 88172645463325252ull;
static uint32_t rnd() {
  state ^= state << 13, state ^= state >> 7, state ^= state << 17;
  return (uint32_t)(state >> 16);
}
static int64_t upto(int64_t n) { return n > 0 ? (int64_t)(rnd() % (uint64_t)(n + 1)) : 0; }
static long trial = -1;
#define CHECK(c)                                                          \
  do {                                                                    \
    if (!(c)) {                                                           \
      std::fprintf(stderr, "trial %ld, line %d: %s\n", trial, __LINE__, #c); \
      std::exit(1);                                                       \
    }                                                                     \
  } while (0)

struct Solo {
  TeamShared common;
  int id() const { return 0; }
  int size() const { return 1; }
  void sync() const {}
  TeamShared &shared() { return common; }
  bool any(bool x) const { return x; }
  int read(const int *p) const { return *p; }
  template <typename T, typename V>
  void add(T *p, V v) const { *p += v; }
  template <typename T>
  T before(T v, T &total) const {
    total = v;
    return 0;
  }
  template <typename T>
  T most_before(T v, T &total) const {
    total = v;
    return 0;
  }
};

struct Batch {
  int q_heads = 8, kv_heads = 2, dim = 64, esize = 2, page = 16, max_q_len = 0, window = 0;
  bool causal = true;
  int64_t tokens = 0, stride = 0;
  std::vector<int32_t> q_start, kv_len, prefix, key_lo, key_hi, group_start, group_len;
  int seqs() const { return (int)kv_len.size(); }
  int groups() const { return (int)group_len.size(); }
};

// ---- the header's rules
struct Model {
  const Batch &b;
  std::vector<char> good_seq, good_group;
  std::vector<int> owner, group;  // of a token: sequence, -1: none, -2: bad ones only; of a sequence
  bool ordered = true;
  explicit Model(const Batch &x) : b(x) {
    const int N = b.seqs();
    int64_t end = 0;
    owner.assign(b.tokens, -1);
    for (int n = 0; n < N; ++n) {
      const int64_t s = b.q_start[n], e = b.q_start[n + 1], kv = b.kv_len[n];
      if (!(0 <= s && s <= e && e <= b.tokens)) ordered = false;
      bool ok = 0 <= s && s <= e && e <= b.tokens && e - s <= b.max_q_len && e - s <= kv && kv <= b.stride * b.page;
      const bool overlaps = ok && e > s && s < end;
      if (ok && e > s) end = std::max(end, e);
      good_seq.push_back(ok && !overlaps);
      for (int64_t t = std::max<int64_t>(s, 0); t < std::min(e, b.tokens); ++t) {
        if (good_seq[n]) owner[t] = n;
        else if (owner[t] == -1) owner[t] = -2;
      }
    }
    group.assign(N, -1);
    int last = 0;
    for (int g = 0; g < b.groups(); ++g) {
      const int s = b.group_start[g], e = b.group_start[g + 1], len = b.group_len[g];
      bool ok = ordered && 0 <= s && s <= e && e <= N && len >= 0 && (s == e || (good_seq[s] && len <= b.kv_len[s]));
      if (ok && e > s) {
        if (s < last) ok = false;
        last = std::max(last, e);
      }
      good_group.push_back(ok);
      for (int n = s; ok && len > 0 && n < e; ++n) group[n] = g;
    }
  }
  void visible(int64_t t, int64_t &lo, int64_t &hi, int64_t &p) const {
    lo = hi = p = 0;
    const int n = owner[t];
    if (n < 0) return;
    const int64_t kv = b.kv_len[n];
    p = kv - (b.q_start[n + 1] - b.q_start[n]) + (t - b.q_start[n]);
    hi = b.causal ? p + 1 : kv;
    if (!b.prefix.empty()) hi = std::max<int64_t>(hi, b.prefix[n]);
    if (b.window) lo = std::max<int64_t>(lo, p + 1 - b.window);
    if (!b.key_lo.empty()) lo = std::max<int64_t>(lo, b.key_lo[t]), hi = std::min<int64_t>(hi, b.key_hi[t]);
    hi = std::min(hi, kv);
    if (hi <= lo) lo = hi = 0;
  }
};

struct Piece {
  int64_t key0, key1;
  int table;
};

static void follow(const Batch &b, bool records_only) {
  const AttnShape sh = attn_shape(b.q_heads, b.kv_heads, (int64_t)b.dim * b.esize, b.esize == 4, b.groups(), b.max_q_len);
  const AttnCaps cap = attn_caps(b.tokens, b.seqs(), b.groups(), sh.heads, sh.group, sh.tile_rows, sh.few_slots);
  const int32_t junk = 0x5a5a5a5a;
  auto ints = [&](int64_t n) { return std::vector<int32_t>((size_t)n, junk); };
  auto at = [](std::vector<int32_t> &v) { return v.empty() ? nullptr : v.data(); };
  std::vector<int32_t> limits = ints(4 * b.tokens), info = ints(kAttnInfoInts), tiles = ints(kAttnTileInts * cap.tiles),
                       few = ints(kAttnItemInts * cap.few_items), slots = ints(kAttnSlotInts * cap.slots),
                       big = ints(kAttnItemInts * cap.tile_items), join = ints(8 * b.tokens),
                       join_list = ints(kAttnJoinInts * b.tokens), seq_end = ints(b.seqs()), group_end = ints(b.groups());
  AttnPlanArgs a = {};
  auto in = [](const std::vector<int32_t> &v) { return v.empty() ? nullptr : v.data(); };
  a.q_start = in(b.q_start), a.kv_len = in(b.kv_len), a.prefix_len = in(b.prefix), a.key_lo = in(b.key_lo);
  a.key_hi = in(b.key_hi), a.group_start = in(b.group_start), a.group_len = in(b.group_len);
  a.tokens = b.tokens, a.table_stride = b.stride, a.seqs = b.seqs(), a.groups = b.groups(), a.max_q_len = b.max_q_len;
  a.page_size = b.page, a.causal = b.causal, a.window = b.window;
  a.heads = sh.heads, a.group = sh.group, a.tile_rows = sh.tile_rows, a.few_slots = sh.few_slots;
  a.max_slots = (int)cap.slots;
  a.limits = at(limits), a.info = info.data(), a.tiles = at(tiles), a.few_items = at(few), a.slots = at(slots);
  a.tile_items = at(big), a.join = at(join), a.join_list = at(join_list);
  a.seq_end = at(seq_end), a.group_end = at(group_end);
  for (int64_t t = 0; t < b.tokens; ++t) reinterpret_cast<AttnLimit *>(a.limits)[t] = limit_of(a, t);
  Solo team;
  attn_plan(a, team);

  const Model m(b);
  if (!records_only) {
    CHECK(info[2] == std::count(m.good_seq.begin(), m.good_seq.end(), 0));
    CHECK(info[3] == std::count(m.good_group.begin(), m.good_group.end(), 0));
  }

  // ---- the kernels' items: slices of the few-row work, then the tiles' (if launched)
  std::vector<AttnItem> items;
  const AttnSlot *slot = reinterpret_cast<AttnSlot *>(a.slots);
  const AttnItem *few_items = reinterpret_cast<AttnItem *>(a.few_items), *tile_items = reinterpret_cast<AttnItem *>(a.tile_items);
  std::set<int> taken;
  for (int k = 0; k < cap.slots - 1; ++k) {
    CHECK(slot[k].first >= 0 && slot[k].end <= info[8] && info[8] <= cap.few_items);
    for (int i = slot[k].first; i < slot[k].end; ++i) {
      CHECK(i != slot[k].first || !std::memcmp(&slot[k].item, &few_items[i], sizeof(AttnItem)));
      CHECK(taken.insert(i).second);
      items.push_back(few_items[i]);
    }
  }
  CHECK((int)taken.size() == info[8]);
  const int64_t slice = info[6];
  for (const AttnItem &it : items) CHECK(it.ntok * sh.group <= kFewRows && (it.key1 - it.key0 <= slice || slice == 0x7fffffff));
  CHECK(info[1] <= cap.tile_items);
  if (!sh.few_only)
    for (int i = 0; i < info[1]; ++i) items.push_back(tile_items[i]);

  const AttnLimit *lim = reinterpret_cast<AttnLimit *>(a.limits);
  std::vector<std::vector<Piece>> seen(b.tokens);
  std::vector<int> writers(b.tokens, 0);
  std::map<std::pair<int64_t, int>, std::pair<int, Piece>> rows;  // (unit, row of it) -> token, piece
  for (const AttnItem &it : items) {
    CHECK(it.tok0 >= 0 && it.ntok >= 0 && it.tok0 + it.ntok <= b.tokens && it.ntok * sh.group <= sh.tile_rows);
    CHECK(it.seq >= 0 && it.seq < b.seqs() && it.key0 >= 0 && it.key0 <= it.key1 && it.key1 <= b.stride * b.page);
    for (int i = 0; i < it.ntok; ++i) {
      const int t = it.tok0 + i;
      // the keys that the kernels take for seen by all
      const int64_t f0 = std::max(it.key0, it.full0), f1 = std::min(it.key1, it.full1);
      CHECK(f0 >= f1 || (lim[t].lo <= f0 && f1 <= lim[t].hi));
      const Piece p{it.key0, it.key1, it.seq};
      if (it.unit < 0) {
        ++writers[t];
        seen[t].push_back(p);
        continue;
      }
      for (int r = i * sh.group; r < (i + 1) * sh.group; ++r) {
        const int64_t unit = it.unit + r / kUnitRows;
        CHECK(unit < cap.units);
        const bool first = rows.emplace(std::make_pair(unit, r % kUnitRows), std::make_pair(t, p)).second;
        CHECK(first);
      }
    }
  }
  const AttnJoin *list = reinterpret_cast<AttnJoin *>(a.join_list);
  CHECK(info[4] >= 0 && info[4] <= b.tokens);
  for (int j = 0; j < info[4]; ++j) {
    const AttnJoin &e = list[j];
    CHECK(e.token >= 0 && e.token < b.tokens);
    ++writers[e.token];
    for (const AttnParts *rec : {&e.shared, &e.own}) {
      CHECK(rec->parts >= 0 && rec->parts <= cap.units);
      for (int p = 0; p < rec->parts; ++p)
        for (int r = rec->row * sh.group; r < (rec->row + 1) * sh.group; ++r) {
          const auto it = rows.find({rec->unit + (int64_t)p * rec->ups + r / kUnitRows, r % kUnitRows});
          CHECK(it != rows.end() && it->second.first == e.token);
          if (r % sh.group == 0) seen[e.token].push_back(it->second.second);
        }
    }
  }

  if (records_only) return;

  // ---- every token: one writer, every key it sees once
  for (int64_t t = 0; t < b.tokens; ++t) {
    int64_t lo, hi, p;
    m.visible(t, lo, hi, p);
    const int n = m.owner[t];
    CHECK(writers[t] == (n != -1));
    CHECK((n >= 0) == (lim[t].seq >= 0 && m.good_seq[lim[t].seq]));
    if (n == -1) {
      CHECK(lim[t].seq == -1 && lim[t].hi == 0);
      continue;
    }
    CHECK(lim[t].lo == lo && lim[t].hi == hi);
    if (n >= 0) CHECK(lim[t].seq == n && lim[t].pos == p);
    std::vector<Piece> got;
    for (Piece q : seen[t]) {
      q.key0 = std::max(q.key0, lo), q.key1 = std::min(q.key1, hi);
      if (q.key0 < q.key1) got.push_back(q);
    }
    std::sort(got.begin(), got.end(), [](const Piece &x, const Piece &y) { return x.key0 < y.key0; });
    int64_t at_key = lo;
    for (const Piece &q : got) {
      CHECK(q.key0 == at_key);
      at_key = q.key1;
      const int g = m.group[n];
      const int64_t len = g < 0 ? 0 : b.group_len[g];
      // shared keys through the first member's table, the others through its own
      CHECK(q.key1 <= len ? q.table == b.group_start[g] : (q.table == n && q.key0 >= len));
    }
    CHECK(at_key == hi);
  }
}

static Batch ordered(bool masks, bool groups) {
  Batch b;
  const int heads[][2] = {{8, 2}, {32, 8}, {1, 1}, {7, 1}, {6, 6}, {34, 2}, {16, 16}, {64, 64}};
  const auto &h = heads[rnd() % 8];
  b.q_heads = h[0], b.kv_heads = h[1];
  b.esize = 1 << (rnd() % 3), b.dim = rnd() % 2 ? 64 : 128, b.page = rnd() % 3 ? 16 : 1 + (int)upto(40);
  const int N = (int)upto(rnd() % 5 ? 12 : 90);
  const bool decode = rnd() % 3 == 0;
  b.q_start.push_back(0);
  int64_t most = 0, most_q = 0;
  for (int n = 0; n < N; ++n) {
    const int64_t q = decode ? rnd() % 9 != 0 : (rnd() % 3 ? upto(4) : upto(rnd() % 4 ? 60 : 300));
    const int64_t kv = q + (rnd() % 3 ? upto(200) : upto(rnd() % 9 ? 3000 : 60000));
    b.q_start.push_back((int32_t)(b.q_start.back() + q));
    b.kv_len.push_back((int32_t)kv);
    most = std::max(most, kv), most_q = std::max(most_q, q);
  }
  b.tokens = b.q_start.back() + (rnd() % 4 ? 0 : upto(3));  // some tokens outside every sequence
  b.stride = (most + b.page - 1) / b.page;
  b.max_q_len = (int)(rnd() % 2 ? most_q : std::max<int64_t>(b.tokens, most_q));
  if (masks) {
    b.causal = rnd() % 3;
    if (rnd() % 2) b.window = 1 + (int)upto(400);
    if (rnd() % 3 == 0)
      for (int n = 0; n < N; ++n) b.prefix.push_back((int32_t)upto(2 * b.kv_len[n]));
    if (rnd() % 3 == 0)
      for (int64_t t = 0; t < b.tokens; ++t) {
        b.key_lo.push_back((int32_t)upto(most) - 10);
        b.key_hi.push_back(b.key_lo.back() + (int32_t)upto(300) - 20);
      }
  }
  if (groups && N) {
    int at = (int)upto(2);
    b.group_start.push_back(std::min(at, N));
    while (b.group_start.back() < N && b.groups() < 8) {
      const int s = b.group_start.back(), e = std::min<int>(N, s + (int)upto(6));
      b.group_start.push_back(e);
      b.group_len.push_back(s < e ? (int32_t)upto(b.kv_len[s]) : (int32_t)upto(50));
    }
    if (b.group_len.empty()) b.group_start.clear();
  }
  return b;
}

static void spoil_lengths(Batch &b) {  // bad by their lengths, bounds in order
  for (int n = 0; n < b.seqs(); ++n)
    if (rnd() % 5 == 0) {
      const int64_t q = b.q_start[n + 1] - b.q_start[n];
      switch (rnd() % 3) {
        case 0: b.kv_len[n] = (int32_t)(b.stride * b.page + 1 + upto(1000)); break;
        case 1: b.kv_len[n] = (int32_t)(q - 1 - upto(3)); break;
        default: b.kv_len[n] = (int32_t)0x80000000 + (int32_t)upto(5);
      }
    }
  if (rnd() % 2) b.max_q_len = (int)upto(b.max_q_len);
}

static void lengthen(Batch &b) {  // as many keys as the table may hold
  if (rnd() % 4 == 0) b.page = 1;
  b.stride = (rnd() % 2 ? 0x7fff0000 : (1 << 25) - (int)upto(2)) / b.page;
  const int64_t most = b.stride * b.page;
  for (int n = 0; n < b.seqs(); ++n)
    if (rnd() % 3) b.kv_len[n] = (int32_t)(rnd() % 2 ? most - upto(70) : most / (1 + upto(40)) - upto(5));
  for (auto &x : b.prefix) x = (int32_t)upto(0x7fffffff);
  for (size_t t = 0; t < b.key_lo.size(); ++t) b.key_lo[t] = (int32_t)upto(most), b.key_hi[t] = (int32_t)upto(0x7fffffff);
  for (int g = 0; g < b.groups(); ++g)
    if (b.group_start[g] < b.group_start[g + 1] && rnd() % 2) b.group_len[g] = (int32_t)upto(b.kv_len[b.group_start[g]]);
}

static void spoil_bounds(Batch &b) {
  const int N = b.seqs();
  if (!N) return;
  for (int k = 1 + (int)upto(2); k > 0; --k) {
    int32_t &x = b.q_start[upto(N)];
    switch (rnd() % 6) {
      case 0: x = 900 + (int32_t)b.tokens; break;
      case 1: x = -1 - (int32_t)upto(9); break;
      case 2: x = (int32_t)0x80000000; break;
      case 3: x = 0x7fffffff; break;
      default: x = (int32_t)upto(b.tokens);
    }
  }
  if (rnd() % 8 == 0)
    for (auto &x : b.q_start) x = (int32_t)(rnd() % 3 ? upto(b.tokens) : rnd());
}

static void spoil_groups(Batch &b) {
  if (!b.groups()) return;
  for (int k = 1 + (int)upto(2); k > 0; --k) {
    int32_t &x = b.group_start[upto(b.groups())];
    switch (rnd() % 5) {
      case 0: x = 100 + b.seqs(); break;
      case 1: x = -1 - (int32_t)upto(9); break;
      case 2: x = (int32_t)rnd(); break;
      default: x = (int32_t)upto(b.seqs());
    }
  }
  if (rnd() % 3 == 0) b.group_len[upto(b.groups() - 1)] = rnd() % 2 ? -1 - (int32_t)upto(5) : 1000000;
}

int main(int argc, char **argv) {
  const std::string kind = argc > 1 ? argv[1] : "ordered";
  const long trials = argc > 2 ? std::atol(argv[2]) : 1000;
  for (trial = 0; trial < trials; ++trial) {
    Batch b = ordered(rnd() % 2, kind == "groups" || kind == "bad_groups" || kind == "everything" || rnd() % 2);
    if (kind == "long") lengthen(b);
    if (kind == "bad_ends" && b.seqs()) {  // the last sequence leaves the batch
      b.q_start.back() = (int32_t)b.tokens + 900;
    }
    if (kind == "bad_lengths" || kind == "everything") spoil_lengths(b);
    if (kind == "bad_bounds" || kind == "everything") spoil_bounds(b);
    if (kind == "bad_groups" || kind == "everything") spoil_groups(b);
    follow(b, argc > 3 && !std::strcmp(argv[3], "records"));
  }
  std::puts("all checks passed");
  return 0;
}
