// lora_attn_plan.h -- the attention metadata's algorithm: which keys a token sees,
// and the work lists.  Internal to the library.  Plain integer code over a Team of
// threads (a workgroup on the device, one thread in the CPU tests, which run it on
// buffers of exactly the workspace's sizes):
//   id(), size()       this thread and how many there are; loops go in steps of size()
//   sync()             what any thread wrote before, every thread reads after
//   before(v, total)   sum of v over the threads before this one, and over all
//   most_before(v, total)   likewise their maximum, of values from 0 on
//   any(x)             whether x holds for any thread
//   shared()           a TeamShared that the threads have in common
//   add(p, v)          atomic add, to it or to memory
//   read(p)            what such adds to memory came to, after sync()
#pragma once

#include "lora_attn.h"

namespace lora {

struct AttnPlanArgs {
  const int32_t *q_start, *kv_len, *prefix_len, *key_lo, *key_hi, *group_start, *group_len;
  int64_t tokens, table_stride;
  int32_t seqs, groups, max_q_len, page_size, causal, window;
  int32_t heads, group, tile_rows, few_slots;
  int32_t max_slots;
  int32_t *limits, *info, *tiles, *few_items, *slots, *tile_items, *join, *join_list;
  int32_t *seq_end, *group_end;  // see seq_ok, group_ok
};

// What a token sees: keys [lo, hi), its position, its sequence.
struct alignas(16) AttnLimit {
  int32_t lo, hi, pos, seq;
};
// Where a token's partial results lie: `parts` runs of `ups` units from `unit` on, the
// token being the row-th of its tile.
struct alignas(16) AttnParts {
  int32_t unit, parts, ups, row;
};
struct alignas(16) AttnJoin {
  int32_t token, pad[3];
  AttnParts own, shared;
};
static_assert(sizeof(AttnJoin) == 4 * kAttnJoinInts, "record size");

struct TeamShared {
  unsigned long long keys;
  int bad_seqs, bad_groups;
};

// Whether bounds are out of order or leave their range anywhere, the same in all threads.
struct AttnOrder {
  bool seqs, groups;
};

LORA_HD int min_i(int a, int b) { return a < b ? a : b; }
LORA_HD int max_i(int a, int b) { return a > b ? a : b; }
LORA_HD int64_t min_l(int64_t a, int64_t b) { return a < b ? a : b; }
LORA_HD int64_t max_l(int64_t a, int64_t b) { return a > b ? a : b; }

// Whether the query tokens of sequence n are an interval of the batch.
LORA_HD bool seq_ordered(const AttnPlanArgs &a, int n) {
  const int64_t q0 = a.q_start[n], q1 = a.q_start[n + 1];
  return q0 >= 0 && q1 >= q0 && q1 <= a.tokens;
}

// Whether sequence n would be usable if it were the only one (see lora_attn_batch).
LORA_HD bool seq_alone_ok(const AttnPlanArgs &a, int n) {
  const int64_t q0 = a.q_start[n], q1 = a.q_start[n + 1], kv = a.kv_len[n];
  return seq_ordered(a, n) && q1 - q0 <= a.max_q_len && kv >= q1 - q0 && kv <= a.table_stride * a.page_size;
}

// Whether sequence n is usable.  Where bounds are out of order, seq_end[n] is the
// furthest end of a sequence up to n, and one that starts before it shares tokens with
// an earlier one: it is bad, so that no token has two sequences.
LORA_HD bool seq_ok(const AttnPlanArgs &a, AttnOrder broken, int n) {
  if (!seq_alone_ok(a, n)) return false;
  return !broken.seqs || n == 0 || a.q_start[n] == a.q_start[n + 1] || a.q_start[n] >= a.seq_end[n - 1];
}

LORA_HD bool group_ordered(const AttnPlanArgs &a, int g) {
  const int s0 = a.group_start[g], s1 = a.group_start[g + 1];
  return s0 >= 0 && s1 >= s0 && s1 <= a.seqs;
}

// Whether group g would be served if it were the only one.  Its tokens are those
// between its first sequence's bound and its last one's, which holds its members'
// only if all bounds ascend.
LORA_HD bool group_alone_ok(const AttnPlanArgs &a, AttnOrder broken, int g) {
  if (broken.seqs || !group_ordered(a, g) || a.group_len[g] < 0) return false;
  const int s0 = a.group_start[g];
  return s0 == a.group_start[g + 1] || (seq_alone_ok(a, s0) && a.group_len[g] <= a.kv_len[s0]);
}

// Whether group g is served.  One rule for its members and for its tiles, since a
// member's join reads what the group's tiles leave.  Where starts are out of order
// (beside a bad group), group_end[g] is the furthest end of a group up to g, and a
// group that starts before it shares sequences with an earlier one: it is bad.
LORA_HD bool group_ok(const AttnPlanArgs &a, AttnOrder broken, int g) {
  if (!group_alone_ok(a, broken, g)) return false;
  const int s0 = a.group_start[g];
  return !broken.groups || g == 0 || s0 == a.group_start[g + 1] || s0 >= a.group_end[g - 1];
}

// Group of sequence n, or -1: the last group that starts at or before n, or the first
// whose furthest end lies past n.
LORA_HD int group_of(const AttnPlanArgs &a, AttnOrder broken, int n) {
  int lo = 0, hi = a.groups;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (broken.groups ? a.group_end[mid] <= n : a.group_start[mid] <= n) lo = mid + 1;
    else hi = mid;
  }
  const int g = broken.groups ? lo : lo - 1;
  if (g < 0 || g >= a.groups || n < a.group_start[g] || n >= a.group_start[g + 1] || a.group_len[g] == 0 ||
      !group_ok(a, broken, g))
    return -1;
  return g;
}

// What token t of the usable sequence n sees.
LORA_HD AttnLimit limit_in(const AttnPlanArgs &a, int n, int64_t t) {
  const int kv = a.kv_len[n];
  AttnLimit r{0, 0, (int)(kv - a.q_start[n + 1] + t), n};
  r.hi = a.causal ? r.pos + 1 : kv;
  if (a.prefix_len) r.hi = max_i(r.hi, a.prefix_len[n]);
  if (a.window > 0) r.lo = max_i(0, r.pos + 1 - a.window);
  if (a.key_lo) r.lo = max_i(r.lo, a.key_lo[t]);
  if (a.key_hi) r.hi = min_i(r.hi, a.key_hi[t]);
  r.hi = min_i(r.hi, kv);
  if (r.hi <= r.lo) r.lo = r.hi = 0;
  return r;
}

// What token t sees, for bounds in order.
LORA_HD AttnLimit limit_of(const AttnPlanArgs &a, int64_t t) {
  int lo = 0, hi = a.seqs;  // first sequence whose tokens start after t
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.q_start[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  const int n = lo - 1;
  if (n < 0 || t >= a.q_start[n + 1]) return AttnLimit{0, 0, 0, -1};
  return seq_alone_ok(a, n) ? limit_in(a, n, t) : AttnLimit{0, 0, 0, n};
}

// Furthest ends up to each of `count` intervals, end(i) being interval i's (0: none).
template <typename Team, typename F>
LORA_HD void furthest_ends(Team &team, int count, int32_t *out, F &&end) {
  int far = 0;
  for (int i0 = 0; i0 < count; i0 += team.size()) {
    const int i = i0 + team.id(), mine = i < count ? end(i) : 0;
    int most;
    const int before = team.most_before(mine, most);
    if (i < count) out[i] = max_i(far, max_i(before, mine));
    far = max_i(far, most);
  }
  team.sync();
}

// Bounds out of order: every token's sequence again, over the furthest ends, which
// ascend (the first that lies past a token is the one sequence that may hold it).  A
// token that only bad sequences hold, by the number of those that begin at or before
// it less that of those that end, gets -2.
template <typename Team>
LORA_HD void limits_out_of_order(const AttnPlanArgs &a, AttnOrder broken, Team &team) {
  AttnLimit *limits = reinterpret_cast<AttnLimit *>(a.limits);
  furthest_ends(team, a.seqs, a.seq_end,
                [&](int n) { return seq_alone_ok(a, n) && a.q_start[n] < a.q_start[n + 1] ? a.q_start[n + 1] : 0; });
  for (int64_t t = team.id(); t < a.tokens; t += team.size()) limits[t] = AttnLimit{0, 0, 0, -1};
  team.sync();
  for (int n = team.id(); n < a.seqs; n += team.size()) {
    const int64_t q0 = max_l(a.q_start[n], 0), q1 = min_l(a.q_start[n + 1], a.tokens);
    if (q0 >= q1 || seq_ok(a, broken, n)) continue;
    team.add(&limits[q0].pos, 1);
    if (q1 < a.tokens) team.add(&limits[q1].pos, -1);
  }
  team.sync();
  int bad = 0;
  for (int64_t t0 = 0; t0 < a.tokens; t0 += team.size()) {
    const int64_t t = t0 + team.id();
    const int step = t < a.tokens ? team.read(&limits[t].pos) : 0;
    int total;
    const int before = bad + team.before(step, total);
    bad += total;
    if (t >= a.tokens) continue;
    int lo = 0, hi = a.seqs;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (a.seq_end[mid] <= t) lo = mid + 1;
      else hi = mid;
    }
    if (lo < a.seqs && a.q_start[lo] <= t && t < a.q_start[lo + 1] && seq_ok(a, broken, lo)) limits[t] = limit_in(a, lo, t);
    else limits[t] = AttnLimit{0, 0, 0, before + step > 0 ? -2 : -1};
  }
  team.sync();
}

// The work lists.  Every token is in one sequence's tiles and in those of at most one
// group, so the lists fit the capacities of attn_caps whatever the arrays hold.
template <typename Team>
LORA_HD void attn_plan(const AttnPlanArgs &a, Team &team) {
  TeamShared &common = team.shared();
  const int tid = team.id(), threads = team.size();
  const AttnLimit *limits = reinterpret_cast<const AttnLimit *>(a.limits);
  AttnTile *tile_list = reinterpret_cast<AttnTile *>(a.tiles);
  AttnParts *rec_list = reinterpret_cast<AttnParts *>(a.join);
  AttnJoin *join_list = reinterpret_cast<AttnJoin *>(a.join_list);
  if (tid == 0) common = TeamShared{0, 0, 0};
  team.sync();

  // ---- tiles per sequence, then per group: which one, and which of its tiles
  const int few_tokens = kFewRows / a.group, tile_tokens = a.tile_rows / a.group;
  int tiles = 0;
  auto list_tiles = [&](int n, int len) {  // of this thread's sequence or group n
    const int count = len <= few_tokens ? (len > 0) : (len + tile_tokens - 1) / tile_tokens;
    int total;
    const int before = tiles + team.before(count, total);
    for (int i = 0; i < count; ++i) {
      tile_list[before + i].seq = n;
      tile_list[before + i].part = i;
    }
    tiles += total;
  };
  AttnOrder broken{false, false};
  auto list_sequences = [&]() {
    for (int n0 = 0; n0 < a.seqs; n0 += threads) {
      const int n = n0 + tid;
      if (!broken.seqs) {
        // (there are no more groups than sequences)
        const bool here = n < a.seqs && !seq_ordered(a, n), group = n < a.groups && !group_ordered(a, n);
        if (a.groups) broken.groups |= team.any(group);
        if (team.any(here)) return false;
      }
      int len = 0;
      if (n < a.seqs) {
        if (seq_ok(a, broken, n)) len = a.q_start[n + 1] - a.q_start[n];
        else team.add(&common.bad_seqs, 1);
      }
      list_tiles(n, len);
    }
    return true;
  };
  if (!list_sequences()) {  // bounds out of order: once more
    broken.seqs = true;
    limits_out_of_order(a, broken, team);
    if (tid == 0) common.bad_seqs = 0;
    team.sync();
    tiles = 0;
    list_sequences();
  }
  const int own = tiles;
  if (broken.groups)
    furthest_ends(team, a.groups, a.group_end, [&](int g) {
      return group_alone_ok(a, broken, g) && a.group_start[g] < a.group_start[g + 1] ? a.group_start[g + 1] : 0;
    });
  for (int g0 = 0; g0 < a.groups; g0 += threads) {
    const int g = g0 + tid;
    int len = 0;
    if (g < a.groups) {
      if (!group_ok(a, broken, g)) team.add(&common.bad_groups, 1);
      else if (a.group_len[g] > 0 && a.group_start[g] < a.group_start[g + 1])
        len = a.q_start[a.group_start[g + 1]] - a.q_start[a.group_start[g]];
    }
    list_tiles(g, len);
  }
  team.sync();  // the counts; the list is written and read by this team alone

  // ---- the tiles' tokens and keys; few-row tiles take their place on the line
  int64_t line = 0;
  unsigned long long keys = 0;
  for (int i0 = 0; i0 < tiles; i0 += threads) {
    const int i = i0 + tid;
    AttnTile r;
    r.few = 0;
    int width = 0;
    if (i < tiles) {
      const int n = tile_list[i].seq, part = tile_list[i].part;
      int64_t q0, q1;
      int shared_len = 0;
      r.shared = 0;
      r.seq = n;
      if (i < own) {
        q0 = a.q_start[n];
        q1 = a.q_start[n + 1];
        const int g = a.groups ? group_of(a, broken, n) : -1;
        if (g >= 0) {
          r.shared = 2;
          shared_len = a.group_len[g];
        }
      } else {
        r.seq = a.group_start[n];
        q0 = a.q_start[r.seq];
        q1 = a.q_start[a.group_start[n + 1]];
        r.shared = 1;
        shared_len = a.group_len[n];
      }
      const int len = (int)(q1 - q0);
      r.few = len <= few_tokens || a.tile_rows == kFewRows;
      const int per = r.few ? few_tokens : tile_tokens;
      r.tok0 = (int)q0 + part * per;
      r.ntok = max_i(0, min_i(per, len - part * per));
      int lo_min = 0x7fffffff, lo_max = 0, hi_min = 0x7fffffff, hi_max = 0;
      const AttnLimit *lim = limits + r.tok0;
      for (int t0 = 0; t0 < r.ntok; t0 += 8) {
        AttnLimit v[8];  // past the end the last token again
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = lim[min_i(t0 + t, r.ntok - 1)];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          if (v[t].hi > v[t].lo) {
            lo_min = min_i(lo_min, v[t].lo);
            hi_max = max_i(hi_max, v[t].hi);
          }
          lo_max = max_i(lo_max, v[t].lo);
          hi_min = min_i(hi_min, v[t].hi);
        }
      }
      r.key0 = r.shared == 2 ? max_i(lo_min, shared_len) : lo_min;
      r.key1 = r.shared == 1 ? min_i(hi_max, shared_len) : hi_max;
      if (r.key1 <= r.key0) r.key0 = r.key1 = 0;
      r.full0 = lo_max;
      r.full1 = hi_min;
      r.part = part;
      if (r.few) width = line_keys(r.key1 - r.key0) / kCutKeys;
      else keys += (unsigned long long)(r.key1 - r.key0);
    }
    // a sum of 32 bits holds the low 20 of every width; tiles of 2^25 keys, rounded up
    // to whole cuts, and more take a second one
    int total, high_total = 0, high = 0;
    const int low = team.before(width & 0xfffff, total);
    if (a.table_stride * a.page_size >> 24 && team.any(width >> 20)) high = team.before(width >> 20, high_total);
    if (i < tiles) {
      r.at = line + ((int64_t)high << 20) + low;
      tile_list[i] = r;
    }
    line += ((int64_t)high_total << 20) + total;
  }
  if (keys) team.add(&common.keys, keys);
  team.sync();
  const int64_t slice = share_of(line * kCutKeys, a.heads, a.few_slots, kFewMinKeys, kCutKeys);
  const int64_t share = share_of((int64_t)common.keys, a.heads, kTileSlots, kTileMinKeys, kPartKeys);
  const int64_t cuts = slice / kCutKeys;  // of a slice
  const int slots = (int)((line + cuts - 1) / cuts);

  // ---- items, slices, partial-result units, tokens to join
  int few_items = 0, tile_items = 0, units = 0, joins = 0;
  AttnItem *few_list = reinterpret_cast<AttnItem *>(a.few_items), *big_list = reinterpret_cast<AttnItem *>(a.tile_items);
  AttnSlot *slot_list = reinterpret_cast<AttnSlot *>(a.slots);
  for (int i0 = 0; i0 < tiles; i0 += threads) {
    const int i = i0 + tid;
    AttnTile r;
    int parts = 0, per = 1, ups = 0;
    bool join = false;
    if (i < tiles) {
      r = tile_list[i];
      const int n = r.key1 - r.key0;
      if (r.few) {
        const int64_t last = r.at + line_keys(n) / kCutKeys - 1;
        parts = (int)(last / cuts - r.at / cuts) + 1;
      } else {
        per = part_keys(n, share);
        parts = max_i(1, (int)ceil_div64(n, per));
      }
      join = parts > 1 || r.shared;
      ups = (r.ntok * a.group + kUnitRows - 1) / kUnitRows;
    }
    const bool few = i < tiles && r.few;
    int nf, nt, nu, nj;
    const int at_few = few_items + team.before(few ? parts : 0, nf);
    const int at_tile = tile_items + team.before(few ? 0 : parts, nt);
    const int unit = units + team.before(join ? parts * ups : 0, nu);
    const int at_join = joins + team.before(join && r.shared != 1 ? r.ntok : 0, nj);
    if (i < tiles) {
      AttnItem item{r.tok0, r.ntok, r.seq, r.key0, r.key1, r.full0, r.full1, -1};
      for (int s = 0; s < parts; ++s) {
        const int at = (few ? at_few : at_tile) + s;
        if (join) item.unit = unit + s * ups;
        if (few) {
          // the piece of the tile on slice k: the line from `from` on
          const int64_t k = r.at / cuts + s, from = max_l(r.at, k * cuts);
          item.key0 = r.key0 + (int)(from - r.at) * kCutKeys;
          item.key1 = (int)min_l(r.key1, r.key0 + ((k + 1) * cuts - r.at) * kCutKeys);
          few_list[at] = item;
          if (from == k * cuts) {
            slot_list[k].first = at;
            slot_list[k].item = item;
            if (k > 0) slot_list[k - 1].end = at;
          }
        } else {
          item.key0 = r.key0 + s * per;
          item.key1 = min_i(r.key1, item.key0 + per);
          big_list[at] = item;
        }
      }
      if (join) {
        for (int t = 0; t < r.ntok; ++t) {
          AttnParts *rec = rec_list + 2 * (int64_t)(r.tok0 + t);
          rec[r.shared == 1] = AttnParts{unit, parts, ups, t};
          if (r.shared == 0) rec[1] = AttnParts{0, 0, 0, 0};
          if (r.shared != 1) join_list[at_join + t].token = r.tok0 + t;
        }
      }
    }
    few_items += nf;
    tile_items += nt;
    units += nu;
    joins += nj;
  }
  // the tokens of bad sequences are in no tile: the join of no parts gives them their
  // zeros
  if (common.bad_seqs) {
    team.sync();
    for (int64_t t0 = 0; t0 < a.tokens; t0 += threads) {
      const int64_t t = t0 + tid;
      const int seq = t < a.tokens ? limits[t].seq : -1;
      const bool bad = seq == -2 || (seq >= 0 && !seq_ok(a, broken, seq));
      int total;
      const int at = joins + team.before((int)bad, total);
      if (bad) {
        rec_list[2 * t] = rec_list[2 * t + 1] = AttnParts{0, 0, 0, 0};
        join_list[at].token = (int)t;
      }
      joins += total;
    }
  }
  if (tid == 0) {
    if (slots > 0) slot_list[slots - 1].end = few_items;
    a.info[0] = slots;
    a.info[1] = tile_items;
    a.info[2] = common.bad_seqs;
    a.info[3] = common.bad_groups;
    a.info[4] = joins;
    a.info[5] = units;
    a.info[6] = (int)min_l(slice, 0x7fffffff);
    a.info[7] = (int)min_l(share, 0x7fffffff);
    a.info[8] = few_items;
    for (int k = 9; k < kAttnInfoInts; ++k) a.info[k] = 0;
  }
  // the list of tokens to join takes their records along
  team.sync();
  for (int j = tid; j < joins; j += threads) {
    AttnJoin &e = join_list[j];
    const AttnParts *rec = rec_list + 2 * (int64_t)e.token;
    e.own = rec[0];
    e.shared = rec[1];
  }
  // slices without work
  for (int k = slots + tid; k < a.max_slots; k += threads) slot_list[k].first = slot_list[k].end = 0;
}

}  // namespace lora
