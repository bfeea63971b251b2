// lora_attn_plan.h -- the attention metadata's algorithm: which keys a token sees,
// and the work lists.  Internal to the library.  Plain integer code over a Team of
// threads (a workgroup on the device, one thread in the CPU tests, which run it on
// buffers of exactly the workspace's sizes):
//   id(), size()       this thread and how many there are; loops go in steps of size()
//   sync()             what any thread wrote before, every thread reads after
//   before(v, total)   sum of v over the threads before this one, and over all
//   most_before(v, total)   likewise their maximum, of values from 0 on
//   shared()           a TeamShared that the threads have in common
//   add(p, v)          atomic add to it
#pragma once

#include "lora_attn.h"

namespace lora {

struct AttnPlanArgs {
  const int32_t *q_start, *kv_len, *prefix_len, *key_lo, *key_hi, *group_start, *group_len;
  int64_t tokens, table_stride;
  int32_t seqs, groups, max_q_len, page_size, causal, window;
  int32_t heads, group, tile_rows, few_slots;
  int32_t max_tiles, max_few_items, max_tile_items, max_units, max_slots;
  int32_t *limits, *info, *tiles, *few_items, *slots, *tile_items, *join, *join_list;
  int32_t *group_end;  // see group_ok
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
  int unordered;         // sequences whose bounds are out of order or leave the batch
  int unordered_groups;  // groups likewise
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

// Whether sequence n is usable (see lora_attn_batch).
LORA_HD bool seq_ok(const AttnPlanArgs &a, int n) {
  const int64_t q0 = a.q_start[n], q1 = a.q_start[n + 1], kv = a.kv_len[n];
  return seq_ordered(a, n) && q1 - q0 <= a.max_q_len && kv >= q1 - q0 && kv <= a.table_stride * a.page_size;
}

LORA_HD bool group_ordered(const AttnPlanArgs &a, int g) {
  const int s0 = a.group_start[g], s1 = a.group_start[g + 1];
  return s0 >= 0 && s1 >= s0 && s1 <= a.seqs;
}

// Whether group g would be served if it were the only one.  Its tokens are those
// between its first sequence's bound and its last one's, which holds its members'
// only if all bounds ascend.
LORA_HD bool group_alone_ok(const AttnPlanArgs &a, const TeamShared &common, int g) {
  if (common.unordered || !group_ordered(a, g) || a.group_len[g] < 0) return false;
  const int s0 = a.group_start[g];
  return s0 == a.group_start[g + 1] || (seq_ok(a, s0) && a.group_len[g] <= a.kv_len[s0]);
}

// Whether group g is served.  One rule for its members and for its tiles, since a
// member's join reads what the group's tiles leave.  Where starts are out of order
// (beside a bad group), group_end[g] is the furthest end of a group up to g, and a
// group that starts before it shares sequences with an earlier one: it is bad.
LORA_HD bool group_ok(const AttnPlanArgs &a, const TeamShared &common, int g) {
  if (!group_alone_ok(a, common, g)) return false;
  const int s0 = a.group_start[g];
  return !common.unordered_groups || g == 0 || s0 == a.group_start[g + 1] || s0 >= a.group_end[g - 1];
}

// Group of sequence n, or -1: the last group that starts at or before n, or the first
// whose furthest end lies past n.
LORA_HD int group_of(const AttnPlanArgs &a, const TeamShared &common, int n) {
  int lo = 0, hi = a.groups;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (common.unordered_groups ? a.group_end[mid] <= n : a.group_start[mid] <= n) lo = mid + 1;
    else hi = mid;
  }
  const int g = common.unordered_groups ? lo : lo - 1;
  if (g < 0 || g >= a.groups || n < a.group_start[g] || n >= a.group_start[g + 1] || a.group_len[g] == 0 || !group_ok(a, common, g)) return -1;
  return g;
}

// What token t sees.
LORA_HD AttnLimit limit_of(const AttnPlanArgs &a, int64_t t) {
  int lo = 0, hi = a.seqs;  // first sequence whose tokens start after t
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.q_start[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  const int n = lo - 1;
  AttnLimit r{0, 0, 0, -1};
  if (n >= 0 && t < a.q_start[n + 1]) {
    r.seq = n;
    if (seq_ok(a, n)) {
      const int kv = a.kv_len[n];
      r.pos = (int)(kv - a.q_start[n + 1] + t);
      r.hi = a.causal ? r.pos + 1 : kv;
      if (a.prefix_len) r.hi = max_i(r.hi, a.prefix_len[n]);
      if (a.window > 0) r.lo = max_i(0, r.pos + 1 - a.window);
      if (a.key_lo) r.lo = max_i(r.lo, a.key_lo[t]);
      if (a.key_hi) r.hi = min_i(r.hi, a.key_hi[t]);
      r.hi = min_i(r.hi, kv);
      if (r.hi <= r.lo) r.lo = r.hi = 0;
    }
  }
  return r;
}

template <typename Team>
LORA_HD void attn_plan(const AttnPlanArgs &a, Team &team) {
  TeamShared &common = team.shared();
  const int tid = team.id(), threads = team.size();
  const AttnLimit *limits = reinterpret_cast<const AttnLimit *>(a.limits);
  AttnTile *tile_list = reinterpret_cast<AttnTile *>(a.tiles);
  AttnParts *rec_list = reinterpret_cast<AttnParts *>(a.join);
  AttnJoin *join_list = reinterpret_cast<AttnJoin *>(a.join_list);
  if (tid == 0) common = TeamShared{0, 0, 0, 0, 0};
  team.sync();

  // ---- tiles per sequence, then per group: which one, and which of its tiles
  const int few_tokens = kFewRows / a.group, tile_tokens = a.tile_rows / a.group;
  int own = 0, tiles = 0;
  for (int pass = 0; pass < 2; ++pass) {
    const int count_all = pass ? a.groups : a.seqs;
    for (int n0 = 0; n0 < count_all; n0 += threads) {
      const int n = n0 + tid;
      int count = 0;
      if (n < count_all) {
        int64_t q0 = 0, q1 = 0;
        if (pass == 0) {
          if (seq_ok(a, n)) q0 = a.q_start[n], q1 = a.q_start[n + 1];
          else team.add(&common.bad_seqs, 1);
          if (!seq_ordered(a, n)) team.add(&common.unordered, 1);
          // (there are no more groups than sequences)
          if (n < a.groups && !group_ordered(a, n)) team.add(&common.unordered_groups, 1);
        } else if (!group_ok(a, common, n)) {
          team.add(&common.bad_groups, 1);
        } else if (a.group_len[n] > 0 && a.group_start[n] < a.group_start[n + 1]) {
          q0 = a.q_start[a.group_start[n]];
          q1 = a.q_start[a.group_start[n + 1]];
        }
        const int len = (int)(q1 - q0);
        count = len <= few_tokens ? (len > 0) : (len + tile_tokens - 1) / tile_tokens;
      }
      int total;
      const int before = tiles + team.before(count, total);
      for (int i = 0; i < count && before + i < a.max_tiles; ++i) {
        tile_list[before + i].seq = n;
        tile_list[before + i].part = i;
      }
      tiles = min_i(tiles + total, a.max_tiles);
    }
    if (pass == 0) own = tiles;
    team.sync();  // the counts; the list is written and read by this team alone
    if (pass == 0 && common.unordered_groups) {
      int end = 0;
      for (int g0 = 0; g0 < a.groups; g0 += threads) {
        const int g = g0 + tid;
        const int mine = g < a.groups && group_alone_ok(a, common, g) && a.group_start[g] < a.group_start[g + 1] ? a.group_start[g + 1] : 0;
        int most;
        const int before = team.most_before(mine, most);
        if (g < a.groups) a.group_end[g] = max_i(end, max_i(before, mine));
        end = max_i(end, most);
      }
      team.sync();
    }
  }

  // ---- the tiles' tokens and keys; few-row tiles take their place on the line
  long long line = 0;
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
        const int g = a.groups ? group_of(a, common, n) : -1;
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
    int total;
    const int before = team.before(width, total);
    if (i < tiles) {
      r.at = line + before;
      tile_list[i] = r;
    }
    line += total;
  }
  if (keys) team.add(&common.keys, keys);
  team.sync();
  const int slice = share_of(line * kCutKeys, a.heads, a.few_slots, kFewMinKeys, kCutKeys);
  const int share = share_of((int64_t)common.keys, a.heads, kTileSlots, kTileMinKeys, kPartKeys);
  const int cuts = slice / kCutKeys;  // of a slice
  const int slots = (int)min_l((line + cuts - 1) / cuts, a.max_slots - 1);

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
        parts = max_i(1, (n + per - 1) / per);
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
      // true for every batch in order, by the capacities' derivation; with a
      // q_start out of order the surplus is dropped
      const bool fits = (few ? at_few + parts <= a.max_few_items : at_tile + parts <= a.max_tile_items) &&
                        unit + parts * ups <= a.max_units;
      AttnItem item{r.tok0, fits ? r.ntok : 0, r.seq, r.key0, r.key1, r.full0, r.full1, -1};
      for (int s = 0; s < parts; ++s) {
        const int at = (few ? at_few : at_tile) + s;
        if (at >= (few ? a.max_few_items : a.max_tile_items)) break;
        if (join) item.unit = unit + s * ups;
        if (few) {
          // the piece of the tile on slice k: the line from `from` on
          const int64_t k = r.at / cuts + s, from = max_l(r.at, k * cuts);
          item.key0 = r.key0 + (int)(from - r.at) * kCutKeys;
          item.key1 = (int)min_l(r.key1, r.key0 + ((k + 1) * cuts - r.at) * kCutKeys);
          few_list[at] = item;
          if (from == k * cuts && k < a.max_slots) {
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
          rec[r.shared == 1] = AttnParts{unit, fits ? parts : 0, ups, t};
          if (r.shared == 0) rec[1] = AttnParts{0, 0, 0, 0};
          if (r.shared != 1 && at_join + t < a.tokens) join_list[at_join + t].token = r.tok0 + t;
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
      const bool bad = t < a.tokens && limits[t].seq >= 0 && !seq_ok(a, limits[t].seq);
      int total;
      const int at = joins + team.before((int)bad, total);
      if (bad && at < a.tokens) {
        rec_list[2 * t] = rec_list[2 * t + 1] = AttnParts{0, 0, 0, 0};
        join_list[at].token = (int)t;
      }
      joins += total;
    }
  }
  few_items = min_i(few_items, a.max_few_items);
  joins = (int)min_l(joins, a.tokens);
  if (tid == 0) {
    if (slots > 0) slot_list[slots - 1].end = few_items;
    a.info[0] = slots;
    a.info[1] = min_i(tile_items, a.max_tile_items);
    a.info[2] = common.bad_seqs;
    a.info[3] = common.bad_groups;
    a.info[4] = joins;
    a.info[5] = min_i(units, a.max_units);
    a.info[6] = slice;
    a.info[7] = share;
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
