// lora_attn_abi.hip -- the extern "C" entry points of the cache append and the
// attention declared in include/lora_mi355x.h: argument checks, workspace
// layout, launches.  Every check that can fail runs before the first HIP call.
#include <algorithm>

#include "../../include/lora_mi355x.h"
#include "lora_attn_host.h"

namespace lora {

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
size_t cache_esize(int32_t dtype) { return dtype == LORA_F32 ? 4 : dtype == LORA_BF16 ? 2 : 1; }
AttnKind kind_of(int32_t dtype) { return dtype == LORA_F32 ? kAttnF32 : dtype == LORA_E4M3 ? kAttnE4m3 : kAttnBf16; }
size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

lora_status check_geometry(const lora_kv_cache *c) {
  if (!c) return LORA_ERR_INVALID_ARG;
  if (c->dtype != LORA_F32 && c->dtype != LORA_BF16 && c->dtype != LORA_E4M3) return LORA_ERR_UNSUPPORTED;
  if (c->head_dim <= 0 || c->num_heads <= 0 || c->page_size <= 0) return LORA_ERR_INVALID_ARG;
  if (c->head_dim > 256 || c->head_dim % (c->dtype == LORA_E4M3 ? 16 : 8) || c->page_size > 65536 || c->num_heads > 1024)
    return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

lora_status check_cache(const lora_kv_cache *c) {
  const lora_status st = check_geometry(c);
  if (st != LORA_OK) return st;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return LORA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->num_pages > 0x7fffffff) return LORA_ERR_INVALID_ARG;
  const int64_t unit = 16 / (int64_t)cache_esize(c->dtype);
  for (int64_t s : {c->page_stride, c->head_stride, c->pos_stride})
    if (s < 0 || s % unit) return LORA_ERR_INVALID_ARG;
  // positions and heads of a page must not overlap
  if ((c->page_size > 1 && c->pos_stride < c->head_dim) || (c->num_heads > 1 && c->head_stride < c->head_dim) ||
      (c->num_pages > 1 && c->page_stride < c->head_dim))
    return LORA_ERR_INVALID_ARG;
  if (c->dtype != LORA_E4M3 && (c->k_scale || c->v_scale)) return LORA_ERR_INVALID_ARG;
  if (!aligned4(c->k_scale) || !aligned4(c->v_scale)) return LORA_ERR_INVALID_ARG;
  return LORA_OK;
}

// Sizes that follow from the batch and the cache's geometry.
struct AttnSizes {
  AttnShape shape;
  AttnCaps caps;
  size_t limits, info, tiles, few, slots, big, join, join_list, seq_end, group_end, total;
};

lora_status attn_sizes(const lora_attn_batch *b, const lora_kv_cache *c, AttnSizes &s) {
  if (!b) return LORA_ERR_INVALID_ARG;
  const lora_status st = check_geometry(c);
  if (st != LORA_OK) return st;
  if (b->num_tokens < 0 || b->num_seqs < 0 || b->max_q_len < 0 || b->num_groups < 0 || b->page_table_stride < 0 ||
      b->num_q_heads <= 0 || b->num_q_heads % c->num_heads || b->window < 0)
    return LORA_ERR_INVALID_ARG;
  if (b->num_tokens > (1 << 24) || b->num_seqs > (1 << 20) || b->num_groups > b->num_seqs ||
      b->num_q_heads > 1024 || b->num_tokens * b->num_q_heads > 0x7fffffff || b->page_table_stride > 0x7fff0000 / c->page_size)
    return LORA_ERR_UNSUPPORTED;
  s.shape = attn_shape(b->num_q_heads, c->num_heads, c->head_dim * (int64_t)cache_esize(c->dtype), c->dtype == LORA_F32,
                       b->num_groups, b->max_q_len);
  s.caps = attn_caps(b->num_tokens, b->num_seqs, b->num_groups, s.shape.heads, s.shape.group, s.shape.tile_rows, s.shape.few_slots);
  // the lists' lengths are 32-bit
  if (std::max(s.caps.few_items, s.caps.tile_items) > 0x7fffffff || s.caps.units > 0x7fffffff)
    return LORA_ERR_UNSUPPORTED;
  size_t at = 0;
  auto take = [&](int64_t ints) {
    const size_t p = at;
    at += round256(4 * (size_t)std::max<int64_t>(ints, 1));
    return p;
  };
  s.info = take(kAttnInfoInts);
  s.limits = take(4 * b->num_tokens);
  s.tiles = take(kAttnTileInts * s.caps.tiles);
  s.few = take(kAttnItemInts * s.caps.few_items);
  s.slots = take(kAttnSlotInts * s.caps.slots);
  s.big = take(kAttnItemInts * s.caps.tile_items);
  s.join = take(8 * b->num_tokens);
  s.join_list = take(kAttnJoinInts * b->num_tokens);
  s.seq_end = take(b->num_seqs);
  s.group_end = take(b->num_groups);
  s.total = at;
  return LORA_OK;
}

lora_status part_bytes(const lora_attn_meta *m, size_t &ml, size_t &total) {
  if (!m) return LORA_ERR_INVALID_ARG;
  if (m->max_units < 0 || m->max_units > 0x7fffffff || m->heads_per_item <= 0 || m->num_q_heads <= 0 || m->head_dim <= 0 ||
      m->head_dim > 256 || m->num_q_heads > 1024 || m->num_q_heads % m->heads_per_item)
    return LORA_ERR_INVALID_ARG;
  const int64_t rows = m->max_units * (m->num_q_heads / m->heads_per_item) * kUnitRows;
  ml = round256((size_t)rows * 8);
  total = ml + round256((size_t)rows * m->head_dim * 4);
  return LORA_OK;
}

}  // namespace

}  // namespace lora

using namespace lora;

extern "C" {

lora_status lora_cache_append(const void *d_qkv, int64_t ldx, int64_t T, lora_dtype dtype, int32_t num_q_heads,
                              const int64_t *offset, const lora_rotation *rot, const int32_t *d_pos,
                              const int64_t *d_slot, const lora_kv_cache *cache, void *d_q, int64_t ldq,
                              int32_t *d_num_bad, void *stream) {
  const lora_status st = check_cache(cache);
  if (st != LORA_OK) return st;
  if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_ERR_UNSUPPORTED;
  if ((dtype == LORA_F32) != (cache->dtype == LORA_F32)) return LORA_ERR_UNSUPPORTED;
  if (T < 0 || num_q_heads < 0 || !offset || ldx < 0 || ldx % 8) return LORA_ERR_INVALID_ARG;
  if (T > 0x7fffffff || num_q_heads > 1024) return LORA_ERR_UNSUPPORTED;
  const int64_t heads[3] = {num_q_heads, cache->num_heads, cache->num_heads};
  for (int s = 0; s < 3; ++s)
    if (offset[s] < 0 || offset[s] % 8 || offset[s] > ldx || heads[s] * cache->head_dim > ldx - offset[s])
      return LORA_ERR_INVALID_ARG;
  if (d_q && (!aligned16(d_q) || ldq % 8 || ldq < (int64_t)num_q_heads * cache->head_dim)) return LORA_ERR_INVALID_ARG;
  if (!aligned4(d_num_bad) || (reinterpret_cast<uintptr_t>(d_slot) & 7) || !aligned4(d_pos)) return LORA_ERR_INVALID_ARG;
  if (rot) {
    if (rot->reserved != 0 || rot->num_axes < 1 || rot->num_axes > 4 || rot->num_pos < 0 || rot->rot_dim <= 0 ||
        rot->rot_dim % 16 || rot->rot_dim > cache->head_dim || !rot->table || !aligned16(rot->table))
      return LORA_ERR_INVALID_ARG;
    if (rot->num_axes > 1) {
      int64_t sum = 0;
      for (int x = 0; x < rot->num_axes; ++x) {
        if (rot->section[x] < 0) return LORA_ERR_INVALID_ARG;
        sum += rot->section[x];
      }
      if (sum != rot->rot_dim / 2) return LORA_ERR_INVALID_ARG;
    }
  }
  if (T == 0) return LORA_OK;
  if (!d_qkv || !aligned16(d_qkv) || !d_slot || (rot && !d_pos)) return LORA_ERR_INVALID_ARG;

  AppendArgs a = {};
  a.x = static_cast<const char *>(d_qkv);
  a.q = num_q_heads ? static_cast<char *>(d_q) : nullptr;
  a.k = static_cast<char *>(cache->k);
  a.v = static_cast<char *>(cache->v);
  a.ldx = ldx;
  a.ldq = ldq;
  a.tokens = T;
  a.off_q = offset[0];
  a.off_k = offset[1];
  a.off_v = offset[2];
  a.page_stride = cache->page_stride;
  a.head_stride = cache->head_stride;
  a.pos_stride = cache->pos_stride;
  a.num_slots = cache->num_pages * cache->page_size;
  a.slot = d_slot;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.num_bad = d_num_bad;
  a.q_heads = num_q_heads;
  a.kv_heads = cache->num_heads;
  a.dim = cache->head_dim;
  a.page_size = cache->page_size;
  const int half = rot ? rot->rot_dim / 2 : 0;
  a.units[0] = divisor((uint32_t)std::max(half / 8, 1));
  a.units[1] = divisor((uint32_t)std::max((a.dim - 2 * half) / 8, 1));
  a.units[2] = divisor((uint32_t)(a.dim / 8));
  a.by_page = divisor((uint32_t)a.page_size);
  if (rot) {
    a.pos = d_pos;
    a.table = rot->table;
    a.num_pos = rot->num_pos;
    a.half = half;
    a.axes = rot->num_axes;
    a.interleaved = rot->interleaved != 0;
    int end = 0;
    for (int x = 0; x < 4; ++x) {
      if (x < rot->num_axes) end += rot->section[x];
      a.axis_end[x] = end;
    }
  }
  return launch_append(a, kind_of(cache->dtype), static_cast<hipStream_t>(stream)) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

lora_status lora_attn_meta_workspace_bytes(const lora_attn_batch *batch, const lora_kv_cache *cache, size_t *bytes) {
  AttnSizes s;
  const lora_status st = attn_sizes(batch, cache, s);
  if (st != LORA_OK) return st;
  if (!bytes) return LORA_ERR_INVALID_ARG;
  *bytes = s.total;
  return LORA_OK;
}

lora_status lora_prepare_attn_meta(const lora_attn_batch *b, const lora_kv_cache *cache, void *d_ws, size_t ws_bytes,
                                   lora_attn_meta *out, void *stream) {
  AttnSizes s;
  const lora_status st = attn_sizes(b, cache, s);
  if (st != LORA_OK) return st;
  if (!out || !d_ws || !aligned16(d_ws)) return LORA_ERR_INVALID_ARG;
  if (ws_bytes < s.total) return LORA_ERR_WORKSPACE;
  if (b->num_seqs > 0 && (!b->d_q_start || !b->d_kv_len || (b->page_table_stride > 0 && !b->d_page_table)))
    return LORA_ERR_INVALID_ARG;
  if (b->num_groups > 0 && (!b->d_group_start || !b->d_group_len)) return LORA_ERR_INVALID_ARG;
  if (!b->d_key_lo != !b->d_key_hi) return LORA_ERR_INVALID_ARG;
  for (const int32_t *p : {b->d_q_start, b->d_kv_len, b->d_page_table, b->d_prefix_len, b->d_key_lo, b->d_key_hi,
                           b->d_group_start, b->d_group_len})
    if (!aligned4(p)) return LORA_ERR_INVALID_ARG;

  char *ws = static_cast<char *>(d_ws);
  auto at = [&](size_t off) { return reinterpret_cast<int32_t *>(ws + off); };
  AttnPlanArgs a = {};
  a.q_start = b->d_q_start;
  a.kv_len = b->d_kv_len;
  a.prefix_len = b->d_prefix_len;
  a.key_lo = b->d_key_lo;
  a.key_hi = b->d_key_hi;
  a.group_start = b->d_group_start;
  a.group_len = b->d_group_len;
  a.tokens = b->num_tokens;
  a.table_stride = b->page_table_stride;
  a.seqs = b->num_seqs;
  a.groups = b->num_groups;
  a.max_q_len = b->max_q_len;
  a.page_size = cache->page_size;
  a.causal = b->causal != 0;
  a.window = b->window;
  a.heads = s.shape.heads;
  a.group = s.shape.group;
  a.tile_rows = s.shape.tile_rows;
  a.few_slots = s.shape.few_slots;
  a.limits = at(s.limits);
  a.info = at(s.info);
  a.tiles = at(s.tiles);
  a.few_items = at(s.few);
  a.tile_items = at(s.big);
  a.join = at(s.join);
  a.join_list = at(s.join_list);
  a.seq_end = at(s.seq_end);
  a.group_end = at(s.group_end);
  a.slots = at(s.slots);
  a.max_slots = (int32_t)s.caps.slots;

  *out = lora_attn_meta{};
  out->num_tokens = a.tokens;
  out->page_table_stride = b->page_table_stride;
  out->max_units = s.caps.units;
  out->num_seqs = b->num_seqs;
  out->num_q_heads = b->num_q_heads;
  out->num_kv_heads = cache->num_heads;
  out->head_dim = cache->head_dim;
  out->page_size = cache->page_size;
  out->dtype = cache->dtype;
  out->heads_per_item = a.group;
  out->head_groups = a.heads / cache->num_heads;
  out->max_tiles = (int32_t)s.caps.tiles;
  out->max_slots = a.max_slots;
  out->max_tile_items = s.shape.few_only ? 0 : (int32_t)s.caps.tile_items;
  out->page_table = b->d_page_table;
  out->limits = a.limits;
  out->info = a.info;
  out->tiles = a.tiles;
  out->few_items = a.few_items;
  out->slots = a.slots;
  out->tile_items = a.tile_items;
  out->join = a.join;
  out->join_list = a.join_list;
  return launch_attn_plan(a, static_cast<hipStream_t>(stream)) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

lora_status lora_attention_workspace_bytes(const lora_attn_meta *meta, size_t *bytes) {
  size_t ml, total;
  const lora_status st = part_bytes(meta, ml, total);
  if (st != LORA_OK) return st;
  if (!bytes) return LORA_ERR_INVALID_ARG;
  *bytes = total;
  return LORA_OK;
}

lora_status lora_attention(const lora_attn_meta *m, const void *d_q, int64_t ldq, const lora_kv_cache *cache, float scale,
                           float cap, const float *d_slopes, void *d_out, int64_t ldo, float *d_lse, void *d_ws,
                           size_t ws_bytes, void *stream) {
  size_t ml, total;
  lora_status st = part_bytes(m, ml, total);
  if (st != LORA_OK) return st;
  st = check_cache(cache);
  if (st != LORA_OK) return st;
  if (m->num_kv_heads != cache->num_heads || m->head_dim != cache->head_dim || m->page_size != cache->page_size ||
      m->dtype != cache->dtype || m->head_groups <= 0 ||
      m->head_groups * m->heads_per_item * m->num_kv_heads != m->num_q_heads || !m->limits || !m->info ||
      !m->few_items || !m->slots || !m->tile_items || !m->join || !m->join_list || m->max_slots < 1 || m->max_slots > 4096 ||
      m->max_tile_items < 0 ||
      m->num_tokens < 0 || m->num_tokens > 0x7fffffff / m->num_q_heads)
    return LORA_ERR_INVALID_ARG;
  const int64_t width = (int64_t)m->num_q_heads * m->head_dim;
  if (ldq % 8 || ldq < width || ldo % 8 || ldo < width || !(cap >= 0.f) || !(cap < __builtin_inff())) return LORA_ERR_INVALID_ARG;
  if (!aligned4(d_slopes) || !aligned4(d_lse)) return LORA_ERR_INVALID_ARG;
  if (m->num_tokens == 0) return LORA_OK;
  if (!d_q || !d_out || !aligned16(d_q) || !aligned16(d_out)) return LORA_ERR_INVALID_ARG;
  if (!d_ws || !aligned16(d_ws)) return LORA_ERR_INVALID_ARG;
  if (ws_bytes < total) return LORA_ERR_WORKSPACE;

  const int64_t e = (int64_t)cache_esize(cache->dtype);
  AttnArgs a = {};
  a.cache.k = static_cast<const char *>(cache->k);
  a.cache.v = static_cast<const char *>(cache->v);
  a.cache.page_bytes = cache->page_stride * e;
  a.cache.head_bytes = cache->head_stride * e;
  a.cache.pos_bytes = cache->pos_stride * e;
  a.cache.num_pages = (uint32_t)cache->num_pages;
  a.cache.page_size = divisor((uint32_t)cache->page_size);
  a.cache.table = m->page_table;
  a.cache.table_stride = m->page_table_stride;
  a.cache.k_scale = cache->k_scale;
  a.cache.v_scale = cache->v_scale;
  a.q = static_cast<const char *>(d_q);
  a.out = static_cast<char *>(d_out);
  a.lse = d_lse;
  a.slopes = d_slopes;
  a.limits = m->limits;
  a.info = m->info;
  a.join_list = m->join_list;
  a.ldq = ldq;
  a.ldo = ldo;
  a.tokens = m->num_tokens;
  a.max_units = m->max_units;
  a.part_ml = static_cast<float *>(d_ws);
  a.part = reinterpret_cast<float *>(static_cast<char *>(d_ws) + ml);
  a.scale = scale;
  a.cap = cap;
  a.group = m->heads_per_item;
  a.heads = m->num_q_heads / m->heads_per_item;
  a.q_heads = m->num_q_heads;
  a.by_heads = divisor((uint32_t)a.heads);
  a.by_group = divisor((uint32_t)a.group);
  a.by_q_heads = divisor((uint32_t)a.q_heads);
  a.by_kv_parts = divisor((uint32_t)m->head_groups);
  a.dim = m->head_dim;

  const AttnKind kind = kind_of(cache->dtype);
  hipStream_t s = static_cast<hipStream_t>(stream);
  a.few_items = m->few_items;
  a.slots = m->slots;
  a.tile_items = m->tile_items;
  a.few_waves = (m->max_slots - 1) * a.heads;
  // more tiles than this are taken in rounds (lora_attn.hip)
  a.tile_blocks = (int32_t)std::min<int64_t>((int64_t)m->max_tile_items * a.heads, kMaxTileBlocks / a.heads * a.heads);
  if (m->max_tile_items > 0 && a.tile_blocks == 0) a.tile_blocks = a.heads;
  hipError_t err = launch_attn(a, kind, s);
  if (err == hipSuccess) err = launch_attn_join(a, kind, s);
  return err == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // extern "C"
