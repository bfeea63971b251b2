/*
 * lora_mi355x.h -- C ABI of the multi-LoRA batched low-rank delta on MI355X
 * (gfx950): slot metadata, shrink, expand, and the fused apply; and of the
 * attention that its q/k/v rows go on to: cache append, attention metadata,
 * attention (the last part of this file, with conventions of its own where it
 * says so).
 *
 * For a batch of T tokens, token t names an adapter slot token_slot[t] in
 * [0, S), or -1 for "no adapter".  The library adds, for every packed output
 * slice s (column window [offset[s], offset[s] + width[s]) of y),
 *
 *     y[t][offset[s] + n] (+)= sum_j u[s][t][j] * B_s[slot][j][n]
 *     u[s][t][j]           =  scale * slot_scale[slot] * sum_k x[t][k] * A_s[slot][k][j]
 *
 * which is y = xW + s*(xA)B of the LoRA forward with the base product xW
 * already in y (page "多 LoRA 服务：分段矩阵乘与适配器调度", section
 * "不合并权重，批量计算"), split into a shrink (x -> rank r, kept in fp32) and
 * an expand (rank r -> output slice) as in page "vLLM 源码完全拆解(十八):多 LoRA
 * 服务", sections "调用链" and "两个低秩 GEMM:shrink、expand 与 fp32 中转缓冲".
 *
 * Conventions shared by every entry point
 *   - Device pointers are HIP device addresses; "host" arrays live in host memory
 *     and are read before the call returns.
 *   - The caller owns every buffer, device and host.  The library never
 *     allocates or frees memory, never synchronises, and keeps no pointer after
 *     a call returns.  All device work is enqueued on `stream` (a hipStream_t
 *     passed as void*, NULL = the null stream), so calls are asynchronous.
 *   - Errors are return codes; nothing is enqueued when a call returns anything
 *     but LORA_OK, except LORA_ERR_HIP, which reports a failed launch.
 *   - Element types: x, A, B and y share one dtype, fp32 or bf16; the rank-r
 *     buffer u is always fp32; scales are fp32.  Accumulation is fp32.  bf16
 *     outputs are rounded once, to nearest even, when y is stored.
 *   - Supported shapes: 1 <= S <= 1023, r_max a multiple of 8 in [8, 128]
 *     (the kernels run at the next of 8, 16, 32, 64, 128 and read ranks past
 *     r_max as zeros; A, B and u keep r_max as their rank extent), d_in and every
 *     slice width a multiple of 8, 1 <= n_slices <= 8, every device pointer
 *     16-byte aligned, ldx and ldy multiples of 8, (r_max + 1) * d_in and
 *     (r_max + 1) * width below 2^28 (one slot's factor matrix is addressed with
 *     32-bit byte offsets).  Row offsets into x, u and y are int64.
 */
#ifndef LORA_MI355X_H
#define LORA_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lora_status {
    LORA_OK = 0,
    LORA_ERR_INVALID_ARG = 1,       /* null pointer, bad size, misalignment, overlap */
    LORA_ERR_UNSUPPORTED = 2,       /* dtype, r_max, slot count or slice count not built */
    LORA_ERR_WORKSPACE = 3,         /* workspace smaller than the *_workspace_bytes value */
    LORA_ERR_HIP = 4,               /* a HIP launch failed (hipGetLastError) */
    /* Range markers, not statuses: with them every int is a value of the type,
     * so a C caller may pass any int and a C++ definition may read it. */
    LORA_STATUS_RANGE_MIN_ = -2147483647 - 1,
    LORA_STATUS_RANGE_MAX_ = 2147483647
} lora_status;

typedef enum lora_dtype {
    LORA_F32 = 0,
    LORA_BF16 = 1,
    LORA_E4M3 = 2,                  /* 8-bit float (1-4-3, no infinities, largest 448):
                                       elements of a lora_kv_cache only */
    LORA_DTYPE_RANGE_MIN_ = -2147483647 - 1,  /* range markers, as above */
    LORA_DTYPE_RANGE_MAX_ = 2147483647
} lora_dtype;

/* How segments are computed.  BGMV: every segment on the vector (matrix-vector)
 * path; SGMV: every segment on the matrix-core tile path (bf16 only; fp32 falls
 * back to the vector path); AUTO: per segment, by its token count. */
typedef enum lora_mode {
    LORA_MODE_AUTO = 0,
    LORA_MODE_BGMV = 1,
    LORA_MODE_SGMV = 2,
    LORA_MODE_RANGE_MIN_ = -2147483647 - 1,  /* range markers, as above */
    LORA_MODE_RANGE_MAX_ = 2147483647
} lora_mode;

/* Layout of a slice's per-slot factor matrices (lora_weight.layout). */
typedef enum lora_layout {
    /* A_s [d_in][r_max] (row stride r_max), B_s [r_max][width_s] (row stride
     * width_s): the layout of page "多 LoRA 服务：分段矩阵乘与适配器调度",
     * section "不合并权重，批量计算". */
    LORA_LAYOUT_DEFAULT = 0,
    /* A only: A_s [r_max][d_in] (row stride d_in), the rank-major layout of
     * page "vLLM 源码完全拆解(十八):多 LoRA 服务", section "包装层的形态".  A
     * slot's ranks are then whole rows, so with per-slot ranks (d_slot_rank)
     * the ranks past a slot's own are never fetched.  bf16 only, r_max >= 16,
     * mode AUTO or SGMV; every slice of A must use it (else
     * LORA_ERR_UNSUPPORTED / LORA_ERR_INVALID_ARG). */
    LORA_LAYOUT_RANK_ROWS = 1,
    /* B only: B_s [width_s][r_max] (row stride r_max), one row of ranks per
     * output column: the output-major B of the same page and section (B
     * stored d_out x r).  A step of the expand then reads one contiguous
     * block of B.  bf16 only, r_max <= 64, mode AUTO or SGMV; every slice of B
     * must use it (else LORA_ERR_UNSUPPORTED / LORA_ERR_INVALID_ARG).
     * lora_apply runs such calls on the tile kernels (matrix-core expand),
     * never on the decode kernels or the long-segment expand. */
    LORA_LAYOUT_OUT_ROWS = 2
} lora_layout;

/* One packed slice of a stacked factor: slot a's matrix starts at
 * ptr + a * slot_stride elements, laid out as `layout` says. */
typedef struct lora_weight {
    const void *ptr;
    int64_t slot_stride;            /* elements between consecutive slots */
    int32_t layout;                 /* a lora_layout value */
    int32_t reserved;               /* must be 0 */
} lora_weight;

/* Bytes at the start of every lora_apply workspace that hold the per-tile call
 * count words of the decode-shaped apply (below, lora_apply_workspace_init). */
#define LORA_APPLY_SYNC_BYTES 295168
/* Word indices, in that region, of two counters the decode-shaped apply keeps
 * (read them as uint32): waits for peer workgroups' partial results that gave
 * up, and peers met on another accelerator die (XCD).  Each case is handled
 * (the waiting workgroup computes the peer's share itself, with the same
 * result); the counters only report that it happened. */
#define LORA_APPLY_WAITS_GAVE_UP_WORD 73728
#define LORA_APPLY_OTHER_XCD_WORD 73729

/* Slot metadata of one batch (page "vLLM 源码完全拆解(十八):多 LoRA 服务",
 * section "LoRAKernelMeta:先按槽位排序").  lora_prepare_meta fills the struct on
 * the host with device pointers into the caller's workspace and enqueues the
 * kernel that writes the arrays:
 *   sorted[T]       token indices grouped by slot: -1 first, then slots in
 *                   ascending order; original order inside a slot (stable)
 *   sorted_slot[T]  slot of each entry of `sorted` (-1 for no adapter)
 *   seg_slot[S+1]   slot id of each segment in that order, then -1 padding
 *   seg_count[S+1]  tokens per segment, then 0 padding
 *   seg_start[S+2]  0, then running sums of seg_count; T past the last segment
 *   info[8]         num_segments, no_lora (1 when no token has a valid slot,
 *                   also for T = 0), num_bad (tokens whose id lies outside
 *                   [-1, S); they are treated as -1), lora_begin (index in
 *                   `sorted` of the first token with an adapter), num_tiles,
 *                   then 3 zeros
 *   tiles           work tiles: every segment (the -1 one included) cut into
 *                   runs of at most 64 consecutive entries of `sorted`; tile i
 *                   is 68 int32 at tiles + 68 i: slot, rows, first position in
 *                   `sorted`, 0, then the rows token indices (the rest
 *                   unspecified).  Tiles follow the order of `sorted`; there
 *                   are num_tiles <= ceil(T / 64) + S + 1 of them.  The compute
 *                   kernels take their work from this list.
 * Past the tiles the workspace holds per-key counts that lora_prepare_meta
 * uses while it builds the arrays (large batches are counted in parts, by
 * several workgroups); they are not part of the result.
 * The struct stays valid until its workspace is reused; rebuild it whenever
 * token_slot changes.  Pass it by pointer to the compute calls.  They only
 * read it, so any number of calls, on any streams, may use one lora_meta at
 * the same time. */
typedef struct lora_meta {
    int64_t num_tokens;             /* rows of the batch */
    int32_t num_slots;              /* keys: slots, or (slot, local expert) pairs */
    int32_t x_row_div;              /* row i of the batch reads row i / x_row_div of x
                                       (1, or top-k for the MoE gate/up LoRA) */
    int32_t *sorted;
    int32_t *sorted_slot;
    int32_t *seg_slot;
    int32_t *seg_count;
    int32_t *seg_start;
    int32_t *info;
    int32_t *tiles;
} lora_meta;

/* Bytes of device workspace lora_prepare_meta needs for T tokens and S slots. */
lora_status lora_meta_workspace_bytes(int64_t num_tokens, int32_t num_slots,
                                      size_t *bytes);

/* Build the slot metadata of a batch.
 *   d_token_slot  device int32 [T], slot per token (-1 = none)
 *   d_ws          device workspace of at least lora_meta_workspace_bytes bytes,
 *                 16-byte aligned; owned by the caller, overwritten
 *   out           host struct, filled with pointers into d_ws
 * Cites page "vLLM 源码完全拆解(十八):多 LoRA 服务", section
 * "LoRAKernelMeta:先按槽位排序" (stable sort, unique counts, running sum whose
 * first entry is 0) and the worked example of section "一个完整的走查:两步
 * decode 里发生了什么".  T = 0 is valid (no_lora = 1).  Sets x_row_div = 1. */
lora_status lora_prepare_meta(const int32_t *d_token_slot, int64_t num_tokens,
                              int32_t num_slots, void *d_ws, size_t ws_bytes,
                              lora_meta *out, void *stream);

/* Per-slot ranks (argument d_slot_rank of lora_shrink, lora_expand and
 * lora_apply): NULL, or device int32 [S] giving the rank r_a <= r_max that slot
 * a's adapter really has.  The stacked buffers are sized for r_max, and an
 * adapter of smaller rank occupies only its first r_a columns of A and rows of
 * B, the rest being zero (page "vLLM 源码完全拆解(十八):多 LoRA 服务", section
 * "两个 LRU 缓存": a slot's buffers are written only in the adapter's valid
 * range).  With d_slot_rank the kernels read only those ranks, rounded up to a
 * multiple of 8, so a batch that mixes ranks no longer moves every adapter at
 * r_max (page "多 LoRA 服务：分段矩阵乘与适配器调度", section "练习": mixed ranks
 * padded to the largest waste memory traffic).  The result equals the padded
 * one whenever the padding holds zeros; u[s][t][j] is written as 0 for
 * j >= r_a.  Values are clamped to [0, r_max]. */

/* MoE LoRA: metadata over the (token, choice) pairs of a top-k routing step,
 * keyed by (slot, local expert).  Page "vLLM 源码完全拆解(十八):多 LoRA 服务",
 * section "融合计算:add_lora_w13 与 add_lora_w2": the experts' LoRA is applied
 * after the gate/up projection (before the activation) and after the down
 * projection (before the top-k weighted sum), on the tokens regrouped by
 * (adapter, expert); section "MoE 的 LoRA:按专家挂载、融合 kernel 与 EP 切片",
 * its buffer list: the factors are stacked per slot and
 * local expert; section "EP 下只装载本地专家的权重": a rank holds only its
 * local experts.
 * Row p = t * topk + j is token t's j-th choice.  Its key is
 *     slot(t) * E_local + local(topk_ids[t][j])
 * where local(e) = d_expert_map[e] when a map is given (-1: the expert lives
 * on another rank) and e otherwise; the key is -1 when the token has no
 * adapter or the expert is not local.  Ids out of range (a slot outside
 * [-1, S), an expert outside [0, E_global), a mapped id outside [-1, E_local),
 * or without a map an expert >= E_local) count as bad (info[2]) and as -1.
 * The result is an ordinary lora_meta over T * topk rows and S * E_local keys
 * (S * E_local <= 1023), with x_row_div = topk: lora_shrink and lora_apply
 * then read x row t for pair p, the token's hidden state (gate/up LoRA).  For
 * the down-projection LoRA, whose input has one row per pair, use a copy of
 * the struct with x_row_div = 1.  Factor slot index = slot * E_local + expert:
 * for stacks [S][E_local][...] pass slot_stride = one expert's matrix.
 *   d_topk_ids    device int32 [T][topk]
 *   d_token_slot  device int32 [T]
 *   d_expert_map  device int32 [E_global] or NULL */
lora_status lora_moe_meta_workspace_bytes(int64_t num_tokens, int32_t topk,
                                          int32_t num_slots,
                                          int32_t num_local_experts,
                                          size_t *bytes);
lora_status lora_prepare_moe_meta(const int32_t *d_topk_ids, int64_t num_tokens,
                                  int32_t topk, const int32_t *d_token_slot,
                                  int32_t num_slots, int32_t num_experts,
                                  int32_t num_local_experts,
                                  const int32_t *d_expert_map, void *d_ws,
                                  size_t ws_bytes, lora_meta *out, void *stream);

/* Bytes of device workspace lora_shrink needs (split-K partial sums; 0 when
 * the shape needs none).  No initialisation is required; calls that run at the
 * same time need workspaces of their own. */
lora_status lora_shrink_workspace_bytes(int64_t num_tokens, int32_t num_slots,
                                        int64_t d_in, int32_t n_slices,
                                        int32_t r_max, lora_dtype dtype,
                                        lora_mode mode, size_t *bytes);

/* Shrink: u[s][t][j] = scale * slot_scale[slot(t)] * sum_k x[t][k] * A_s[slot(t)][k][j]
 * for every token t with an adapter and every slice s; rows of tokens without
 * an adapter are not written.
 *   meta          metadata from lora_prepare_meta for this batch
 *   d_x           device [T][ldx] of dtype; the first d_in columns are read
 *   A             host array of n_slices descriptors (device pointers)
 *   scale         fp32 multiplier; d_slot_scale: device fp32 [S] or NULL (= 1)
 *   d_slot_rank   device int32 [S] or NULL (= r_max for every slot), see above
 *   d_u           device fp32 [n_slices][T][r_max], contiguous
 *   d_ws          workspace of lora_shrink_workspace_bytes bytes (may be NULL
 *                 when that size is 0)
 * Cites page "vLLM 源码完全拆解(十八):多 LoRA 服务", section "两个低秩 GEMM:
 * shrink、expand 与 fp32 中转缓冲" (the shrink kernel, its scaling argument and
 * the fp32 buffer laid out [slice][token][rank]). */
lora_status lora_shrink(const lora_meta *meta, const void *d_x, int64_t ldx,
                        int64_t d_in, lora_dtype dtype, int32_t n_slices,
                        const lora_weight *A, int32_t r_max, float scale,
                        const float *d_slot_scale, const int32_t *d_slot_rank,
                        float *d_u, lora_mode mode, void *d_ws, size_t ws_bytes,
                        void *stream);

/* Expand: for every token t and slice s, columns [offset[s], offset[s]+width[s])
 * of row t of y become (add_into_y ? y : 0) + sum_j u[s][t][j] * B_s[slot(t)][j][n];
 * a token without an adapter contributes 0 (its row is left as is when
 * add_into_y != 0 and its windows are set to 0 otherwise).  Columns outside
 * every window are never touched.
 *   d_u           device fp32 [n_slices][T][r_max] from lora_shrink
 *   B             host array of n_slices descriptors
 *   width, offset host int64 arrays [n_slices]; windows must not overlap and
 *                 must lie inside [0, ldy)
 *   d_slot_rank   device int32 [S] or NULL; ranks j >= r_a of u and B are not read
 *   d_y           device [T][ldy] of dtype, updated in place
 * Cites page "vLLM 源码完全拆解(十八):多 LoRA 服务", section "两个低秩 GEMM:
 * shrink、expand 与 fp32 中转缓冲" (the expand kernel: per-slice width and start
 * column, ADD_INPUTS) and section "双流:让 LoRA 与基座前向并行" (rows without an
 * adapter and a cleared output). */
lora_status lora_expand(const lora_meta *meta, const float *d_u, int32_t n_slices,
                        const lora_weight *B, const int64_t *width,
                        const int64_t *offset, int32_t r_max,
                        const int32_t *d_slot_rank, void *d_y, int64_t ldy,
                        lora_dtype dtype, int add_into_y, lora_mode mode,
                        void *stream);

/* Bytes of device workspace lora_apply needs for these sizes (a workspace
 * sized for the largest call can serve every smaller one).  Layout: the
 * count words (LORA_APPLY_SYNC_BYTES), the fp32 rank-r buffer, then the
 * partial sums of a shrink that splits d_in or of the decode-shaped kernel.
 * Only the count words need initialising: see lora_apply_workspace_init. */
lora_status lora_apply_workspace_bytes(int64_t num_tokens, int32_t num_slots,
                                       int64_t d_in, int32_t n_slices,
                                       int32_t r_max, lora_dtype dtype,
                                       lora_mode mode, size_t *bytes);

/* Zero the count words of an apply workspace (its first
 * LORA_APPLY_SYNC_BYTES bytes; enqueued on `stream`).  Call it once, before
 * the first lora_apply on a workspace; zero-filled memory needs no call.  The
 * decode-shaped apply (page "多 LoRA 服务：分段矩阵乘与适配器调度", section
 * "不合并权重，批量计算": the fused form for decode batches) spreads each work
 * tile over several workgroups that exchange partial results tagged with the
 * tile, the slice range and the call count, which these words keep.  Every
 * call leaves them consistent for the next call on the same workspace,
 * whatever its shapes.
 * The words must not be written between calls.
 *   d_ws      device workspace, 16-byte aligned
 *   ws_bytes  its size, at least LORA_APPLY_SYNC_BYTES (else LORA_ERR_WORKSPACE) */
lora_status lora_apply_workspace_init(void *d_ws, size_t ws_bytes, void *stream);

/* Shrink then expand on one stream: the whole delta of one layer, added into
 * (or stored to) the slices of y.  Arguments as in lora_shrink and lora_expand;
 * the rank-r buffer lives in d_ws.  Decode-shaped calls (few tokens per slot,
 * small per-token factors, mode AUTO or BGMV, r_max one of 8, 16, 32, 64,
 * default factor layouts) run as one fused kernel that keeps each token's
 * rank-r vector on chip; the others run the shrink and expand kernels.  Cites
 * page "vLLM 源码完全拆解(十八):多 LoRA
 * 服务", section "调用链" (add_lora_linear = shrink into an fp32 buffer, then
 * expand into the output slices).
 *   d_ws      workspace of at least lora_apply_workspace_bytes bytes, 16-byte
 *             aligned, whose count words were initialised once
 *             (lora_apply_workspace_init) and not written since except by
 *             lora_apply.  Calls that run at the same time need workspaces of
 *             their own; calls in stream order may share one. */
lora_status lora_apply(const lora_meta *meta, const void *d_x, int64_t ldx,
                       int64_t d_in, lora_dtype dtype, int32_t n_slices,
                       const lora_weight *A, const lora_weight *B,
                       const int64_t *width, const int64_t *offset,
                       int32_t r_max, float scale, const float *d_slot_scale,
                       const int32_t *d_slot_rank, void *d_y, int64_t ldy,
                       int add_into_y, lora_mode mode, void *d_ws,
                       size_t ws_bytes, void *stream);

/* Size of the device array that lora_apply_noalloc uses as its workspace. */
#define LORA_NOALLOC_SCRATCH_BYTES (64u << 20)

/* lora_apply for callers that cannot allocate device memory or pass a
 * workspace: code under HIP graph capture, tight serving loops, harnesses that
 * forbid allocation.  Same arguments, checks and results as lora_apply,
 * without d_ws and ws_bytes: the workspace is a static device array of the
 * library, LORA_NOALLOC_SCRATCH_BYTES (64 MiB) per device, which each device
 * holds from the library's first use there until the process ends (zero at
 * load, so no lora_apply_workspace_init is needed).  Calls whose
 * lora_apply_workspace_bytes exceed that size return LORA_ERR_WORKSPACE and
 * enqueue nothing.  Allocates nothing: no hipMalloc, no hipFree, no allocating
 * library routine; the first call on a device looks up that device's copy of
 * the array once (hipGetSymbolAddress; LORA_ERR_HIP if that fails).  Every call
 * on a device shares its array: calls in stream order are fine, but calls
 * that overlap on one device (other streams, graphs replayed at the same time)
 * race and give wrong results. */
lora_status lora_apply_noalloc(const lora_meta *meta, const void *d_x, int64_t ldx,
                               int64_t d_in, lora_dtype dtype, int32_t n_slices,
                               const lora_weight *A, const lora_weight *B,
                               const int64_t *width, const int64_t *offset,
                               int32_t r_max, float scale, const float *d_slot_scale,
                               const int32_t *d_slot_rank, void *d_y, int64_t ldy,
                               int add_into_y, lora_mode mode, void *stream);

/* ---------------------------------------------------------------------------
 * Attention next to the q/k/v delta.  A layer's q/k/v projection leaves one
 * packed row q | k | v per token (lora_apply adds the adapters' share into it);
 * the entry points below rotate q and k, append k and v to a paged cache, and
 * attend.  The keys and values of a request carry its adapter's delta, so
 * cached pages may be shared by requests of one adapter only.
 * ------------------------------------------------------------------------- */

/* A paged key/value cache.  Element d of the key at position i of page p for
 * key head h is k[p * page_stride + h * head_stride + i * pos_stride + d], and
 * likewise in v: [page][head][position][dim], [page][position][head][dim] and
 * k and v interleaved in one buffer are all expressed by the strides.
 *   dtype         LORA_BF16 or LORA_E4M3 (with bf16 queries), LORA_F32 (with
 *                 fp32 queries)
 *   k_scale, v_scale  device fp32 [num_heads] or NULL (= 1): with LORA_E4M3 a
 *                 stored value stands for value * scale[head], scales positive;
 *                 must be NULL for the other types
 * Supported: head_dim a multiple of 8 (16 with LORA_E4M3), at most 256, page_size in [1, 65536],
 * num_pages in [1, 2^31 - 1], at most 1024 heads, strides whose byte size is a
 * multiple of 16.  Offsets are int64. */
typedef struct lora_kv_cache {
    void *k, *v;
    int64_t page_stride, head_stride, pos_stride;   /* elements, k and v alike */
    int64_t num_pages;
    int32_t page_size, num_heads, head_dim;
    int32_t dtype;                  /* a lora_dtype value */
    const float *k_scale, *v_scale;
} lora_kv_cache;

/* Rotary positions.  Pair j < rot_dim / 2 of a head is turned by the angle
 * whose cosine and sine are table[pos][j] and table[pos][rot_dim / 2 + j]:
 *     a' = a cos - b sin,  b' = b cos + a sin     (fp32, rounded once)
 * with (a, b) = elements (j, j + rot_dim / 2), or (2j, 2j + 1) if interleaved;
 * elements from rot_dim on are copied.  With num_axes = 2..4 (time, height,
 * width of images and video) pair j takes its position from the axis whose
 * section holds j: the first section[0] pairs from axis 0, the next section[1]
 * from axis 1, and so on; the sections add up to rot_dim / 2 (num_axes = 1:
 * section is not read).
 *   table         device fp32 [num_pos][rot_dim], contiguous, 16-byte aligned
 * rot_dim is a multiple of 16, at most head_dim. */
typedef struct lora_rotation {
    const float *table;
    int64_t num_pos;
    int32_t rot_dim;
    int32_t interleaved;
    int32_t num_axes;
    int32_t section[4];
    int32_t reserved;               /* must be 0 */
} lora_rotation;

/* Rotate q and k of every token, write q to d_q and k, v to their place in the
 * cache, in one pass.
 *   d_qkv         device [T][ldx] of dtype (LORA_F32 or LORA_BF16): num_q_heads
 *                 heads of q at column offset[0], cache->num_heads heads of k at
 *                 offset[1] and of v at offset[2], head_dim columns each
 *   offset        host int64 [3], multiples of 8
 *   rot           NULL: no rotation (d_pos is then not read)
 *   d_pos         device int32 [num_axes][T]
 *   d_slot        device int64 [T]: page * page_size + position in the page, or
 *                 -1: the token's k and v are not kept.  Two tokens of a call
 *                 must not name one slot.
 *   d_q           device [T][ldq] of dtype, or NULL: q is not written.  It may
 *                 be the q columns of d_qkv themselves (in place: d_q = d_qkv +
 *                 offset[0], ldq = ldx) and must not overlap d_qkv otherwise.
 *   d_num_bad     device int32 or NULL: the number of bad tokens is added to it
 * A bad token (a slot outside [-1, num_pages * page_size), or with a rotation a
 * position outside [0, num_pos)) leaves q and the cache as they are.  E4M3
 * values are value / scale rounded to nearest even, beyond +-448 (infinities
 * too) +-448; NaN stays NaN.  fp32 values go to an fp32 cache, bf16 ones to a
 * bf16 or an e4m3 cache (else LORA_ERR_UNSUPPORTED). */
lora_status lora_cache_append(const void *d_qkv, int64_t ldx, int64_t num_tokens,
                              lora_dtype dtype, int32_t num_q_heads,
                              const int64_t *offset, const lora_rotation *rot,
                              const int32_t *d_pos, const int64_t *d_slot,
                              const lora_kv_cache *cache, void *d_q, int64_t ldq,
                              int32_t *d_num_bad, void *stream);

/* One step's batch of sequences, for lora_prepare_attn_meta.  Sequence n has
 * the query tokens [q_start[n], q_start[n + 1]) and kv_len[n] cached keys, those
 * of its query tokens included: query token i stands at position
 * p = kv_len[n] - q_len + i and sees the keys j in [lo, hi) with
 *     lo = max(0, window > 0 ? p + 1 - window : 0, key_lo ? key_lo[t] : 0)
 *     hi = min(kv_len[n], key_hi ? key_hi[t] : kv_len[n],
 *              max(causal ? p + 1 : kv_len[n], prefix_len ? prefix_len[n] : 0))
 * (key_lo and key_hi, per query token, bound a document; prefix_len, per
 * sequence, is a prefix that every token of it sees).  A token that sees no
 * key gets zeros, and -inf as the logarithm of its sum.
 *   d_q_start     device int32 [num_seqs + 1], non-decreasing, in [0, num_tokens]
 *   d_kv_len      device int32 [num_seqs]
 *   d_page_table  device int32 [num_seqs][page_table_stride]: the pages of each
 *                 sequence's keys in order; it has to stay valid, unchanged,
 *                 for every call that takes the metadata
 *   max_q_len     no sequence has more query tokens (else it is bad)
 *   groups        num_groups runs of consecutive sequences that share leading
 *                 keys: group g holds the sequences [d_group_start[g],
 *                 d_group_start[g + 1]) and its first d_group_len[g] keys are
 *                 the same for all of them.  They are read once for the whole
 *                 group, through the table of its first sequence.  num_groups
 *                 = 0: none.
 * A sequence is bad if its q_start leaves the bounds above, if it begins before the
 * end of an earlier good one, if it has more
 * query tokens than max_q_len or than keys, or if its keys do not fit
 * page_table_stride pages; its tokens see no key.  Tokens that a good sequence holds
 * too are that one's.  Supported: num_tokens <=
 * 2^24, num_tokens * num_q_heads < 2^31, num_seqs <= 2^20, num_q_heads <= 1024, page_table_stride * page_size <=
 * 2^31 - 2^16.  A group is bad, and ignored,
 * if its bounds are not ascending in [0, num_seqs], if it begins before the end of
 * an earlier good one, if its length is negative or
 * beyond the keys of its first sequence; all groups are where any bound of
 * q_start is out of order or leaves the batch.  The sequences of an ignored group
 * read all their keys through their own tables.  Keys in a page whose id lies outside
 * [0, num_pages) are not seen.  Bad sequences and groups are counted in info. */
typedef struct lora_attn_batch {
    const int32_t *d_q_start, *d_kv_len, *d_page_table;
    int64_t page_table_stride;
    int64_t num_tokens;
    int32_t num_seqs, max_q_len;
    int32_t num_q_heads;            /* a multiple of the cache's num_heads */
    int32_t causal, window;
    int32_t num_groups;
    const int32_t *d_prefix_len;    /* [num_seqs] or NULL */
    const int32_t *d_key_lo, *d_key_hi;   /* [num_tokens], both or neither */
    const int32_t *d_group_start, *d_group_len;
} lora_attn_batch;

/* Attention metadata of one step: which keys every token sees, and the work
 * list of the attention kernels.  Filled by lora_prepare_attn_meta with
 * pointers into the caller's workspace; shared, like a lora_meta, by every
 * layer of the step with this mask and cache geometry, and only read by them.
 *   limits        int32 [num_tokens][4]: lo, hi, p, sequence of every token (-1: in
 *                 none; -2: q_start is out of order, and only bad ones hold it)
 *   info          int32 [16]: slices of the few-row work, items of the tile
 *                 work, bad sequences, bad groups, tokens to join,
 *                 partial-result units, keys per slice, most keys per item of
 *                 the tile work, pieces of the slices, then zeros
 * The other arrays are work lists whose contents are internal. */
typedef struct lora_attn_meta {
    int64_t num_tokens, page_table_stride, max_units;
    int32_t num_seqs, num_q_heads, num_kv_heads, head_dim, page_size;
    int32_t dtype;                  /* the cache's */
    int32_t heads_per_item, head_groups;   /* query heads of one work item; items per key head */
    int32_t max_tiles, max_slots, max_tile_items;
    const int32_t *page_table;
    int32_t *limits, *info, *tiles, *few_items, *slots, *tile_items, *join, *join_list;
} lora_attn_meta;

/* Device workspace of lora_prepare_attn_meta for this batch and cache (sizes
 * only: no device array is read). */
lora_status lora_attn_meta_workspace_bytes(const lora_attn_batch *batch,
                                           const lora_kv_cache *cache, size_t *bytes);

/* Build the attention metadata of a step (two launches).  Of the cache only
 * num_heads, head_dim, page_size and dtype are read.  d_ws is 16-byte aligned. */
lora_status lora_prepare_attn_meta(const lora_attn_batch *batch,
                                   const lora_kv_cache *cache, void *d_ws,
                                   size_t ws_bytes, lora_attn_meta *out,
                                   void *stream);

/* Device workspace of lora_attention (partial results of split key ranges);
 * no initialisation is required. */
lora_status lora_attention_workspace_bytes(const lora_attn_meta *meta, size_t *bytes);

/* Attention of every query token over the cached keys it sees:
 *     x[j]      = cap(scale * q . k_j) - slope[h] * |p - j|
 *     cap(x)    = cap > 0 ? cap * tanh(x / cap) : x
 *     lse[t][h] = log sum_j exp(x[j]),   out[t][h] = sum_j exp(x[j] - lse) v_j
 * Query head h reads key head h / (num_q_heads / num_kv_heads).  Scores,
 * maxima, sums and products are kept in fp32; with a bf16 or e4m3 cache the
 * weights exp(.) go to the product with v in bf16, as the matrix cores take them:
 * as two terms (2^-16 of a weight is lost) for sequences of at most 16 rows, a
 * query token and one of the heads_per_item heads being a row, rounded once (2^-8)
 * for longer ones and for the shared keys of groups of more.
 *   d_q           device [T][ldq] (bf16, or fp32 with an fp32 cache): head h at
 *                 column h * head_dim
 *   d_out         device [T][ldo] of the same type, likewise; not overlapping q
 *   d_slopes      device fp32 [num_q_heads] or NULL (no bias)
 *   d_lse         device fp32 [T][num_q_heads] or NULL, contiguous
 * Tokens outside every sequence are not written.  A non-finite key or value
 * reaches the tokens that see it (a key possibly as NaN where its score is -inf) and
 * no others.  The query heads of a key head are taken in equal parts of at most 16,
 * and each part reads the keys: counts above 16 without a divisor near it (17, 71)
 * read them many times.  Calls that run at the same
 * time need workspaces of their own. */
lora_status lora_attention(const lora_attn_meta *meta, const void *d_q, int64_t ldq,
                           const lora_kv_cache *cache, float scale, float cap,
                           const float *d_slopes, void *d_out, int64_t ldo,
                           float *d_lse, void *d_ws, size_t ws_bytes, void *stream);

/* Human-readable name of a status code (static storage). */
const char *lora_status_string(lora_status status);

/* Library version, for the binding's sanity check. */
int32_t lora_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LORA_MI355X_H */
