"""Python binding of the MI355X multi-LoRA shrink/expand library.

Argument marshalling only: every step of the path runs in the HIP kernels of
``liblora_mi355x.so`` (C ABI in ``include/lora_mi355x.h``).  PyTorch provides
device memory and the current HIP stream.  The functions carry the names of the
C entry points.

There is no fallback: importing this package fails loudly when the built
library is missing (build it with ``python segmented_gather_rank_amd/build.py``
or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import contextlib
import ctypes as C
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# LORA_MI355X_LIB names another build of the same library (a measurement
# build, say); by default the in-tree one is loaded
LIB_PATH = os.environ.get("LORA_MI355X_LIB") or os.path.join(_HERE, "liblora_mi355x.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the HIP library first "
        "(python segmented_gather_rank_amd/build.py)")

_cdll = C.CDLL(LIB_PATH)

LORA_OK, LORA_ERR_INVALID_ARG, LORA_ERR_UNSUPPORTED, LORA_ERR_WORKSPACE, LORA_ERR_HIP = range(5)
LORA_F32, LORA_BF16, LORA_E4M3 = 0, 1, 2
MODES = {"auto": 0, "bgmv": 1, "sgmv": 2}


class LoraError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {lora_status_string(status)}")
        self.status = status


class lora_weight(C.Structure):
    _fields_ = [("ptr", C.c_void_p), ("slot_stride", C.c_int64), ("layout", C.c_int32), ("reserved", C.c_int32)]


LORA_LAYOUT_DEFAULT, LORA_LAYOUT_RANK_ROWS, LORA_LAYOUT_OUT_ROWS = 0, 1, 2


class lora_meta(C.Structure):
    _fields_ = [("num_tokens", C.c_int64), ("num_slots", C.c_int32), ("x_row_div", C.c_int32),
                ("sorted", C.c_void_p), ("sorted_slot", C.c_void_p), ("seg_slot", C.c_void_p),
                ("seg_count", C.c_void_p),
                ("seg_start", C.c_void_p), ("info", C.c_void_p), ("tiles", C.c_void_p)]


class lora_kv_cache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("page_stride", C.c_int64), ("head_stride", C.c_int64),
                ("pos_stride", C.c_int64), ("num_pages", C.c_int64), ("page_size", C.c_int32),
                ("num_heads", C.c_int32), ("head_dim", C.c_int32), ("dtype", C.c_int32),
                ("k_scale", C.c_void_p), ("v_scale", C.c_void_p)]


class lora_rotation(C.Structure):
    _fields_ = [("table", C.c_void_p), ("num_pos", C.c_int64), ("rot_dim", C.c_int32), ("interleaved", C.c_int32),
                ("num_axes", C.c_int32), ("section", C.c_int32 * 4), ("reserved", C.c_int32)]


class lora_attn_batch(C.Structure):
    _fields_ = [("d_q_start", C.c_void_p), ("d_kv_len", C.c_void_p), ("d_page_table", C.c_void_p),
                ("page_table_stride", C.c_int64), ("num_tokens", C.c_int64), ("num_seqs", C.c_int32),
                ("max_q_len", C.c_int32), ("num_q_heads", C.c_int32), ("causal", C.c_int32),
                ("window", C.c_int32), ("num_groups", C.c_int32), ("d_prefix_len", C.c_void_p),
                ("d_key_lo", C.c_void_p), ("d_key_hi", C.c_void_p), ("d_group_start", C.c_void_p),
                ("d_group_len", C.c_void_p)]


class lora_attn_meta(C.Structure):
    _fields_ = [("num_tokens", C.c_int64), ("page_table_stride", C.c_int64), ("max_units", C.c_int64),
                ("num_seqs", C.c_int32), ("num_q_heads", C.c_int32), ("num_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("page_size", C.c_int32), ("dtype", C.c_int32),
                ("heads_per_item", C.c_int32), ("head_groups", C.c_int32), ("max_tiles", C.c_int32),
                ("max_slots", C.c_int32), ("max_tile_items", C.c_int32), ("page_table", C.c_void_p),
                ("limits", C.c_void_p), ("info", C.c_void_p), ("tiles", C.c_void_p), ("few_items", C.c_void_p), ("slots", C.c_void_p),
                ("tile_items", C.c_void_p), ("join", C.c_void_p), ("join_list", C.c_void_p)]


class lora_routing(C.Structure):
    _fields_ = [("num_experts", C.c_int32), ("topk", C.c_int32), ("score", C.c_int32), ("num_groups", C.c_int32),
                ("topk_groups", C.c_int32), ("group_top", C.c_int32), ("renormalize", C.c_int32), ("scale", C.c_float),
                ("d_bias", C.c_void_p)]


class lora_int8_weight(C.Structure):
    _fields_ = [("ptr", C.c_void_p), ("expert_stride", C.c_int64), ("row_stride", C.c_int64), ("scale", C.c_void_p),
                ("bias", C.c_void_p), ("d_in", C.c_int64), ("d_out", C.c_int64), ("num_experts", C.c_int32),
                ("reserved", C.c_int32)]


_p, _i32, _i64, _sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
_decl = {
    "lora_abi_version": ([], _i32),
    "lora_status_string": ([_i32], C.c_char_p),
    "lora_meta_workspace_bytes": ([_i64, _i32, C.POINTER(_sz)], _i32),
    "lora_prepare_meta": ([_p, _i64, _i32, _p, _sz, C.POINTER(lora_meta), _p], _i32),
    "lora_moe_meta_workspace_bytes": ([_i64, _i32, _i32, _i32, C.POINTER(_sz)], _i32),
    "lora_prepare_moe_meta": ([_p, _i64, _i32, _p, _i32, _i32, _i32, _p, _p, _sz, C.POINTER(lora_meta), _p],
                              _i32),
    "lora_shrink_workspace_bytes": ([_i64, _i32, _i64, _i32, _i32, _i32, _i32, C.POINTER(_sz)], _i32),
    "lora_shrink": ([C.POINTER(lora_meta), _p, _i64, _i64, _i32, _i32, C.POINTER(lora_weight), _i32,
                     C.c_float, _p, _p, _p, _i32, _p, _sz, _p], _i32),
    "lora_expand": ([C.POINTER(lora_meta), _p, _i32, C.POINTER(lora_weight), C.POINTER(_i64),
                     C.POINTER(_i64), _i32, _p, _p, _i64, _i32, C.c_int, _i32, _p], _i32),
    "lora_apply_workspace_bytes": ([_i64, _i32, _i64, _i32, _i32, _i32, _i32, C.POINTER(_sz)], _i32),
    "lora_apply_workspace_init": ([_p, _sz, _p], _i32),
    "lora_apply_noalloc": ([C.POINTER(lora_meta), _p, _i64, _i64, _i32, _i32, C.POINTER(lora_weight),
                            C.POINTER(lora_weight), C.POINTER(_i64), C.POINTER(_i64), _i32, C.c_float, _p,
                            _p, _p, _i64, C.c_int, _i32, _p], _i32),
    "lora_apply": ([C.POINTER(lora_meta), _p, _i64, _i64, _i32, _i32, C.POINTER(lora_weight),
                    C.POINTER(lora_weight), C.POINTER(_i64), C.POINTER(_i64), _i32, C.c_float, _p,
                    _p, _p, _i64, C.c_int, _i32, _p, _sz, _p], _i32),
    "lora_cache_append": ([_p, _i64, _i64, _i32, _i32, C.POINTER(_i64), C.POINTER(lora_rotation), _p, _p,
                           C.POINTER(lora_kv_cache), _p, _i64, _p, _p], _i32),
    "lora_attn_meta_workspace_bytes": ([C.POINTER(lora_attn_batch), C.POINTER(lora_kv_cache), C.POINTER(_sz)],
                                       _i32),
    "lora_prepare_attn_meta": ([C.POINTER(lora_attn_batch), C.POINTER(lora_kv_cache), _p, _sz,
                                C.POINTER(lora_attn_meta), _p], _i32),
    "lora_attention_workspace_bytes": ([C.POINTER(lora_attn_meta), C.POINTER(_sz)], _i32),
    "lora_attention": ([C.POINTER(lora_attn_meta), _p, _i64, C.POINTER(lora_kv_cache), C.c_float, C.c_float, _p,
                        _p, _i64, _p, _p, _sz, _p], _i32),
    "lora_moe_route": ([C.POINTER(lora_routing), _p, _i64, _i64, _i32, _p, _p, _p], _i32),
    "lora_quantize": ([_p, _i64, _i64, _i64, _i32, _i32, C.POINTER(lora_meta), _p, _i64, _p, _p, _i64, _p], _i32),
    "lora_int8_matmul_workspace_bytes": ([_i64, C.POINTER(lora_int8_weight), C.POINTER(_sz)], _i32),
    "lora_int8_matmul": ([C.POINTER(lora_meta), _p, _i64, _p, _i64, C.POINTER(lora_int8_weight), _p, _i64, _i32, _p,
                          _sz, _p], _i32),
    "lora_moe_combine": ([_p, _i64, _i64, _i32, _p, _p, _i64, _i32, _i32, _i32, _p, _p, _i64, _p, _i64, _p], _i32),
}



class _Exact:
    """A C function that takes exactly its declared arguments (ctypes itself
    would silently pass extra ones)."""

    def __init__(self, f):
        self.f, self.n = f, len(f.argtypes)

    def __call__(self, *args):
        if len(args) != self.n:
            raise TypeError(f"{self.f.__name__} takes {self.n} arguments, got {len(args)}")
        return self.f(*args)


class _Lib:
    def __init__(self, cdll, decl):
        for name, (args, res) in decl.items():
            f = getattr(cdll, name)
            f.argtypes, f.restype = args, res
            setattr(self, name, _Exact(f))


_lib = _Lib(_cdll, _decl)

if _lib.lora_abi_version() != 10:
    raise ImportError("liblora_mi355x.so has an unexpected ABI version; rebuild it")


def lora_abi_version() -> int:
    return int(_lib.lora_abi_version())


def lora_status_string(status: int) -> str:
    return _lib.lora_status_string(int(status)).decode()


def _check(fn: str, st: int) -> None:
    if st != LORA_OK:
        raise LoraError(fn, st)


def _stream(stream) -> C.c_void_p:
    return C.c_void_p(_stream_handle(stream))


def _stream_handle(stream) -> int:
    if stream is None:
        # the current stream's handle without building a Stream object (3 us)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on(stream, device):
    """Where memory for work on `stream` (None: the current one; a Stream or a raw
    handle) is allocated and cleared: on that stream, from its own pool.  Earlier work on
    another stream may still use what that one's pool gives out, and would get this back
    before the work here has ended."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream_handle(stream), device)
    return torch.cuda.stream(stream)


def _empty_for(stream, size, dtype, device) -> torch.Tensor:
    with _on(stream, device):
        return torch.empty(size, dtype=dtype, device=device)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LORA_F32
    if t.dtype == torch.bfloat16:
        return LORA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: float32 or bfloat16")


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.data_ptr()


def _weights(ws, name: str, inner_shape_ok, layout: int = 0) -> tuple:
    """Per-slice stacked factors [S][rows][cols] -> lora_weight array.  The
    matrices must be contiguous; the slot stride is taken from the tensor."""
    if isinstance(ws, torch.Tensor):
        ws = [ws]
    arr = (lora_weight * len(ws))()
    for i, w in enumerate(ws):
        if w.dim() != 3 or w.stride(2) != 1 or w.stride(1) != w.shape[2]:
            raise ValueError(f"{name}[{i}] must be [S][rows][cols] with contiguous matrices")
        inner_shape_ok(i, w)
        arr[i].ptr = _dev(w, f"{name}[{i}]")
        arr[i].slot_stride = w.stride(0)
        arr[i].layout = layout
    return arr, list(ws)


def _a_weights(A, a_rank_rows: bool):
    """A as [S][d_in][r] (default) or, with a_rank_rows, [S][r][d_in] (the
    rank-major layout); returns the descriptors, the tensors and r."""
    A_arr, A_list = _weights(A, "A", lambda i, w: None, LORA_LAYOUT_RANK_ROWS if a_rank_rows else LORA_LAYOUT_DEFAULT)
    return A_arr, A_list, A_list[0].shape[1] if a_rank_rows else A_list[0].shape[2]


TILE_ROWS = 64          # sorted positions per work tile of the metadata
TILE_INTS = 4 + TILE_ROWS
# the apply workspace's count words (LORA_APPLY_SYNC_BYTES and the two
# counter indices of the C header)
APPLY_SYNC_BYTES = 295168
WAITS_GAVE_UP_WORD = 73728
OTHER_XCD_WORD = 73729
SPLIT_MEMBERS = 16      # count words per work tile and slice range
SPLIT_RANGES = 4        # slice ranges per work tile


def max_tiles(num_tokens: int, num_slots: int) -> int:
    """Capacity of the metadata's work-tile list."""
    return (num_tokens + TILE_ROWS - 1) // TILE_ROWS + num_slots + 1


@dataclass
class LoraMeta:
    """Slot metadata of one batch on the device (see ``lora_meta`` in the C header).

    ``workspace`` owns the device arrays; keep this object alive while kernels
    that use it are in flight."""
    c: lora_meta
    workspace: torch.Tensor

    @property
    def num_tokens(self) -> int:
        return int(self.c.num_tokens)

    @property
    def num_slots(self) -> int:
        return int(self.c.num_slots)

    def _view(self, ptr, n):
        off = ptr - self.workspace.data_ptr()
        return self.workspace[off:off + 4 * n].view(torch.int32)

    def with_x_row_div(self, div: int) -> "LoraMeta":
        """The same metadata with another x row divisor (MoE: 1 for the
        down-projection LoRA, whose input has one row per pair)."""
        c = lora_meta()
        C.pointer(c)[0] = self.c
        c.x_row_div = int(div)
        return LoraMeta(c, self.workspace)

    def tensors(self) -> dict:
        """Device int32 views of the metadata arrays."""
        T, S = self.num_tokens, self.num_slots
        return dict(sorted=self._view(self.c.sorted, T), sorted_slot=self._view(self.c.sorted_slot, T),
                    seg_slot=self._view(self.c.seg_slot, S + 1),
                    seg_count=self._view(self.c.seg_count, S + 1),
                    seg_start=self._view(self.c.seg_start, S + 2), info=self._view(self.c.info, 8),
                    tiles=self._view(self.c.tiles, TILE_INTS * max_tiles(T, S)).view(-1, TILE_INTS))


def lora_meta_workspace_bytes(num_tokens: int, num_slots: int) -> int:
    b = _sz(0)
    _check("lora_meta_workspace_bytes", _lib.lora_meta_workspace_bytes(num_tokens, num_slots, C.byref(b)))
    return int(b.value)


def lora_prepare_meta(token_slot: torch.Tensor, num_slots: int, workspace: torch.Tensor | None = None,
                      stream=None) -> LoraMeta:
    if token_slot.dtype != torch.int32 or token_slot.dim() != 1 or not token_slot.is_contiguous():
        raise ValueError("token_slot must be a contiguous int32 vector")
    T = token_slot.shape[0]
    need = lora_meta_workspace_bytes(T, num_slots)
    if workspace is None:
        workspace = _empty_for(stream, need, torch.uint8, token_slot.device)
    m = lora_meta()
    st = _lib.lora_prepare_meta(_dev(token_slot, "token_slot") if T else None, T, num_slots,
                                _dev(workspace, "workspace"), workspace.numel(), C.byref(m), _stream(stream))
    _check("lora_prepare_meta", st)
    return LoraMeta(m, workspace)


def lora_moe_meta_workspace_bytes(num_tokens: int, topk: int, num_slots: int, num_local_experts: int) -> int:
    b = _sz(0)
    _check("lora_moe_meta_workspace_bytes",
           _lib.lora_moe_meta_workspace_bytes(num_tokens, topk, num_slots, num_local_experts, C.byref(b)))
    return int(b.value)


def lora_prepare_moe_meta(topk_ids: torch.Tensor, token_slot: torch.Tensor, num_slots: int, num_experts: int,
                          num_local_experts: int, expert_map: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None) -> LoraMeta:
    """Metadata over the (token, choice) pairs of a top-k routing step, keyed by
    (slot, local expert); topk_ids int32 [T][topk], token_slot int32 [T],
    expert_map int32 [num_experts] or None."""
    for name, t in (("topk_ids", topk_ids), ("token_slot", token_slot)):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous int32")
    if topk_ids.dim() != 2 or token_slot.dim() != 1 or topk_ids.shape[0] != token_slot.shape[0]:
        raise ValueError("topk_ids must be [T][topk] and token_slot [T]")
    T, K = topk_ids.shape
    need = lora_moe_meta_workspace_bytes(T, K, num_slots, num_local_experts)
    if workspace is None:
        workspace = _empty_for(stream, need, torch.uint8, topk_ids.device)
    em = None
    if expert_map is not None:
        if expert_map.dtype != torch.int32 or expert_map.numel() != num_experts:
            raise ValueError("expert_map must be int32 [num_experts]")
        em = _dev(expert_map, "expert_map")
    m = lora_meta()
    st = _lib.lora_prepare_moe_meta(_dev(topk_ids, "topk_ids") if T else None, T, K,
                                    _dev(token_slot, "token_slot") if T else None, num_slots, num_experts,
                                    num_local_experts, em, _dev(workspace, "workspace"), workspace.numel(),
                                    C.byref(m), _stream(stream))
    _check("lora_prepare_moe_meta", st)
    return LoraMeta(m, workspace)


def lora_shrink_workspace_bytes(num_tokens, num_slots, d_in, n_slices, r_max, dtype, mode="auto") -> int:
    b = _sz(0)
    dt = dtype if isinstance(dtype, int) else _dtype(torch.empty(0, dtype=dtype))
    _check("lora_shrink_workspace_bytes",
           _lib.lora_shrink_workspace_bytes(num_tokens, num_slots, d_in, n_slices, r_max, dt,
                                            MODES[mode], C.byref(b)))
    return int(b.value)


def lora_apply_workspace_bytes(num_tokens, num_slots, d_in, n_slices, r_max, dtype, mode="auto") -> int:
    b = _sz(0)
    dt = dtype if isinstance(dtype, int) else _dtype(torch.empty(0, dtype=dtype))
    _check("lora_apply_workspace_bytes",
           _lib.lora_apply_workspace_bytes(num_tokens, num_slots, d_in, n_slices, r_max, dt,
                                           MODES[mode], C.byref(b)))
    return int(b.value)


def lora_apply_workspace_init(workspace: torch.Tensor, stream=None) -> torch.Tensor:
    """Zero the count words at the start of an apply workspace (once,
    before its first lora_apply)."""
    _check("lora_apply_workspace_init",
           _lib.lora_apply_workspace_init(_dev(workspace, "workspace"), workspace.numel(), _stream(stream)))
    return workspace


def apply_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A zero-filled apply workspace of at least nbytes (and at least the
    count words), ready for lora_apply."""
    return torch.zeros(max(int(nbytes), APPLY_SYNC_BYTES), dtype=torch.uint8, device=device)


def apply_workspace_counters(workspace: torch.Tensor) -> dict:
    """The decode-shaped apply's counters in a workspace: waits that gave up
    and waits that met a peer on another XCD (0 and 0 in normal runs; either
    case is still computed right).  Synchronises with the device."""
    w = workspace[:APPLY_SYNC_BYTES].view(torch.int32)
    v = w[WAITS_GAVE_UP_WORD:OTHER_XCD_WORD + 1].cpu().tolist()
    return {"gave_up": int(v[0]) & 0xFFFFFFFF, "other_xcd": int(v[1]) & 0xFFFFFFFF}


def apply_workspace_flags(workspace: torch.Tensor, tiles: int) -> torch.Tensor:
    """The count words of the first `tiles` work tiles, [tile][range][member]
    (int32 view of uint32 words: the call count in bits 31:17, the tile in
    16:6, the range in 5:4, an XCD in 3:0)."""
    w = workspace[:APPLY_SYNC_BYTES].view(torch.int32)
    return w[:tiles * SPLIT_RANGES * SPLIT_MEMBERS].view(tiles, SPLIT_RANGES, SPLIT_MEMBERS)


def _x_args(x: torch.Tensor):
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be [T][ldx] with unit column stride")
    return _dev(x, "x"), x.stride(0), x.shape[1]


def _ranks(slot_rank):
    if slot_rank is None:
        return None
    if slot_rank.dtype != torch.int32:
        raise TypeError("slot_rank must be int32")
    return _dev(slot_rank, "slot_rank")


def lora_shrink(meta: LoraMeta, x: torch.Tensor, A, u: torch.Tensor, scale: float = 1.0,
                slot_scale: torch.Tensor | None = None, mode: str = "auto",
                workspace: torch.Tensor | None = None, stream=None,
                slot_rank: torch.Tensor | None = None, a_rank_rows: bool = False) -> torch.Tensor:
    """u[s][t][:] = scale * slot_scale[slot] * x[t] @ A[s][slot]; A: list of [S][d_in][r]
    (or [S][r][d_in] with a_rank_rows).  slot_rank: optional int32 [S], ranks
    each slot's adapter really has."""
    xp, ldx, d_in = _x_args(x)
    A_arr, A_list, r = _a_weights(A, a_rank_rows)
    n = len(A_list)
    need = lora_shrink_workspace_bytes(meta.num_tokens, meta.num_slots, d_in, n, r, x.dtype, mode)
    if workspace is None:
        workspace = _empty_for(stream, max(need, 16), torch.uint8, x.device)
    ss = None if slot_scale is None else _dev(slot_scale, "slot_scale")
    st = _lib.lora_shrink(C.byref(meta.c), xp, ldx, d_in, _dtype(x), n, A_arr, r, float(scale), ss,
                          _ranks(slot_rank), _dev(u, "u"), MODES[mode], _dev(workspace, "workspace"),
                          workspace.numel(), _stream(stream))
    _check("lora_shrink", st)
    return u


def _b_weights(B, b_out_rows: bool):
    """B as [S][r][w] (default) or, with b_out_rows, [S][w][r] (one row of
    ranks per output column); returns the descriptors, the tensors and r."""
    B_arr, B_list = _weights(B, "B", lambda i, w: None, LORA_LAYOUT_OUT_ROWS if b_out_rows else LORA_LAYOUT_DEFAULT)
    return B_arr, B_list, B_list[0].shape[2] if b_out_rows else B_list[0].shape[1]


def _slices(B_list, offsets, b_out_rows: bool = False):
    n = len(B_list)
    width = (C.c_int64 * n)(*[b.shape[1] if b_out_rows else b.shape[2] for b in B_list])
    offs = (C.c_int64 * n)(*[int(o) for o in offsets])
    return width, offs


def lora_expand(meta: LoraMeta, u: torch.Tensor, B, offsets, y: torch.Tensor, add: bool = True,
                mode: str = "auto", stream=None, slot_rank: torch.Tensor | None = None,
                b_out_rows: bool = False) -> torch.Tensor:
    """y[t][off_s:off_s+w_s] (+)= u[s][t] @ B[s][slot]; B: list of [S][r][w_s]
    (or [S][w_s][r] with b_out_rows)."""
    B_arr, B_list, rb = _b_weights(B, b_out_rows)
    width, offs = _slices(B_list, offsets, b_out_rows)
    if y.dim() != 2 or y.stride(1) != 1:
        raise ValueError("y must be [T][ldy] with unit column stride")
    st = _lib.lora_expand(C.byref(meta.c), _dev(u, "u"), len(B_list), B_arr, width, offs,
                          rb, _ranks(slot_rank), _dev(y, "y"), y.stride(0), _dtype(y),
                          int(bool(add)), MODES[mode], _stream(stream))
    _check("lora_expand", st)
    return y


def lora_apply(meta: LoraMeta, x: torch.Tensor, A, B, offsets, y: torch.Tensor, scale: float = 1.0,
               slot_scale: torch.Tensor | None = None, add: bool = True, mode: str = "auto",
               workspace: torch.Tensor | None = None, stream=None,
               slot_rank: torch.Tensor | None = None, a_rank_rows: bool = False,
               b_out_rows: bool = False) -> torch.Tensor:
    """Shrink then expand into the slices of y (the whole delta of one layer).
    A: list of [S][d_in][r], or [S][r][d_in] with a_rank_rows; B: list of
    [S][r][w_s], or [S][w_s][r] with b_out_rows."""
    xp, ldx, d_in = _x_args(x)
    A_arr, A_list, r = _a_weights(A, a_rank_rows)
    B_arr, B_list, _ = _b_weights(B, b_out_rows)
    width, offs = _slices(B_list, offsets, b_out_rows)
    n = len(A_list)
    if len(B_list) != n:
        raise ValueError("A and B need one entry per slice")
    need = lora_apply_workspace_bytes(meta.num_tokens, meta.num_slots, d_in, n, r, x.dtype, mode)
    if workspace is None:
        with _on(stream, x.device):
            workspace = apply_workspace(need, x.device)
    if y.dim() != 2 or y.stride(1) != 1:
        raise ValueError("y must be [T][ldy] with unit column stride")
    ss = None if slot_scale is None else _dev(slot_scale, "slot_scale")
    if y.dtype != x.dtype:
        raise TypeError("x and y must share one dtype")
    st = _lib.lora_apply(C.byref(meta.c), xp, ldx, d_in, _dtype(x), n, A_arr, B_arr, width, offs, r,
                         float(scale), ss, _ranks(slot_rank), _dev(y, "y"), y.stride(0), int(bool(add)),
                         MODES[mode], _dev(workspace, "workspace"), workspace.numel(), _stream(stream))
    _check("lora_apply", st)
    return y


NOALLOC_SCRATCH_BYTES = 64 << 20   # LORA_NOALLOC_SCRATCH_BYTES of the C header


def lora_apply_noalloc(meta: LoraMeta, x: torch.Tensor, A, B, offsets, y: torch.Tensor, scale: float = 1.0,
                       slot_scale: torch.Tensor | None = None, add: bool = True, mode: str = "auto", stream=None,
                       slot_rank: torch.Tensor | None = None, a_rank_rows: bool = False,
                       b_out_rows: bool = False) -> torch.Tensor:
    """lora_apply with the library's own device scratch as its workspace (no
    workspace argument, nothing allocated).  Calls that overlap on one device
    share that scratch and race."""
    xp, ldx, d_in = _x_args(x)
    A_arr, A_list, r = _a_weights(A, a_rank_rows)
    B_arr, B_list, _ = _b_weights(B, b_out_rows)
    width, offs = _slices(B_list, offsets, b_out_rows)
    if len(B_list) != len(A_list):
        raise ValueError("A and B need one entry per slice")
    if y.dim() != 2 or y.stride(1) != 1:
        raise ValueError("y must be [T][ldy] with unit column stride")
    if y.dtype != x.dtype:
        raise TypeError("x and y must share one dtype")
    ss = None if slot_scale is None else _dev(slot_scale, "slot_scale")
    st = _lib.lora_apply_noalloc(C.byref(meta.c), xp, ldx, d_in, _dtype(x), len(A_list), A_arr, B_arr, width,
                                 offs, r, float(scale), ss, _ranks(slot_rank), _dev(y, "y"),
                                 y.stride(0), int(bool(add)), MODES[mode], _stream(stream))
    _check("lora_apply_noalloc", st)
    return y


class KvCache:
    """A paged key/value cache: k and v indexed [page][head][position][dim],
    views of any strides with contiguous dims (a [page][position][head][dim]
    cache is passed as its transpose(1, 2)); float32, bfloat16 or float8_e4m3fn.
    k_scale and v_scale: float32 [heads], for float8_e4m3fn only."""

    _types = {torch.float32: LORA_F32, torch.bfloat16: LORA_BF16, torch.float8_e4m3fn: LORA_E4M3}

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride():
            raise ValueError("k and v must be [page][head][position][dim] of one shape, dtype and stride")
        if k.stride(3) != 1:
            raise ValueError("the dims of a head must be contiguous")
        if k.dtype not in self._types:
            raise TypeError(f"unsupported cache dtype {k.dtype}")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None and (t.dtype != torch.float32 or t.shape != (k.shape[1],) or not t.is_contiguous()):
                raise ValueError(f"{name} must be float32 [heads]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.num_heads, self.page_size, self.head_dim = k.shape
        # queries (and appended rows) that go with this cache
        self.query_dtype = torch.float32 if k.dtype == torch.float32 else torch.bfloat16
        self.c = lora_kv_cache(_dev(k, "k"), _dev(v, "v"), k.stride(0), k.stride(1), k.stride(2), self.num_pages,
                               self.page_size, self.num_heads, self.head_dim, self._types[k.dtype],
                               None if k_scale is None else _dev(k_scale, "k_scale"),
                               None if v_scale is None else _dev(v_scale, "v_scale"))
        self.ref = C.byref(self.c)
        self._packed = {}

    def packed_offsets(self, num_q_heads: int):
        """Columns of q, k and v in a row that holds nothing else, and its width."""
        if num_q_heads not in self._packed:
            k = num_q_heads * self.head_dim
            v = k + self.num_heads * self.head_dim
            self._packed[num_q_heads] = (C.c_int64 * 3)(0, k, v), v + self.num_heads * self.head_dim
        return self._packed[num_q_heads]


class Rotation:
    """Rotary positions: table float32 [num_pos][rot_dim], cosines then sines of
    the rot_dim / 2 pairs; sections: pairs per axis (one entry or none: one axis)."""

    def __init__(self, table: torch.Tensor, sections=None, interleaved: bool = False):
        if table.dim() != 2 or table.dtype != torch.float32 or not table.is_contiguous():
            raise ValueError("table must be contiguous float32 [num_pos][rot_dim]")
        sections = [table.shape[1] // 2] if not sections else [int(n) for n in sections]
        if len(sections) > 4:
            raise ValueError("at most 4 axes")
        self.table, self.num_axes = table, len(sections)
        self.c = lora_rotation(_dev(table, "table"), table.shape[0], table.shape[1], int(bool(interleaved)),
                               len(sections), (C.c_int32 * 4)(*sections), 0)
        self.ref = C.byref(self.c)


def lora_cache_append(qkv: torch.Tensor, cache: KvCache, slot: torch.Tensor, q_out: torch.Tensor | None = None,
                      pos: torch.Tensor | None = None, rotation: Rotation | None = None, num_q_heads: int | None = None,
                      offsets=None, num_bad: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Rotate q and k of the packed rows qkv [T][ldx] and write q to q_out [T][ldq]
    and k, v to their slots (int64 [T], page * page_size + position, -1: not
    kept) of the cache.  pos: int32 [T] or [axes][T].  offsets: columns of q, k
    and v (default: q | k | v without gaps, num_q_heads from q_out's width or
    from the row's)."""
    if qkv.dim() != 2 or qkv.stride(1) != 1:
        raise ValueError("qkv must be [T][ldx] with unit column stride")
    if slot.dtype != torch.int64 or slot.dim() != 1 or not slot.is_contiguous() or slot.shape[0] != qkv.shape[0]:
        raise ValueError("slot must be a contiguous int64 vector, one entry per row")
    T, width = qkv.shape
    D, kvh = cache.head_dim, cache.num_heads
    if num_q_heads is None:
        num_q_heads = (q_out.shape[1] if q_out is not None else width - 2 * kvh * D) // D
    if offsets is None:
        offs, need = cache.packed_offsets(num_q_heads)
    else:
        offs = (C.c_int64 * 3)(*offsets)
        need = max(offs[0] + num_q_heads * D, offs[1] + kvh * D, offs[2] + kvh * D)
    if width < need:
        raise ValueError("qkv has fewer columns than its heads need")
    q_ptr, ldq = None, 0
    if q_out is not None:
        if q_out.dim() != 2 or q_out.stride(1) != 1 or q_out.shape[0] != T or q_out.dtype != qkv.dtype:
            raise ValueError("q_out must be [T][ldq] of qkv's dtype with unit column stride")
        if q_out.shape[1] < num_q_heads * D:
            raise ValueError("q_out has fewer columns than its heads need")
        q_ptr, ldq = _dev(q_out, "q_out") if T else None, q_out.stride(0) if T > 1 else q_out.shape[1]
    rot = pos_ptr = None
    if rotation is not None:
        axes = rotation.num_axes
        if pos is None or pos.dtype != torch.int32 or not pos.is_contiguous() or pos.numel() != axes * T or (
                axes > 1 and pos.dim() > 1 and pos.shape != (axes, T)):
            raise ValueError("pos must be contiguous int32 [axes][T]")
        rot, pos_ptr = rotation.ref, _dev(pos, "pos") if T else None
    if num_bad is not None and num_bad.dtype != torch.int32:
        raise ValueError("num_bad must be int32")
    st = _lib.lora_cache_append(
        _dev(qkv, "qkv") if T else None, qkv.stride(0) if T > 1 else width, T, _dtype(qkv), num_q_heads, offs, rot,
        pos_ptr, _dev(slot, "slot") if T else None, cache.ref, q_ptr, ldq,
        None if num_bad is None else _dev(num_bad, "num_bad"), _stream_handle(stream))
    _check("lora_cache_append", st)
    return q_out


class AttnMeta:
    """Attention metadata of one step (see ``lora_attn_meta`` in the C header).
    ``workspace`` owns the device arrays and ``page_table`` is read by every
    call; keep this object alive while kernels that use it are in flight."""

    def __init__(self, c: lora_attn_meta, workspace: torch.Tensor, page_table: torch.Tensor):
        self.c, self.workspace, self.page_table = c, workspace, page_table
        self.ref = C.byref(c)
        b = _sz(0)
        _check("lora_attention_workspace_bytes", _lib.lora_attention_workspace_bytes(self.ref, C.byref(b)))
        self.attention_bytes = int(b.value)

    def tensors(self) -> dict:
        """Device int32 views of the documented arrays."""
        def view(ptr, n):
            off = ptr - self.workspace.data_ptr()
            return self.workspace[off:off + 4 * n].view(torch.int32)
        return dict(info=view(self.c.info, 16), limits=view(self.c.limits, 4 * self.c.num_tokens).view(-1, 4))


def _attn_batch(q_start, kv_len, page_table, num_q_heads, num_tokens, max_q_len, causal, window, prefix_len, key_lo,
                key_hi, group_start, group_len) -> lora_attn_batch:
    N = kv_len.shape[0]
    vectors = {"q_start": (q_start, N + 1), "kv_len": (kv_len, N), "prefix_len": (prefix_len, N),
               "key_lo": (key_lo, num_tokens), "key_hi": (key_hi, num_tokens)}
    if (group_start is None) != (group_len is None):
        raise ValueError("group_start and group_len go together")
    groups = 0 if group_len is None else group_len.shape[0]
    if groups:
        vectors.update(group_start=(group_start, groups + 1), group_len=(group_len, groups))
    ptr = {}
    for name, (t, n) in vectors.items():
        if t is None:
            ptr[name] = None
            continue
        if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.shape[0] != n:
            raise ValueError(f"{name} must be a contiguous int32 vector of {n}")
        ptr[name] = _dev(t, name)
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != N or (
            page_table.shape[1] and page_table.stride(1) != 1):
        raise ValueError("page_table must be int32 [sequences][pages] with contiguous rows")
    if N > 1 and page_table.stride(0) != page_table.shape[1]:
        raise ValueError("page_table must be contiguous")
    return lora_attn_batch(ptr["q_start"], ptr["kv_len"], _dev(page_table, "page_table"), page_table.shape[1],
                           num_tokens, N, num_tokens if max_q_len is None else max_q_len, num_q_heads,
                           int(bool(causal)), int(window), groups, ptr["prefix_len"], ptr["key_lo"], ptr["key_hi"],
                           ptr.get("group_start"), ptr.get("group_len"))


def lora_prepare_attn_meta(q_start: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor, cache: KvCache,
                           num_q_heads: int, num_tokens: int, max_q_len: int | None = None, causal: bool = True,
                           window: int = 0, prefix_len: torch.Tensor | None = None,
                           key_lo: torch.Tensor | None = None, key_hi: torch.Tensor | None = None,
                           group_start: torch.Tensor | None = None, group_len: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, stream=None) -> AttnMeta:
    """Attention metadata of a batch: q_start int32 [N + 1], kv_len int32 [N],
    page_table int32 [N][pages]; the masks and groups of ``lora_attn_batch``.
    max_q_len: the most query tokens of a sequence (default num_tokens); a batch
    that states it has few, as in decode, has no tile work to launch."""
    b = _attn_batch(q_start, kv_len, page_table, num_q_heads, num_tokens, max_q_len, causal, window, prefix_len,
                    key_lo, key_hi, group_start, group_len)
    need = _sz(0)
    _check("lora_attn_meta_workspace_bytes", _lib.lora_attn_meta_workspace_bytes(C.byref(b), cache.ref, C.byref(need)))
    if workspace is None:
        workspace = _empty_for(stream, int(need.value), torch.uint8, kv_len.device)
    m = lora_attn_meta()
    st = _lib.lora_prepare_attn_meta(C.byref(b), cache.ref, _dev(workspace, "workspace"), workspace.numel(),
                                     C.byref(m), _stream(stream))
    _check("lora_prepare_attn_meta", st)
    return AttnMeta(m, workspace, page_table)


def lora_attn_meta_workspace_bytes(q_start, kv_len, page_table, cache: KvCache, num_q_heads: int, num_tokens: int,
                                   num_groups: int = 0, max_q_len: int | None = None) -> int:
    """Bytes of lora_prepare_attn_meta's workspace for a batch of these sizes;
    max_q_len as given there, or None: enough for any."""
    most = 0
    for q_len in (0, num_tokens) if max_q_len is None else (max_q_len,):
        b = lora_attn_batch(page_table_stride=page_table.shape[1], num_tokens=num_tokens, num_seqs=kv_len.shape[0],
                            max_q_len=q_len, num_q_heads=num_q_heads, num_groups=num_groups)
        need = _sz(0)
        _check("lora_attn_meta_workspace_bytes",
               _lib.lora_attn_meta_workspace_bytes(C.byref(b), cache.ref, C.byref(need)))
        most = max(most, int(need.value))
    return most


def lora_attention_workspace_bytes(meta: AttnMeta) -> int:
    return meta.attention_bytes


def lora_attention(meta: AttnMeta, q: torch.Tensor, cache: KvCache, out: torch.Tensor | None = None,
                   scale: float | None = None, cap: float = 0.0, slopes: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Attention of q [T][heads][dim] (or [T][heads * dim]) over the cached keys
    that meta says it sees; returns out, or (out, lse) when lse (float32
    [T][heads]) is given.  scale: default 1 / sqrt(dim); cap: tanh cap of the
    scores (0: none); slopes: float32 [heads], bias per unit of distance.  An out
    or workspace that is not given is allocated on the stream of the call."""
    c = meta.c
    if out is None:
        out = _empty_for(stream, q.shape, q.dtype, q.device)
    width = c.num_q_heads * c.head_dim
    for name, t in (("q", q), ("out", out)):
        rows = t.shape[0] == c.num_tokens and t.dtype == cache.query_dtype and t.stride(-1) == 1
        if not rows or (t.dim() == 2 and t.shape[1] != width) or t.dim() not in (2, 3) or (
                t.dim() == 3 and (t.shape[1:] != (c.num_q_heads, c.head_dim) or t.stride(1) != c.head_dim)):
            raise ValueError(f"{name} must be [T][heads][dim] or [T][heads * dim] of {cache.query_dtype}, heads contiguous")
    if slopes is not None and (slopes.dtype != torch.float32 or slopes.shape != (c.num_q_heads,) or not slopes.is_contiguous()):
        raise ValueError("slopes must be float32 [heads]")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (c.num_tokens, c.num_q_heads) or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous float32 [T][heads]")
    if workspace is None:
        workspace = _empty_for(stream, meta.attention_bytes, torch.uint8, q.device)
    st = _lib.lora_attention(
        meta.ref, _dev(q, "q"), q.stride(0) if c.num_tokens > 1 else width, cache.ref,
        c.head_dim ** -0.5 if scale is None else scale, cap, None if slopes is None else _dev(slopes, "slopes"),
        _dev(out, "out"), out.stride(0) if c.num_tokens > 1 else width, None if lse is None else _dev(lse, "lse"),
        _dev(workspace, "workspace"), workspace.numel(), _stream_handle(stream))
    _check("lora_attention", st)
    return out if lse is None else (out, lse)


SCORES = {"softmax": 0, "sigmoid": 1}
ACTIVATIONS = {None: 0, "silu_mul": 1}


def _apart(device: int, *tensors) -> None:
    """Refuses tensors that do not lie on the device of that index."""
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensors on {t.device} and on device {device}")


def _elsewhere(device: int) -> bool:
    """Whether a call's tensors lie on another device than the current one, to which launches go."""
    return device >= 0 and device != torch._C._cuda_getDevice()


def _rows(t: torch.Tensor, name: str, dtype, rows: int, cols: int) -> tuple:
    """Address and row stride of a matrix of rows x cols."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] != cols or t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype} of {rows} x {cols}, not {t.dtype} of {tuple(shape)}")
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    # the stride of a single row says nothing
    return (_dev(t, name) if rows and cols else None), (ld if rows > 1 else cols)


def _vector(t: torch.Tensor, name: str, dtype, shape) -> int | None:
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} of {tuple(shape)}, not {t.dtype} of {tuple(t.shape)}")
    return _dev(t, name)


class Routing:
    """How a router's logits become expert choices (see ``lora_routing`` in the C
    header).  bias: float32 [experts], decides but does not weigh."""

    def __init__(self, num_experts: int, topk: int, score: str = "softmax", bias: torch.Tensor | None = None,
                 num_groups: int = 1, topk_groups: int = 1, group_top: int = 2, renormalize: bool = True,
                 scale: float = 1.0):
        if score not in SCORES:
            raise ValueError(f"score must be one of {sorted(SCORES)}")
        self.num_experts, self.topk, self.bias = int(num_experts), int(topk), bias
        self.c = lora_routing(self.num_experts, self.topk, SCORES[score], num_groups, topk_groups, group_top,
                              int(bool(renormalize)), float(scale),
                              None if bias is None else _vector(bias, "bias", torch.float32, (self.num_experts,)))
        self.ref = C.byref(self.c)


def lora_moe_route(logits: torch.Tensor, routing: Routing, topk_ids: torch.Tensor | None = None,
                   weights: torch.Tensor | None = None, stream=None):
    """Expert choices of every token: logits [T][experts] (float32 or bfloat16, rows of
    any stride) -> topk_ids int32 [T][topk], as lora_prepare_moe_meta takes them, and
    weights float32 [T][topk]; outputs that are not given are allocated on the stream of
    the call."""
    device = logits.get_device()
    if _elsewhere(device):
        with torch.cuda.device(device):
            return lora_moe_route(logits, routing, topk_ids, weights, stream)
    if logits.dim() != 2:
        raise ValueError("logits must be [T][experts]")
    T, K = logits.shape[0], routing.topk
    ptr, ld = _rows(logits, "logits", logits.dtype, T, routing.num_experts)
    if topk_ids is None:
        topk_ids = _empty_for(stream, (T, K), torch.int32, logits.device)
    if weights is None:
        weights = _empty_for(stream, (T, K), torch.float32, logits.device)
    _apart(device, routing.bias, topk_ids, weights)
    st = _lib.lora_moe_route(routing.ref, ptr, ld, T, _dtype(logits), _vector(topk_ids, "topk_ids", torch.int32, (T, K)),
                             _vector(weights, "weights", torch.float32, (T, K)), _stream_handle(stream))
    _check("lora_moe_route", st)
    return topk_ids, weights


def lora_quantize(x: torch.Tensor, q: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                  activation: str | None = None, act: torch.Tensor | None = None, meta: LoraMeta | None = None,
                  stream=None):
    """Rows of x [rows][width] as 8-bit integers q and a scale each (q * scale is near x).
    activation "silu_mul": x is gate | up and silu(gate) * up is what is rounded, which
    act, if given, takes in x's type.  meta: only the rows that it gives a key.  q and
    scale that are not given are allocated on the stream of the call (with meta, rows
    without a key hold anything)."""
    device = x.get_device()
    if _elsewhere(device):
        with torch.cuda.device(device):
            return lora_quantize(x, q, scale, activation, act, meta, stream)
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}")
    if x.dim() != 2:
        raise ValueError("x must be [rows][width]")
    rows, width = x.shape
    xp, ldx = _rows(x, "x", x.dtype, rows, width)
    if activation:
        if width % 2:
            raise ValueError("x must be gate | up, of one width")
        width //= 2
    elif act is not None:
        raise ValueError("act goes with an activation")
    if q is None:
        q = _empty_for(stream, (rows, width), torch.int8, x.device)
    if scale is None:
        scale = _empty_for(stream, (rows,), torch.float32, x.device)
    _apart(device, q, scale, act, None if meta is None else meta.workspace)
    qp, ldq = _rows(q, "q", torch.int8, rows, width)
    ap, lda = (None, 0) if act is None else _rows(act, "act", x.dtype, rows, width)
    st = _lib.lora_quantize(xp, ldx, rows, width, _dtype(x), ACTIVATIONS[activation],
                            None if meta is None else C.byref(meta.c), qp, ldq,
                            _vector(scale, "scale", torch.float32, (rows,)), ap, lda, _stream_handle(stream))
    _check("lora_quantize", st)
    return q, scale


class Int8Weight:
    """8-bit base weights: w int8 [d_out][d_in], or [experts][d_out][d_in] (bytes of a row
    contiguous; strides multiples of 16; experts one after the other or side by side, as
    in a transposed [d_out][experts][d_in]), scale float32 [d_out] or [experts][d_out],
    bias likewise or None."""

    def __init__(self, w: torch.Tensor, scale: torch.Tensor, bias: torch.Tensor | None = None):
        if w.dim() not in (2, 3) or w.dtype != torch.int8 or w.stride(-1) != 1:
            raise ValueError("w must be int8 [d_out][d_in] or [experts][d_out][d_in] with contiguous rows")
        shape = w.shape[:-1]
        _apart(w.get_device(), scale, bias)
        self.w, self.scale, self.bias = w, scale, bias
        self.num_experts, self.d_out, self.d_in = (w.shape[0] if w.dim() == 3 else 1), w.shape[-2], w.shape[-1]
        self.c = lora_int8_weight(_dev(w, "w"), w.stride(0) if w.dim() == 3 and len(w) > 1 else 0,
                                  w.stride(-2) if self.d_out > 1 else self.d_in,
                                  _vector(scale, "scale", torch.float32, shape),
                                  None if bias is None else _vector(bias, "bias", torch.float32, shape), self.d_in,
                                  self.d_out, self.num_experts, 0)
        self.ref = C.byref(self.c)


def lora_int8_matmul_workspace_bytes(num_rows: int, weight: Int8Weight) -> int:
    """Bytes of lora_int8_matmul's workspace: 0, no form needs one."""
    b = _sz(0)
    _check("lora_int8_matmul_workspace_bytes", _lib.lora_int8_matmul_workspace_bytes(num_rows, weight.ref, C.byref(b)))
    return int(b.value)


def lora_int8_matmul(x: torch.Tensor, x_scale: torch.Tensor, weight: Int8Weight, out: torch.Tensor | None = None,
                     meta: LoraMeta | None = None, dtype: torch.dtype = torch.bfloat16,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[i] = (x[i] @ w.T) * x_scale[i] * w_scale (+ bias), x int8 [rows][d_in] as
    lora_quantize leaves it.  meta: metadata of the output's rows, keyed by expert (row i
    of the output reads row i / x_row_div of x; rows without a key are not written).  An
    out that is not given is allocated on the stream of the call, of type dtype.  No form
    needs a workspace."""
    device = x.get_device()
    if _elsewhere(device):
        with torch.cuda.device(device):
            return lora_int8_matmul(x, x_scale, weight, out, meta, dtype, workspace, stream)
    if x.dim() != 2:
        raise ValueError("x must be [rows][d_in]")
    x_rows = rows = x.shape[0]
    if meta is not None:
        rows, div = meta.num_tokens, int(meta.c.x_row_div)
        if x_rows != -(-rows // div):
            raise ValueError(f"x must have {-(-rows // div)} rows, one for {div} of the metadata's")
    xp, ldx = _rows(x, "x", torch.int8, x_rows, weight.d_in)
    if out is None:
        out = _empty_for(stream, (rows, weight.d_out), dtype, x.device)
    _apart(device, x_scale, weight.w, out, workspace, None if meta is None else meta.workspace)
    yp, ldy = _rows(out, "out", out.dtype, rows, weight.d_out)
    st = _lib.lora_int8_matmul(None if meta is None else C.byref(meta.c), xp, ldx,
                               _vector(x_scale, "x_scale", torch.float32, (x_rows,)), rows, weight.ref, yp, ldy,
                               _dtype(out), None if workspace is None else _dev(workspace, "workspace"),
                               0 if workspace is None else workspace.nbytes, _stream_handle(stream))
    _check("lora_int8_matmul", st)
    return out


def lora_moe_combine(y: torch.Tensor, weights: torch.Tensor, topk_ids: torch.Tensor, out: torch.Tensor | None = None,
                     num_experts: int | None = None, num_local_experts: int | None = None,
                     expert_map: torch.Tensor | None = None, add: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = add[t] + sum of weights[t][j] * y[t * topk + j] over the choices whose
    expert is local (as in lora_prepare_moe_meta; without a map ids below
    num_local_experts, by default all).  add may be out itself."""
    device = y.get_device()
    if _elsewhere(device):
        with torch.cuda.device(device):
            return lora_moe_combine(y, weights, topk_ids, out, num_experts, num_local_experts, expert_map, add, stream)
    if topk_ids.dim() != 2 or y.dim() != 2:
        raise ValueError("topk_ids must be [T][topk], y [T * topk][width]")
    T, K = topk_ids.shape
    width = y.shape[1]
    yp, ldy = _rows(y, "y", y.dtype, T * K, width)
    if expert_map is not None:
        if num_local_experts is None:
            raise ValueError("an expert_map needs num_local_experts")
        if num_experts is None:
            num_experts = expert_map.shape[0]
    if num_experts is None:
        num_experts = num_local_experts if num_local_experts is not None else 0x7fffffff
    if num_local_experts is None:
        num_local_experts = num_experts
    if out is None:
        out = _empty_for(stream, (T, width), y.dtype, y.device)
    _apart(device, weights, topk_ids, out, expert_map, add)
    op, ldout = _rows(out, "out", y.dtype, T, width)
    ap, ldadd = (None, 0) if add is None else _rows(add, "add", y.dtype, T, width)
    st = _lib.lora_moe_combine(
        yp, ldy, width, _dtype(y), _vector(topk_ids, "topk_ids", torch.int32, (T, K)),
        _vector(weights, "weights", torch.float32, (T, K)), T, K, num_experts, num_local_experts,
        None if expert_map is None else _vector(expert_map, "expert_map", torch.int32, (num_experts,)), ap, ldadd, op, ldout,
        _stream_handle(stream))
    _check("lora_moe_combine", st)
    return out


__all__ = ["Routing", "Int8Weight", "lora_moe_route", "lora_quantize", "lora_int8_matmul",
           "lora_int8_matmul_workspace_bytes", "lora_moe_combine", "lora_routing", "lora_int8_weight", "KvCache", "Rotation", "AttnMeta", "lora_cache_append", "lora_prepare_attn_meta",
           "lora_attn_meta_workspace_bytes", "lora_attention", "lora_attention_workspace_bytes", "lora_kv_cache",
           "lora_rotation", "lora_attn_batch", "lora_attn_meta", "LORA_E4M3",
           "lora_apply_noalloc", "NOALLOC_SCRATCH_BYTES", "lora_abi_version", "lora_status_string", "lora_meta_workspace_bytes", "lora_prepare_meta",
           "lora_moe_meta_workspace_bytes", "lora_prepare_moe_meta",
           "lora_shrink_workspace_bytes", "lora_shrink", "lora_expand", "lora_apply_workspace_bytes",
           "lora_apply_workspace_init", "apply_workspace", "apply_workspace_counters", "apply_workspace_flags",
           "lora_apply", "LoraMeta", "LoraError", "lora_weight", "lora_meta", "LIB_PATH", "LORA_LAYOUT_DEFAULT",
           "LORA_LAYOUT_RANK_ROWS", "LORA_LAYOUT_OUT_ROWS"]
