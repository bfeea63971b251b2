"""The binding of the attention without a GPU: what it sizes, checks and refuses before
any device call."""
import ctypes as C
from types import SimpleNamespace

import pytest
import torch

import segmented_gather_rank_amd as L


def cache(dtype, heads, dim, page=16):
    c = L.lora_kv_cache(page_size=page, num_heads=heads, head_dim=dim, dtype=dtype)
    return SimpleNamespace(c=c, ref=C.byref(c))


@pytest.mark.parametrize("dtype", [L.LORA_BF16, L.LORA_E4M3, L.LORA_F32])
@pytest.mark.parametrize("dim", [16, 64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (32, 8), (8, 8)])
@pytest.mark.parametrize("groups", [0, 2])
def test_metadata_bytes_cover_every_query_length(dtype, dim, hq, hkv, groups):
    """A workspace sized without max_q_len takes a batch that states any."""
    kv_len, table = torch.zeros(9, dtype=torch.int32), torch.zeros((9, 10), dtype=torch.int32)
    kv = cache(dtype, hkv, dim)
    given = L.lora_attn_meta_workspace_bytes(None, kv_len, table, kv, hq, 30, groups)
    for most in (0, 1, 2, 3, 4, 5, 16, 17, 30, 1000):
        b = L.lora_attn_batch(page_table_stride=10, num_tokens=30, num_seqs=9, max_q_len=most, num_q_heads=hq,
                              num_groups=groups)
        need = C.c_size_t(0)
        assert L._lib.lora_attn_meta_workspace_bytes(C.byref(b), kv.ref, C.byref(need)) == L.LORA_OK
        assert given >= need.value
        assert L.lora_attn_meta_workspace_bytes(None, kv_len, table, kv, hq, 30, groups, max_q_len=most) == need.value


@pytest.mark.parametrize("axes,shape,ok", [
    (1, (5,), True), (1, (1, 5), True), (1, (6,), False), (3, (3, 5), True), (3, (15,), True),
    (3, (5, 3), False), (2, (5, 2), False), (2, (2, 4), False),
])
def test_positions_are_axes_by_tokens(monkeypatch, axes, shape, ok):
    """pos is [axes][T]: [T][axes] would be taken for other tokens' positions."""
    kv = cache(L.LORA_BF16, 1, 16)
    kv.head_dim, kv.num_heads, kv.packed_offsets = 16, 1, lambda n: ((C.c_int64 * 3)(0, 16, 32), 48)
    rotation = SimpleNamespace(num_axes=axes, ref=C.byref(L.lora_rotation()))
    monkeypatch.setattr(L, "_dev", lambda t, name: 0)
    monkeypatch.setattr(L, "_stream_handle", lambda stream: 0)
    call = lambda: L.lora_cache_append(torch.zeros((5, 48), dtype=torch.bfloat16), kv,  # noqa: E731
                                       torch.zeros(5, dtype=torch.int64), num_q_heads=1, rotation=rotation,
                                       pos=torch.zeros(shape, dtype=torch.int32))
    if ok:                                   # the library then refuses the null pointers
        with pytest.raises(L.LoraError):
            call()
    else:
        with pytest.raises(ValueError, match="pos"):
            call()
