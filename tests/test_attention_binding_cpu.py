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
