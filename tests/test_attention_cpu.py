"""The cache append and the attention without a GPU: refusals of the C entry
points (each before any HIP call) and of the binding, workspace sizes, the plan's
arithmetic under sanitizers, and the float64 form against plain loops."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

import attn_ref as R
import segmented_gather_rank_amd as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANGXX = "/opt/rocm/llvm/bin/clang++"
INVALID, UNSUPPORTED, WORKSPACE = L.LORA_ERR_INVALID_ARG, L.LORA_ERR_UNSUPPORTED, L.LORA_ERR_WORKSPACE
P = 0x7F0000000000                          # nothing below reads through it


def cache(**kw):
    c = dict(k=P, v=P, page_stride=2 * 16 * 64, head_stride=16 * 64, pos_stride=64, num_pages=9, page_size=16,
             num_heads=2, head_dim=64, dtype=L.LORA_BF16)
    c.update(kw)
    return L.lora_kv_cache(**c)


def rotation(**kw):
    c = dict(table=P, num_pos=100, rot_dim=64, interleaved=0, num_axes=1, reserved=0)
    c.update({k: v for k, v in kw.items() if k != "section"})
    r = L.lora_rotation(**c)
    for i, n in enumerate(kw.get("section", ())):
        r.section[i] = n
    return r


def append(c=None, rot=None, **kw):
    a = dict(qkv=P, ldx=512, T=3, dtype=L.LORA_BF16, hq=4, offset=(0, 256, 384), pos=P, slot=P, q=P, ldq=256, bad=None)
    a.update(kw)
    offs = None if a["offset"] is None else (C.c_int64 * 3)(*a["offset"])
    c = cache() if c is None else c
    return L._lib.lora_cache_append(a["qkv"], a["ldx"], a["T"], a["dtype"], a["hq"], offs,
                                    None if rot is None else C.byref(rot), a["pos"], a["slot"], C.byref(c), a["q"],
                                    a["ldq"], a["bad"], None)


CACHES = [
    (dict(k=None), INVALID), (dict(v=P + 8), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=2 ** 31), INVALID),
    (dict(page_size=0), INVALID), (dict(page_size=65537), UNSUPPORTED), (dict(head_dim=0), INVALID),
    (dict(head_dim=264), UNSUPPORTED), (dict(head_dim=60), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED),
    (dict(dtype=L.LORA_E4M3, head_dim=72), UNSUPPORTED), (dict(pos_stride=66), INVALID), (dict(pos_stride=-64), INVALID),
    (dict(pos_stride=56), INVALID), (dict(head_stride=0), INVALID), (dict(page_stride=8), INVALID),
    (dict(dtype=L.LORA_E4M3, pos_stride=72), INVALID), (dict(k_scale=P), INVALID), (dict(num_heads=1025), UNSUPPORTED),
    (dict(dtype=L.LORA_E4M3, v_scale=P + 2), INVALID),
]


@pytest.mark.parametrize("kw,status", CACHES, ids=lambda v: str(v))
def test_cache_refusals(kw, status):
    assert append(cache(**kw)) == status
    m, bytes_ = meta(), 1 << 40
    for f in ("num_kv_heads", "head_dim", "page_size", "dtype"):
        setattr(m, f, kw.get({"num_kv_heads": "num_heads"}.get(f, f), getattr(m, f)))
    assert L._lib.lora_attention(C.byref(m), P, 256, C.byref(cache(**kw)), 1.0, 0.0, None, P, 256, None, P, bytes_,
                                 None) in (status, INVALID)


@pytest.mark.parametrize("kw,status", [
    (dict(qkv=None), INVALID), (dict(qkv=P + 4), INVALID), (dict(slot=None), INVALID), (dict(slot=P + 4), INVALID),
    (dict(T=-1), INVALID), (dict(T=2 ** 31), UNSUPPORTED), (dict(dtype=L.LORA_E4M3), UNSUPPORTED),
    (dict(dtype=L.LORA_F32), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(offset=None), INVALID),
    (dict(offset=(0, 256, 392)), INVALID), (dict(offset=(4, 256, 384)), INVALID), (dict(offset=(-8, 256, 384)), INVALID),
    (dict(offset=(0, 1 << 62, 384)), INVALID), (dict(ldx=508), INVALID), (dict(ldx=504), INVALID), (dict(hq=-1), INVALID),
    (dict(hq=2000), UNSUPPORTED), (dict(q=P + 2), INVALID), (dict(ldq=248), INVALID), (dict(ldq=260), INVALID),
    (dict(bad=P + 1), INVALID),
], ids=lambda v: str(v))
def test_append_refusals(kw, status):
    assert append(**kw) == status


@pytest.mark.parametrize("kw", [
    dict(table=None), dict(table=P + 4), dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=80), dict(num_axes=0),
    dict(num_axes=5), dict(num_pos=-1), dict(reserved=1), dict(num_axes=2, section=(30, 1)),
    dict(num_axes=2, section=(33, -1)), dict(num_axes=3, section=(16, 16, 1)),
], ids=lambda v: str(v))
def test_rotation_refusals(kw):
    assert append(rot=rotation(**kw)) == INVALID


def test_append_of_nothing():
    assert append(T=0, qkv=None, slot=None, q=None) == L.LORA_OK
    assert append(rot=rotation(), pos=None) == INVALID


def batch(**kw):
    b = dict(d_q_start=P, d_kv_len=P, d_page_table=P, page_table_stride=10, num_tokens=20, num_seqs=5, max_q_len=20,
             num_q_heads=4, causal=1)
    b.update(kw)
    return L.lora_attn_batch(**b)


BATCHES = [
    (dict(num_tokens=-1), INVALID), (dict(num_seqs=-1), INVALID), (dict(max_q_len=-1), INVALID),
    (dict(num_q_heads=3), INVALID), (dict(num_q_heads=0), INVALID), (dict(window=-1), INVALID),
    (dict(num_groups=-1), INVALID), (dict(num_groups=6), UNSUPPORTED), (dict(num_tokens=2 ** 25), UNSUPPORTED),
    (dict(num_seqs=2 ** 21), UNSUPPORTED), (dict(num_q_heads=1026), UNSUPPORTED),
    (dict(page_table_stride=2 ** 27), UNSUPPORTED), (dict(page_table_stride=-1), INVALID),
]


@pytest.mark.parametrize("kw,status", BATCHES, ids=lambda v: str(v))
def test_batch_refusals(kw, status):
    n = C.c_size_t(0)
    assert L._lib.lora_attn_meta_workspace_bytes(C.byref(batch(**kw)), C.byref(cache()), C.byref(n)) == status
    m = L.lora_attn_meta()
    assert L._lib.lora_prepare_attn_meta(C.byref(batch(**kw)), C.byref(cache()), P, 1 << 40, C.byref(m), None) == status


@pytest.mark.parametrize("kw", [
    dict(d_q_start=None), dict(d_kv_len=None), dict(d_page_table=None), dict(d_kv_len=P + 2), dict(d_key_lo=P),
    dict(d_key_hi=P), dict(num_groups=1), dict(num_groups=1, d_group_start=P), dict(d_prefix_len=P + 1),
], ids=lambda v: str(v))
def test_prepare_refusals(kw):
    m = L.lora_attn_meta()
    assert L._lib.lora_prepare_attn_meta(C.byref(batch(**kw)), C.byref(cache()), P, 1 << 40, C.byref(m), None) == INVALID


def test_workspaces():
    n, m = C.c_size_t(0), L.lora_attn_meta()
    assert L._lib.lora_attn_meta_workspace_bytes(C.byref(batch()), C.byref(cache()), C.byref(n)) == L.LORA_OK
    assert n.value % 256 == 0 and n.value > 20 * 48
    call = L._lib.lora_prepare_attn_meta
    assert call(C.byref(batch()), C.byref(cache()), P, n.value - 1, C.byref(m), None) == WORKSPACE
    assert call(C.byref(batch()), C.byref(cache()), None, n.value, C.byref(m), None) == INVALID
    assert call(C.byref(batch()), C.byref(cache()), P + 8, n.value, C.byref(m), None) == INVALID
    assert call(C.byref(batch()), C.byref(cache()), P, n.value, None, None) == INVALID
    assert call(None, C.byref(cache()), P, n.value, C.byref(m), None) == INVALID
    assert call(C.byref(batch()), None, P, n.value, C.byref(m), None) == INVALID
    assert L._lib.lora_attention_workspace_bytes(None, C.byref(n)) == INVALID
    assert L._lib.lora_attention_workspace_bytes(C.byref(meta()), None) == INVALID


def meta(**kw):
    m = dict(num_tokens=20, page_table_stride=10, max_units=50, num_seqs=5, num_q_heads=4, num_kv_heads=2, head_dim=64,
             page_size=16, dtype=L.LORA_BF16, heads_per_item=2, head_groups=1, max_tiles=5, max_slots=9,
             max_tile_items=9, page_table=P, limits=P, info=P, tiles=P, few_items=P, slots=P, tile_items=P, join=P, join_list=P)
    m.update(kw)
    return L.lora_attn_meta(**m)


@pytest.mark.parametrize("kw,mk,ck,status", [
    (dict(q=None), {}, {}, INVALID), (dict(q=P + 2), {}, {}, INVALID), (dict(out=None), {}, {}, INVALID),
    (dict(ldq=248), {}, {}, INVALID), (dict(ldo=260), {}, {}, INVALID), (dict(cap=-1.0), {}, {}, INVALID),
    (dict(cap=float("nan")), {}, {}, INVALID), (dict(cap=float("inf")), {}, {}, INVALID), (dict(ws=None), {}, {}, INVALID),
    (dict(ws=P + 4), {}, {}, INVALID), (dict(nbytes=16), {}, {}, WORKSPACE), (dict(lse=P + 2), {}, {}, INVALID),
    (dict(slopes=P + 2), {}, {}, INVALID), ({}, dict(head_dim=72), {}, INVALID), ({}, dict(num_kv_heads=4), {}, INVALID),
    ({}, dict(page_size=32), {}, INVALID), ({}, dict(dtype=L.LORA_F32), {}, INVALID), ({}, dict(limits=None), {}, INVALID),
    ({}, dict(heads_per_item=3), {}, INVALID), ({}, dict(heads_per_item=0), {}, INVALID), ({}, dict(max_units=-1), {}, INVALID),
    ({}, {}, dict(k=None), INVALID),
], ids=lambda v: str(v))
def test_attention_refusals(kw, mk, ck, status):
    a = dict(q=P, ldq=256, out=P, ldo=256, cap=0.0, slopes=None, lse=None, ws=P, nbytes=1 << 40)
    a.update(kw)
    assert L._lib.lora_attention(C.byref(meta(**mk)), a["q"], a["ldq"], C.byref(cache(**ck)), 1.0, a["cap"], a["slopes"],
                                 a["out"], a["ldo"], a["lse"], a["ws"], a["nbytes"], None) == status


def test_attention_of_nothing():
    assert L._lib.lora_attention(C.byref(meta(num_tokens=0)), None, 256, C.byref(cache()), 1.0, 0.0, None, None, 256,
                                 None, None, 0, None) == L.LORA_OK


def test_binding_refusals():
    k = torch.zeros((2, 1, 4, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        L.KvCache(k, k.clone())
    with pytest.raises(ValueError, match="stride"):
        L.KvCache(k, torch.zeros((2, 4, 1, 16), dtype=torch.bfloat16).transpose(1, 2).contiguous()[:1])
    with pytest.raises(ValueError, match="contiguous"):
        L.KvCache(k.transpose(2, 3), k.transpose(2, 3))
    with pytest.raises(TypeError):
        L.KvCache(k.half(), k.half())
    with pytest.raises(ValueError, match="k_scale"):
        L.KvCache(k, k.clone(), torch.ones(2))
    with pytest.raises(ValueError, match="table"):
        L.Rotation(torch.zeros(4, 4, dtype=torch.float64))
    with pytest.raises(ValueError, match="axes"):
        L.Rotation(torch.zeros(4, 16), sections=[1, 1, 1, 1, 4])


@pytest.mark.skipif(not os.path.exists(CLANGXX), reason="ROCm toolchain not found")
def test_plan_arithmetic_under_sanitizers(tmp_path):
    exe = str(tmp_path / "plan_check")
    subprocess.run([CLANGXX, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-o", exe, os.path.join(ROOT, "tests", "attn_plan_check.cpp")], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "all checks passed" in r.stdout, r.stdout + r.stderr


def test_reference_against_loops():
    """The test's own float64 form, element by element, on a small batch."""
    b = R.Batch([2, 3], [5, 3], 4, 2, 8, 2, "e4m3", seed=1, window=3, prefix_len=np.array([0, 2]))
    out, lse, _, _ = b.reference(cap=2.0, slopes=[0.1, 0.2, 0.3, 0.4])
    kk, vv = b.views()
    for n in range(2):
        for i in range(b.q_len[n]):
            t, p = int(b.q_start[n]) + i, b.kv_len[n] - b.q_len[n] + i
            for h in range(4):
                num, den = np.zeros(8), 0.0
                for j in range(b.kv_len[n]):
                    pre = [0, 2][n]
                    if j <= p - 3 or (j > p and j >= pre):
                        continue
                    pg, at = b.table[n, j // 2], j % 2
                    k = kk[pg, h // 2, at].to(torch.float64).numpy() * float(b.k_scale[h // 2])
                    v = vv[pg, h // 2, at].to(torch.float64).numpy() * float(b.v_scale[h // 2])
                    x = float(k @ b.q[t, h].to(torch.float64).numpy()) / np.sqrt(8)
                    x = 2 * np.tanh(x / 2) - [0.1, 0.2, 0.3, 0.4][h] * abs(p - j)
                    num, den = num + np.exp(x) * v, den + np.exp(x)
                np.testing.assert_allclose(out[t, h], num / den, rtol=1e-12, atol=1e-12)
                np.testing.assert_allclose(lse[t, h], np.log(den), rtol=1e-12, atol=1e-12)


def test_e4m3_rounding_against_torch():
    x = torch.cat([torch.randn(4000) * 50, torch.randn(4000) * 0.01, torch.arange(-500, 500).float() / 7])
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    np.testing.assert_array_equal(R.e4m3_round(x.to(torch.float64).numpy()), want)
    assert R.e4m3_round(np.array([np.inf, -np.inf])).tolist() == [448.0, -448.0] and np.isnan(R.e4m3_round(np.nan))
