"""lora_cache_append against the float64 form: rotation in both pairings and
with several axes, every cache type, strides, slots that are not kept, bad tokens."""
import numpy as np
import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import segmented_gather_rank_amd as lib
    return lib


CASES = [
    # T, hq, hkv, D, rot (0: none), page, dtype, cache, interleaved, sections, layout, gaps
    (1, 1, 1, 8, 0, 1, "bf16", "bf16", False, None, "heads", 0),
    (1, 32, 8, 128, 128, 16, "bf16", "bf16", False, None, "heads", 0),
    (7, 4, 2, 64, 64, 7, "bf16", "bf16", True, None, "tokens", 8),
    (33, 7, 1, 96, 48, 16, "bf16", "bf16", False, None, "heads", 16),
    (33, 6, 3, 72, 64, 5, "bf16", "bf16", True, None, "tokens", 0),
    (50, 8, 2, 128, 128, 16, "bf16", "bf16", False, [22, 21, 21], "heads", 0),
    (50, 8, 2, 128, 96, 16, "bf16", "e4m3", True, [0, 10, 38], "heads", 8),
    (50, 8, 2, 64, 32, 64, "bf16", "e4m3", False, [1, 2, 3, 10], "tokens", 0),
    (129, 4, 4, 256, 256, 32, "bf16", "e4m3", False, None, "heads", 0),
    (20, 4, 2, 256, 256, 16, "f32", "f32", False, [128, 0], "heads", 8),
    (20, 3, 1, 40, 16, 16, "f32", "f32", True, None, "tokens", 0),
    (300, 16, 16, 96, 0, 16, "bf16", "e4m3", False, None, "heads", 0),
]
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def make(case, seed=3):
    T, hq, hkv, D, rot, page, dtype, cache, inter, sections, layout, gap = case
    r = np.random.Generator(np.random.PCG64(seed))
    width = (hq + 2 * hkv) * D + 3 * gap
    qkv = torch.from_numpy((3 * r.standard_normal((T, width))).astype(np.float32)).to(TORCH[dtype])
    pages = (T + page - 1) // page + 4
    shape = (pages, hkv, page, D) if layout == "heads" else (pages, page, hkv, D)
    k = torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(TORCH[cache])
    v = torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(TORCH[cache])
    slot = torch.from_numpy(r.permutation(pages * page)[:T].astype(np.int64))
    scales = [torch.from_numpy(r.uniform(0.01, 2, hkv).astype(np.float32)) for _ in range(2)] if cache == "e4m3" else [None, None]
    offs = (gap, hq * D + 2 * gap, (hq + hkv) * D + 2 * gap)
    table = pos = None
    if rot:
        table = torch.from_numpy(r.uniform(-1, 1, (50, rot)).astype(np.float32))
        pos = torch.from_numpy(r.integers(0, 50, (len(sections or [0]), T)).astype(np.int32))
    return qkv, k, v, slot, scales, offs, table, pos


def f64(t):
    return t.to(torch.float64).numpy()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
@pytest.mark.parametrize("kind", ["apart", "in_place", "no_q"])
def test_append(L, case, kind):
    T, hq, hkv, D, rot, page, dtype, cache, inter, sections, layout, gap = case
    qkv, k, v, slot, scales, offs, table, pos = make(case)
    if T > 4:
        slot[1], slot[3] = -1, -5                    # not kept; bad
        slot[4] = k.numel() // (hkv * D)             # bad: one past the last
        if rot and T > 8:
            pos[0, 6], pos[-1, 7] = 50, -1           # bad positions
    swap = (lambda x: x.transpose(1, 2)) if layout == "tokens" else (lambda x: x)
    ref_q, ref_k, ref_v, bad = R.append(
        f64(qkv), hq, hkv, D, offs, slot.numpy(), f64(swap(k)), f64(swap(v)), *[None if s is None else s.numpy() for s in scales],
        table=None if table is None else table.numpy(), pos=None if pos is None else pos.numpy(), rot=rot,
        interleaved=inter, sections=sections or [rot // 2], e4m3=cache == "e4m3", page_size=page)
    dk, dv, dx = k.cuda(), v.cuda(), qkv.cuda()
    kv = L.KvCache(swap(dk), swap(dv), *[None if s is None else s.cuda() for s in scales])
    rotation = L.Rotation(table.cuda(), sections=sections, interleaved=inter) if rot else None
    marker = 7.0
    out = None
    if kind == "apart":
        out = torch.full((T, hq * D + 16), marker, dtype=dx.dtype, device="cuda")[:, :hq * D + 8]
    elif kind == "in_place":
        out = dx[:, offs[0]:offs[0] + hq * D]
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lora_cache_append(dx, kv, slot.cuda(), out, pos=None if pos is None else pos.cuda(), rotation=rotation,
                        num_q_heads=hq, offsets=offs, num_bad=count)
    torch.cuda.synchronize()
    assert int(count) == bad
    if kind != "in_place":
        assert torch.equal(dx.cpu().view(torch.uint8), qkv.view(torch.uint8))
    half = R.F32_HALF if dtype == "f32" else R.BF16_HALF
    # two products and a sum in fp32 of values up to |a| + |b|, one rounding
    slack = 3 * R.F32_HALF * 2 * np.abs(f64(qkv)).max()
    if out is not None:
        got = f64(out[:, :hq * D].cpu())
        rows = ~np.isnan(ref_q).any(1)
        assert np.all(np.abs(got - ref_q)[rows] <= half * np.abs(ref_q[rows]) + slack)
        before = marker if kind == "apart" else f64(qkv)[:, offs[0]:offs[0] + hq * D][~rows]
        assert np.all(got[~rows] == before)
        if kind == "apart":
            assert torch.all(out[:, hq * D:] == marker)
    got_k, got_v = f64(swap(dk).cpu()), f64(swap(dv).cpu())
    if cache == "e4m3":
        # half a step of e4m3: 2^-4 of the value, or half of the smallest number
        near = torch.finfo(torch.float8_e4m3fn).eps / 2
        bound = near * np.abs(ref_k) + 2.0 ** -10 + slack * 200
        assert np.all(np.abs(got_k - np.clip(ref_k, -448, 448)) <= bound)
        assert np.array_equal(got_v, ref_v)
        if not rot:
            touched = got_k != f64(swap(k))
            assert np.array_equal(got_k[touched], R.e4m3_round(ref_k.astype(np.float32))[touched])
    else:
        assert np.all(np.abs(got_k - ref_k) <= half * np.abs(ref_k) + slack)
        assert np.array_equal(got_v, ref_v)


def test_e4m3_values(L):
    """Saturation, NaN, the smallest numbers and ties, with and without a scale."""
    vals = [0.0, -0.0, 1.0, 448.0, 449.0, 463.9, 464.0, 480.0, 1e30, -1e30, float("inf"), -float("inf"), float("nan"),
            2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -10, -2.0 ** -11, 17.0, 19.0, 0.0171, 240.0, 248.0, 1.0625, 1.1875]
    x = torch.zeros((1, 96), dtype=torch.bfloat16)
    x[0, 64:64 + len(vals)] = torch.tensor(vals).to(torch.bfloat16)
    x[0, 32:32 + len(vals)] = torch.tensor(vals).to(torch.bfloat16)
    for scale in (None, 0.375):
        k = torch.zeros((1, 1, 1, 32), dtype=torch.float8_e4m3fn, device="cuda")
        v = torch.zeros_like(k)
        s = None if scale is None else torch.tensor([scale], device="cuda")
        L.lora_cache_append(x.cuda(), L.KvCache(k, v, s, s), torch.zeros(1, dtype=torch.int64, device="cuda"),
                            num_q_heads=1)
        y = x[0, 64:].to(torch.float32).numpy()
        ref = R.e4m3_round(y if scale is None else y / np.float32(scale))
        for t in (k, v):
            np.testing.assert_array_equal(t.cpu().to(torch.float64).numpy().ravel(), ref)


def test_far_offsets(L):
    """A cache whose last page lies beyond 2^32 elements."""
    page, D = 1024, 256
    pages = (1 << 32) // (page * D * 4) + 3
    k = torch.empty((pages, 4, page, D), dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.empty_like(k)
    x = torch.randn((2, 12 * D), device="cuda").to(torch.bfloat16)
    slot = torch.tensor([pages * page - 1, 0], device="cuda")
    L.lora_cache_append(x, L.KvCache(k, v), slot, num_q_heads=4)
    want_k = x[:, 4 * D:8 * D].to(torch.float8_e4m3fn).view(2, 4, D)
    want_v = x[:, 8 * D:].to(torch.float8_e4m3fn).view(2, 4, D)
    for i, (p, at) in enumerate(((pages - 1, page - 1), (0, 0))):
        assert torch.equal(k[p, :, at].float(), want_k[i].float())
        assert torch.equal(v[p, :, at].float(), want_v[i].float())


def test_nothing_to_do(L):
    k = torch.zeros((2, 1, 4, 16), dtype=torch.bfloat16, device="cuda")
    e = torch.empty((0, 48), dtype=torch.bfloat16, device="cuda")
    L.lora_cache_append(e, L.KvCache(k, k.clone()), torch.empty(0, dtype=torch.int64, device="cuda"), num_q_heads=1)
    torch.cuda.synchronize()
    assert not k.any()
