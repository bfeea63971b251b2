"""lora_attention against the float64 form: head layouts, head sizes, page sizes,
lengths, masks that leave rows empty, cap and bias, groups with shared keys, bad
sequences and pages, infinities in hidden places, graphs, streams."""
import numpy as np
import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import segmented_gather_rank_amd as lib
    return lib


def dev(a):
    return None if a is None else torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).cuda()


class Dev:
    def __init__(self, L, b, max_q_len="fit"):
        self.k, self.v = b.k_store.cuda(), b.v_store.cuda()
        swap = (lambda x: x.transpose(1, 2)) if b.layout == "tokens" else (lambda x: x)
        self.cache = L.KvCache(swap(self.k), swap(self.v), *[None if s is None else s.cuda() for s in (b.k_scale, b.v_scale)])
        self.args = (dev(b.q_start), dev(b.kv_len), dev(b.table))
        self.kw = dict(max_q_len=max(b.q_len + [0]) if max_q_len == "fit" else max_q_len, causal=b.causal,
                       window=b.window, prefix_len=dev(b.prefix_len), key_lo=dev(b.key_lo), key_hi=dev(b.key_hi),
                       group_start=dev(b.groups), group_len=dev(b.group_len))
        self.q = b.q.cuda()
        self.b = b

    def meta(self, L, **kw):
        return L.lora_prepare_attn_meta(*self.args, self.cache, self.b.hq, self.b.T, **{**self.kw, **kw})


def check(b, out, lse, ref, what=""):
    ro, rl, to, tl = ref
    got, gl = out.cpu().to(torch.float64).numpy(), lse.cpu().to(torch.float64).numpy()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), empty), what
    assert np.all(got[empty] == 0), what
    err = np.abs(got - ro)
    bad = ~(err <= to)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of tolerance, first {np.argwhere(bad)[0]}: " \
        f"{got[bad][0]} for {ro[bad][0]} (tolerance {to[bad][0]})"
    e = np.abs(gl[~empty] - rl[~empty])
    assert np.all(e <= tl[~empty]), f"{what}: lse off by {e.max()}"


def run(L, b, cap=0.0, slopes=None, scale=None, max_q_len="fit", strided=False):
    d = Dev(L, b, max_q_len)
    meta = d.meta(L)
    T, w = b.T, b.hq * b.D
    q, out = d.q, None
    marker = 3.0
    if strided:
        big = torch.zeros((T, w + 40), dtype=q.dtype, device="cuda")
        big[:, 16:16 + w] = q.view(T, w)
        q = big[:, 16:16 + w]
        hold = torch.full((T, w + 24), marker, dtype=q.dtype, device="cuda")
        out = hold[:, 8:8 + w]
    lse = torch.full((T, b.hq), 5.0, device="cuda")
    ws = torch.full((max(16, L.lora_attention_workspace_bytes(meta)),), 255, dtype=torch.uint8, device="cuda")
    o, _ = L.lora_attention(meta, q, d.cache, out, scale=scale, cap=cap, lse=lse, workspace=ws,
                            slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32).cuda())
    torch.cuda.synchronize()
    if strided:
        assert torch.all(hold[:, :8] == marker) and torch.all(hold[:, 8 + w:] == marker)
    return o.reshape(T, b.hq, b.D), lse, meta, d


HEADS = [(1, 1), (8, 2), (7, 1), (34, 2), (32, 1), (6, 6)]
DIMS = [8, 40, 64, 72, 128, 136, 256]


@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_decode_heads(L, hq, hkv, cache):
    """One token each, lengths around the 32-key step, the item and the page."""
    kv = [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300]
    b = R.Batch([1] * len(kv), kv, hq, hkv, 64, 16, cache, "tokens", seed=hq)
    o, lse, _, _ = run(L, b)
    check(b, o, lse, b.reference())


@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("D", DIMS)
def test_head_sizes(L, D, cache):
    if cache == "e4m3" and D % 16:
        D += 8
    b = R.Batch([1, 40, 3, 1], [70, 45, 131, 257], 4, 2, D, 5, cache, "heads", seed=D)
    o, lse, _, _ = run(L, b, strided=True)
    check(b, o, lse, b.reference())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [1, 3, 16, 64, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_mixed_lengths(L, page, causal, cache):
    """Decode, short extensions, prompts and sequences without queries or keys,
    either side of 16 and of 128 rows."""
    q = [1, 0, 4, 5, 32, 33, 64, 100, 1, 0]
    kv = [1, 0, 4, 77, 32, 160, 65, 100, 500, 40]
    b = R.Batch(q, kv, 8, 2, 64, page, cache, seed=page, causal=causal)
    o, lse, meta, _ = run(L, b)
    check(b, o, lse, b.reference())
    info = meta.tensors()["info"].cpu().numpy()
    assert info[0] > 0 and info[1] > 0 and info[2] == 0


@pytest.mark.parametrize("q,kv,heads", [([1], [9000], (8, 1)), ([40], [3000], (8, 2)), ([128, 1], [2500, 2500], (4, 4))])
@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_split_ranges(L, q, kv, heads, cache):
    """Few rows, long contexts: results in parts, joined."""
    b = R.Batch(q, kv, *heads, 64, 16, cache, seed=5)
    o, lse, meta, _ = run(L, b)
    assert int(meta.tensors()["info"][4]) > 0
    check(b, o, lse, b.reference())


def masks(kind, q, kv, rng):
    T = sum(q)
    starts = np.concatenate([[0], np.cumsum(q)])
    if kind == "window":
        return dict(window=37)
    if kind == "prefix":
        return dict(prefix_len=np.array([0, kv[1] // 2, 10 ** 6, 1][:len(q)]))
    lo, hi = np.zeros(T, np.int64), np.zeros(T, np.int64)
    for n in range(len(q)):
        for i in range(q[n]):
            t, p = starts[n] + i, kv[n] - q[n] + i
            doc = p // 29
            lo[t], hi[t] = doc * 29, min(kv[n], doc * 29 + 29)
    if kind == "documents":
        return dict(key_lo=lo, key_hi=hi, causal=False)
    if kind == "empty_rows":
        cut = rng.random(T) < 0.4
        hi[cut] = lo[cut] - rng.integers(0, 5, cut.sum())
        return dict(key_lo=lo, key_hi=hi)
    if kind == "all_empty":
        return dict(key_lo=lo + 5, key_hi=lo)
    if kind == "negative_bounds":
        return dict(key_lo=lo * 0 - 2 ** 31, key_hi=lo * 0 + 2 ** 31 - 1)
    if kind == "ragged":                      # every row an interval of its own
        kvt = np.repeat(kv, q)
        a = rng.integers(0, kvt)
        return dict(key_lo=a, key_hi=a + rng.integers(0, 80, T), causal=False)
    raise KeyError(kind)


@pytest.mark.parametrize("kind", ["window", "prefix", "documents", "empty_rows", "all_empty", "negative_bounds", "ragged"])
@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
def test_masks(L, kind, cache):
    q, kv = [1, 70, 3, 130], [200, 190, 100, 130]
    b = R.Batch(q, kv, 4, 2, 64, 16, cache, seed=11, **masks(kind, q, kv, np.random.default_rng(4)))
    o, lse, _, _ = run(L, b)
    check(b, o, lse, b.reference())


@pytest.mark.parametrize("cap,slope,scale", [(30.0, False, None), (0.0, True, None), (5.0, True, 0.5), (50.0, False, -0.2)])
@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
def test_cap_and_bias(L, cap, slope, scale, cache):
    b = R.Batch([1, 50, 2], [300, 120, 64], 8, 4, 128, 16, cache, seed=2, window=100,
                prefix_len=np.array([5, 110, 0]))
    slopes = [2.0 ** -(h + 1) for h in range(8)] if slope else None
    o, lse, _, _ = run(L, b, cap=cap, slopes=slopes, scale=scale)
    check(b, o, lse, b.reference(scale=scale, cap=cap, slopes=slopes))


GROUPS = [
    # q_len, kv_len, group starts, lengths
    ([1] * 6, [100, 90, 300, 81, 200, 120], [0, 6], [80]),
    ([1] * 6, [100, 90, 300, 81, 200, 120], [0, 2, 2, 6], [64, 7, 33]),
    ([1, 5, 40, 1, 1], [700, 705, 740, 650, 30], [0, 4], [601]),
    ([1] * 40, [200 + n for n in range(40)], [4, 39], [200]),
    ([2, 20, 1], [50, 60, 70], [0, 3], [48]),          # a prefix that ends at the first token's position
    ([1, 1, 1], [40, 64, 40], [0, 3], [40]),           # sequences that end inside the shared keys' end
    ([1] * 3, [20, 30, 40], [0, 3], [0]),
]


@pytest.mark.parametrize("case", GROUPS, ids=range(len(GROUPS)))
@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("heads", [(8, 2), (3, 3)])
def test_groups(L, case, cache, heads):
    q, kv, starts, lens = case
    b = R.Batch(q, kv, *heads, 64, 16, cache, seed=9, groups=starts, group_len=lens)
    d_plain = R.Batch.reference(b)
    o, lse, meta, _ = run(L, b)
    assert int(meta.tensors()["info"][3]) == 0
    check(b, o, lse, d_plain)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_many_rows_to_join(L, cache):
    """More rows in parts than the join gives a workgroup each (1024)."""
    n = 150
    b = R.Batch([1] * n, [70 + i % 40 for i in range(n)], 8, 2, 128, 16, cache, seed=4, groups=[0, 100, n],
                group_len=[64, 70])
    o, lse, meta, _ = run(L, b)
    assert int(meta.tensors()["info"][4]) == n
    check(b, o, lse, b.reference())


def test_more_tiles_than_workgroups(L):
    """Tile items that the workgroups take in rounds: over 4096 of them."""
    n = 140
    b = R.Batch([17] * n, [17 + i % 50 for i in range(n)], 32, 32, 16, 16, "bf16", seed=4)
    o, lse, meta, _ = run(L, b)
    assert int(meta.tensors()["info"][1]) * 32 > 4096
    check(b, o, lse, b.reference())


def test_groups_with_masks(L):
    q, kv = [1, 6, 1, 30, 1], [300, 306, 290, 330, 500]
    r = np.random.default_rng(1)
    T = sum(q)
    lo = r.integers(0, 280, T)
    b = R.Batch(q, kv, 8, 2, 64, 16, "bf16", seed=9, groups=[0, 3, 5], group_len=[256, 200], window=150,
                key_lo=lo, key_hi=lo + r.integers(0, 200, T), prefix_len=np.array([0, 300, 0, 250, 0]))
    o, lse, _, _ = run(L, b, cap=20.0, slopes=[0.01 * h for h in range(8)])
    check(b, o, lse, b.reference(cap=20.0, slopes=[0.01 * h for h in range(8)]))


def test_bad_sequences_groups_and_pages(L):
    q, kv = [1, 3, 1, 20, 1, 1, 30], [50, 60, 40, 90, 45, 33, 64]
    b = R.Batch(q, kv, 4, 2, 64, 16, "bf16", seed=3, groups=[0, 2, 4, 4], group_len=[16, 10, 3])
    b.group_len = [16, 500, 3]
    b.table[0, 2], b.table[6, 1], b.table[5, 0] = -1, b.pages, 2 ** 31 - 1      # ids outside the cache
    d = Dev(L, b)
    # too many keys for the table; fewer keys than queries
    kv_dev = np.array(b.kv_len)
    kv_dev[2], kv_dev[3] = 10 ** 6, 19
    d.args = (d.args[0], dev(kv_dev), d.args[2])
    meta = d.meta(L)
    lse = torch.empty((b.T, 4), device="cuda")
    o, _ = L.lora_attention(meta, d.q, d.cache, lse=lse)
    check(b, o, lse, b.reference(bad_seqs=(2, 3)))
    info = meta.tensors()["info"].cpu().tolist()
    assert info[2] == 2 and info[3] == 1      # group 1: longer than its first sequence; group 2 is empty
    # more query tokens than stated
    meta = d.meta(L, max_q_len=2)
    assert int(meta.tensors()["info"][2]) == 4


def test_query_bounds_out_of_order(L):
    """q_start that is not ascending or leaves the batch: those sequences are bad,
    nothing is written out of bounds, the others are right."""
    b = R.Batch([2, 2, 2, 2], [40, 50, 60, 70], 4, 2, 64, 16, "bf16", seed=3)
    d = Dev(L, b)
    for starts in ([0, 2, 1, 6, 8], [-5, 2, 4, 6, 8], [0, 2, 4, 6, 900], [0, 900, 4, 6, 8], [8, 8, 8, 8, 8], [3, 2, 1, 0, -1]):
        d.args = (dev(starts), d.args[1], d.args[2])
        hold = torch.full((b.T + 2, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        meta = d.meta(L, max_q_len=2)
        L.lora_attention(meta, d.q, d.cache, hold[1:-1])
        torch.cuda.synchronize()
        assert torch.all(hold[0] == 9) and torch.all(hold[-1] == 9)
        bad = sum(not (0 <= a <= e <= b.T and e - a <= 2 and e - a <= k) for a, e, k in zip(starts, starts[1:], b.kv_len))
        assert int(meta.tensors()["info"][2]) == bad


@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("q", [3, 100])
@pytest.mark.parametrize("D", [64, 72])
def test_hidden_infinities(L, q, cache, D):
    """Infinite and NaN keys and values beyond a sequence's end, before its window
    and after a row's position reach no row that does not see them."""
    if cache == "e4m3" and D % 16:
        D = 80
    b = R.Batch([q], [q + 90], 4, 2, D, 16, cache, seed=8, window=60)
    clean = R.Batch([q], [q + 90], 4, 2, D, 16, cache, seed=8, window=60)
    for x in b.views():
        inf = float("nan") if cache == "e4m3" else float("inf")
        x[b.table[0, (q + 90) // 16], :, (q + 90) % 16:] = float("nan")       # past the end
        x[b.table[0, 0], :, 3] = inf                                          # seen by no row or the first ones
        key = q + 88                                                          # seen by the last two rows
        x[b.table[0, key // 16], 0, key % 16, 1] = -inf
        x[b.table[0, key // 16], 0, key % 16, 2] = inf
        x[b.table[0, key // 16], 1, key % 16, D - 1] = float("nan")
    unused = [p for p in range(b.pages) if p not in set(b.table[0])]
    for x in b.views():
        for p in unused:
            x[p] = float("nan")
    o, lse, _, _ = run(L, b)
    ro, rl, to, tl = clean.reference()
    got = o.cpu().to(torch.float64).numpy()
    hidden = np.array([not any(b.limits(0, i)[0] <= j < b.limits(0, i)[1] for j in (3, q + 88)) for i in range(q)])
    assert hidden.any()
    assert np.all(np.abs(got - ro)[hidden] <= to[hidden])
    assert np.all(np.abs(lse.cpu().numpy() - rl)[hidden] <= tl[hidden])
    seen = ~hidden
    assert not np.isfinite(got[seen]).all()


def test_infinite_values_seen(L):
    """An infinite value reaches the rows that see it, at its element only."""
    for q in (2, 40):
        b = R.Batch([q], [q + 60], 2, 1, 64, 16, "bf16", seed=8)
        _, v = b.views()
        key = q + 59                                                          # the last row's own
        v[b.table[0, key // 16], 0, key % 16, 5] = float("inf")
        v[b.table[0, key // 16], 0, key % 16, 6] = -float("inf")
        o, _, _, _ = run(L, b)
        got = o.float().cpu().numpy()
        assert np.isposinf(got[-1, :, 5]).all() and np.isneginf(got[-1, :, 6]).all()
        assert np.isfinite(np.delete(got[-1], (5, 6), axis=1)).all() and np.isfinite(got[:-1]).all()


def test_large_scores(L):
    """Scores far beyond exp's range, of both signs."""
    b = R.Batch([1, 40], [500, 100], 4, 2, 64, 16, "bf16", seed=8)
    o, lse, _, _ = run(L, b, scale=40.0)
    check(b, o, lse, b.reference(scale=40.0))


def test_far_pages(L):
    """Pages beyond 2^32 bytes and elements."""
    D, page, hkv = 256, 1024, 4
    pages = (1 << 32) // (page * D * hkv) + 2
    b = R.Batch([1, 20], [100, 60], 8, hkv, D, page, "e4m3", seed=8)
    k = torch.zeros((pages, hkv, page, D), dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros_like(k)
    far = {int(b.table[0, 0]): pages - 1, int(b.table[1, 0]): pages - 2}
    for a, p in far.items():
        k[p], v[p] = b.k_store[a].cuda(), b.v_store[a].cuda()
    cache = L.KvCache(k, v, b.k_scale.cuda(), b.v_scale.cuda())
    table = np.array([[pages - 1], [pages - 2]])
    meta = L.lora_prepare_attn_meta(dev(b.q_start), dev(b.kv_len), dev(table), cache, 8, b.T)
    lse = torch.empty((b.T, 8), device="cuda")
    o, _ = L.lora_attention(meta, b.q.cuda(), cache, lse=lse)
    check(b, o, lse, b.reference())


def test_results_repeat(L):
    """The same call gives the same bits, whatever the workspace held."""
    b = R.Batch([1, 1, 60], [4000, 3, 900], 8, 2, 128, 16, "bf16", seed=1, groups=[0, 2], group_len=[3])
    first = run(L, b)[:2]
    again = run(L, b, max_q_len=b.T)[:2]
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_graph_replays(L):
    """Metadata, append and attention captured once; lengths, pages and rows change
    between the replays, with eager work in between."""
    b = R.Batch([1] * 9, [1000] * 9, 8, 2, 128, 16, "bf16", seed=1)
    d = Dev(L, b)
    T, w = b.T, 12 * 128
    qkv = torch.zeros((T, w), dtype=torch.bfloat16, device="cuda")
    slot = torch.zeros(T, dtype=torch.int64, device="cuda")
    q = torch.zeros((T, 8 * 128), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((T, 8), device="cuda")
    mws = torch.empty(L.lora_attn_meta_workspace_bytes(*d.args, d.cache, 8, T), dtype=torch.uint8, device="cuda")
    ws = torch.empty(L.lora_attention_workspace_bytes(d.meta(L)), dtype=torch.uint8, device="cuda")

    def step():
        L.lora_cache_append(qkv, d.cache, slot, q)
        meta = d.meta(L, workspace=mws)
        L.lora_attention(meta, q, d.cache, out, lse=lse, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    r = np.random.default_rng(0)
    for rep in range(4):
        kv = r.integers(1, 1000, 9)
        d.args[1].copy_(dev(kv))
        table = d.args[2].cpu().numpy()
        slot.copy_(torch.tensor([table[n, (kv[n] - 1) // 16] * 16 + (kv[n] - 1) % 16 for n in range(9)]))
        qkv.copy_(torch.randn((T, w), device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone(), d.k.clone()
        out.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse) and torch.equal(got[2], d.k), rep


def test_streams(L):
    """Two streams share one metadata, with workspaces of their own."""
    b = R.Batch([1, 30, 1], [2000, 500, 700], 8, 2, 128, 16, "bf16", seed=1)
    d = Dev(L, b)
    meta = d.meta(L)
    ref = L.lora_attention(meta, d.q, d.cache)
    torch.cuda.synchronize()
    outs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append([L.lora_attention(meta, d.q, d.cache) for _ in range(3)])
    torch.cuda.synchronize()
    assert all(torch.equal(ref, o) for os in outs for o in os)


def test_after_the_adapters_delta(L):
    """The path of a layer: delta into q | k | v, append, attention."""
    r = np.random.Generator(np.random.PCG64(5))
    b = R.Batch([1, 1, 30, 1], [90, 33, 30, 200], 8, 2, 64, 16, "bf16", seed=6)
    T, width, rank = b.T, 12 * 64, 16
    t = lambda *s: torch.from_numpy((0.2 * r.standard_normal(s)).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    x, y = t(T, 256), t(T, width)
    A = [t(3, 256, rank) for _ in range(3)]
    B = [t(3, rank, n * 64) for n in (8, 2, 2)]
    slots = torch.tensor([0] * 1 + [-1] + [2] * 30 + [1], dtype=torch.int32, device="cuda")
    d = Dev(L, b)
    slot = torch.tensor([int(b.table[n, p // 16]) * 16 + p % 16 for n in range(b.N)
                         for p in range(b.kv_len[n] - b.q_len[n], b.kv_len[n])], device="cuda")
    L.lora_apply(L.lora_prepare_meta(slots, 3), x, A, B, [0, 512, 640], y)
    q = torch.empty((T, 512), dtype=torch.bfloat16, device="cuda")
    L.lora_cache_append(y, d.cache, slot, q)
    lse = torch.empty((T, 8), device="cuda")
    o, _ = L.lora_attention(d.meta(L), q, d.cache, lse=lse)
    b.q = q.cpu().view(T, 8, 64)
    b.k_store, b.v_store = d.k.cpu(), d.v.cpu()
    assert torch.equal(b.q, y[:, :512].cpu().view(T, 8, 64))
    check(b, o.view(T, 8, 64), lse, b.reference())
