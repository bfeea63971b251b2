"""lora_cache_append and lora_attention where earlier tests do not reach: scores far
apart on tiles without hidden keys, groups in batches with bad bounds.  Against the
float64 form."""
import numpy as np
import pytest
import torch

import attn_ref as R
from test_gpu_14_attention import Dev, check, dev, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import segmented_gather_rank_amd as lib
    return lib


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", [0.0, 3000.0])
def test_large_scores_of_full_tiles(L, D, cache, cap):
    """Scores hundreds apart, most of each in the last dimensions, on a prompt and on
    decode tokens whose tiles of keys are seen by every row."""
    b = R.Batch([200, 1, 1], [900, 1500, 200], 2, 1, D, 16, cache, seed=D)
    if cache == "e4m3":
        b.k_scale = torch.ones(1)
    k, _ = b.views()
    k[..., D - 16:] = (k[..., D - 16:].float() * 8).to(k.dtype)
    b.q[..., D - 16:] *= 4
    o, lse, _, _ = run(L, b, scale=1.0, cap=cap)
    out, rl, out_tol, lse_tol = b.reference(scale=1.0, cap=cap)
    assert np.ptp(rl) > 100
    # weights that fp32 cannot hold are zeros: each is off by less than its smallest
    # normal number, times a value
    out_tol = out_tol + max(b.kv_len) * np.finfo(np.float32).tiny * float(b.v_store.float().abs().max())
    check(b, o, lse, (out, rl, out_tol, lse_tol))


def poisoned(L, b, d, **kw):
    """Metadata and attention in memory full of garbage: out, lse, info."""
    need = L.lora_attn_meta_workspace_bytes(*d.args, d.cache, b.hq, b.T, len(b.group_len or []))
    meta = d.meta(L, workspace=torch.full((need,), 0x5a, dtype=torch.uint8, device="cuda"), **kw)
    ws = torch.full((max(16, L.lora_attention_workspace_bytes(meta)),), 255, dtype=torch.uint8, device="cuda")
    hold = torch.full((b.T + 2, b.hq, b.D), 9.0, dtype=d.q.dtype, device="cuda")
    lse = torch.full((b.T, b.hq), 5.0, device="cuda")
    L.lora_attention(meta, d.q, d.cache, hold[1:-1], lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert torch.all(hold[0] == 9) and torch.all(hold[-1] == 9)
    return hold[1:-1], lse, meta.tensors()["info"].cpu().tolist()


def rows_of(b, seqs):
    return [t for n in seqs for t in range(b.q_start[n], b.q_start[n + 1])]


def check_rows(b, out, lse, ref, rows):
    check(b, out[rows], lse[rows], tuple(r[rows] for r in ref))


@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("ends,good", [((0, 1, 2, 900), (0, 1)), ((0, 1, 2, -4), (0, 1))])
def test_group_whose_last_sequence_leaves_the_batch(L, cache, ends, good):
    b = R.Batch([1, 1, 1], [80, 90, 100], 8, 2, 64, 16, cache, seed=2, groups=[0, 3], group_len=[70])
    d = Dev(L, b)
    d.args = (dev(np.array(ends)), d.args[1], d.args[2])
    out, lse, info = poisoned(L, b, d, max_q_len=3)
    assert info[2] == 1 and info[3] == 1
    check_rows(b, out, lse, b.reference(), rows_of(b, good))


def test_good_groups_beside_bad_ones(L):
    """Bounds of groups out of order: the groups beside them are served, their keys
    read once, over more groups than the plan has threads."""
    n = 2100
    starts = list(range(0, n + 1, 2))
    b = R.Batch([1] * n, [40 + i % 30 for i in range(n)], 2, 1, 16, 16, "bf16", seed=7, groups=starts,
                group_len=[16 + i % 20 for i in range(len(starts) - 1)])
    ref = b.reference()
    for spoiled in ([], [1], [0, 3, 70, 71, 300, 1049], list(range(10, 1045, 7))):
        got = np.array(starts)
        got[spoiled] = [10 ** 6 if i % 2 else -3 for i in range(len(spoiled))]
        b.groups = got
        d = Dev(L, b)
        out, lse, info = poisoned(L, b, d)
        bad = {g for s in spoiled for g in (s - 1, s) if 0 <= g < len(starts) - 1}
        assert info[2] == 0 and info[3] == len(bad)
        # every sequence of a good group is joined from the group's keys (others may be
        # where their keys are cut)
        assert info[4] >= n - 2 * len(bad)
        check(b, out, lse, ref)


@pytest.mark.parametrize("cache,hq,hkv", [("bf16", 8, 2), ("e4m3", 32, 8), ("f32", 8, 2), ("bf16", 6, 6)])
@pytest.mark.parametrize("most", [1, 2, 5, 100])
@pytest.mark.parametrize("grouped", [False, True])
def test_rows_of_bad_sequences(L, cache, hq, hkv, most, grouped):
    """More query tokens than stated, more keys than the table holds, fewer than
    queries, a negative count: zeros and -inf for those tokens, the others as ever."""
    q, kv = [1, 20, 1, 1, 2, 40, 1, 3], [50, 60, 70, 33, 45, 90, 1, 64]
    groups = dict(groups=[2, 4, 8], group_len=[33, 1]) if grouped else {}
    b = R.Batch(q, kv, hq, hkv, 64, 16, cache, seed=3, **groups)
    d = Dev(L, b)
    kv_dev = np.array(kv)
    kv_dev[2], kv_dev[5], kv_dev[6] = 10 ** 6, 39, -1
    d.args = (d.args[0], dev(kv_dev), d.args[2])
    bad = tuple(n for n in range(len(q)) if n in (2, 5, 6) or q[n] > most)
    out, lse, info = poisoned(L, b, d, max_q_len=most)
    assert info[2] == len(bad)
    check(b, out, lse, b.reference(bad_seqs=bad))


@pytest.mark.parametrize("most", [1, 30])
def test_rows_of_a_sequence_that_leaves_the_batch(L, most):
    """Its tokens inside the batch get zeros, those of no sequence are not written."""
    b = R.Batch([1, 1, 1, 25], [50, 60, 70, 40], 8, 2, 64, 16, "bf16", seed=3)
    d = Dev(L, b)
    for ends, bad, outside in (([0, 1, 2, 3, 900], [3], []), ([1, 2, 3, 3, 3], [], [0] + list(range(3, 28)))):
        d.args = (dev(np.array(ends)), d.args[1], d.args[2])
        out, lse, info = poisoned(L, b, d, max_q_len=most)
        assert info[2] == len(bad)
        if bad:
            check(b, out, lse, b.reference(bad_seqs=(3,)))
        assert torch.all(out[outside] == 9) and torch.all(lse[outside] == 5)


def owners(starts, kv, most, T):
    """The header's rules: which sequences are good, and of every token its sequence,
    -1 if it is in none, -2 if in bad ones only."""
    good, owner, end = [], [-1] * T, 0
    for n, (s, e) in enumerate(zip(starts, starts[1:])):
        ok = 0 <= s <= e <= T and e - s <= most and e - s <= kv[n]
        good.append(ok and (s == e or s >= end))
        end = max(end, e) if ok else end
        for t in range(max(s, 0), min(e, T)):
            owner[t] = n if good[-1] else (-2 if owner[t] == -1 else owner[t])
    return good, owner


STARTS = [[0, 2, 1, 6, 8], [-5, 2, 4, 6, 8], [0, 2, 4, 6, 900], [0, 900, 4, 6, 8], [8, 8, 8, 8, 8], [3, 2, 1, 0, -1],
          [0, 5, 3, 8, 8], [4, 8, 0, 4, 2], [0, 8, 1, 3, 7], [6, 8, 8, 0, 6], [2, 4, 3, 5, -2 ** 31]]


@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("starts", STARTS, ids=str)
@pytest.mark.parametrize("most", [1, 2, 8])
@pytest.mark.parametrize("groups", [None, ([0, 2, 4], [30, 9])], ids=["alone", "groups"])
def test_bounds_out_of_order(L, cache, starts, most, groups):
    kv = [40, 50, 60, 70]
    b = R.Batch([2, 2, 2, 2], kv, 4, 2, 64, 16, cache, seed=3)
    good, owner = owners(starts, kv, most, 8)
    b.q_start, b.q_len = np.array(starts), [e - s if ok else 0 for s, e, ok in zip(starts, starts[1:], good)]
    if groups:
        b.groups, b.group_len = groups
        b.share()
    d = Dev(L, b)
    out, lse, info = poisoned(L, b, d, max_q_len=most)
    ref = b.reference()
    assert info[2] == 4 - sum(good)
    inside = [t for t in range(8) if owner[t] != -1]
    outside = [t for t in range(8) if owner[t] == -1]
    check_rows(b, out, lse, ref, inside)
    assert torch.all(out[outside] == 9) and torch.all(lse[outside] == 5)


def test_many_bounds_out_of_order(L):
    """More sequences and more tokens than the plan has threads."""
    r = np.random.default_rng(3)
    N, T = 1500, 2600
    base = np.sort(r.integers(0, T, N + 1))
    for wild in (1, 40, N + 1):
        starts = base.copy()
        at = r.choice(N + 1, wild, replace=False)
        starts[at] = r.integers(-5, T + 50, wild)
        starts, kv = starts.tolist(), [int(x) for x in r.integers(1, 60, N)]
        b = R.Batch([1] * T, [1] * T, 2, 1, 16, 16, "bf16", seed=wild)      # tokens and their queries
        c = R.Batch([0] * N, kv, 2, 1, 16, 16, "bf16", seed=wild + 1)       # the cache
        good, owner = owners(starts, kv, T, T)
        c.q, c.T = b.q, T
        c.q_start, c.q_len = np.array(starts), [e - s if ok else 0 for s, e, ok in zip(starts, starts[1:], good)]
        d = Dev(L, c)
        out, lse, info = poisoned(L, c, d, max_q_len=T)
        assert info[2] == N - sum(good)
        check_rows(c, out, lse, c.reference(), [t for t in range(T) if owner[t] != -1])
        outside = [t for t in range(T) if owner[t] == -1]
        assert torch.all(out[outside] == 9) and torch.all(lse[outside] == 5)


@pytest.mark.parametrize("q", [1, 40])
def test_as_many_keys_as_a_table_holds(L, q):
    """2^31 - 2^16 keys of one sequence, two pages over and over: the first half of
    them one page, the second half the other."""
    D, page, n = 8, 65536, 32767
    r = np.random.default_rng(5)
    k, v = (r.standard_normal((2, 1, page, D)).astype(np.float32) for _ in range(2))
    v[1] += 4
    k, v = (torch.from_numpy(x).to(torch.bfloat16) for x in (k, v))
    table = np.full((1, n), 1, np.int32)
    table[0, :n // 2] = 0
    cache = L.KvCache(k.cuda(), v.cuda())
    qs = torch.from_numpy(r.standard_normal((q, 1, D)).astype(np.float32)).to(torch.bfloat16)
    meta = L.lora_prepare_attn_meta(dev(np.array([0, q])), dev(np.array([n * page])), dev(table), cache, 1, q, causal=False)
    lse = torch.empty((q, 1), device="cuda")
    out, _ = L.lora_attention(meta, qs.cuda(), cache, lse=lse)
    kk, vv = (x.double().numpy()[:, 0] for x in (k, v))
    x = np.einsum("pjd,qd->qpj", kk, qs.double().numpy()[:, 0]) / np.sqrt(D)
    w = np.exp(x) * np.array([n // 2, n - n // 2])[:, None]
    total = w.sum((1, 2))
    want = np.einsum("qpj,pjd->qd", w, vv) / total[:, None]
    spread = np.einsum("qpj,pjd->qd", w, np.abs(vv)) / total[:, None]
    # a lane adds a quarter of a slice's (part's) keys one after the other in fp32
    keys = int(meta.tensors()["info"][6 if q == 1 else 7])
    sums = min(keys, n * page) / 4 * R.F32_HALF
    assert np.all(np.abs(lse.cpu().double().numpy()[:, 0] - np.log(total)) <= sums + 1e-3)
    assert np.all(np.abs(out.cpu().double().numpy()[:, 0] - want) <= (2 * sums + 2 * R.BF16_HALF + 1e-3) * spread)


@pytest.mark.parametrize("cap", [1e-40, 1e-3, 0.5, 30.0, 1e4, 1e6, 1e8, 1e30, 3e38])
@pytest.mark.parametrize("cache,tokens", [("bf16", 1), ("e4m3", 1), ("f32", 1), ("bf16", 300), ("e4m3", 300)])
def test_capped_score_alone(L, cap, cache, tokens):
    """Every row sees one key, so that its log-sum is its capped score: small and large
    against the cap, on both sides of a quarter of it."""
    D, T, page = 16, 300, 16
    x = np.concatenate([np.geomspace(1e-4, 3e4, 120), cap * np.geomspace(1e-3, 20, 60), cap * np.linspace(0.2, 0.3, 90)])
    x = np.concatenate([x, -x])[np.linspace(0, 2 * len(x) - 1, T).astype(int)]
    x[0] = 0
    scale = 0.731
    q_type = torch.float32 if cache == "f32" else torch.bfloat16
    q = torch.zeros((T, 1, D), dtype=q_type)
    q[:, 0, 3] = torch.from_numpy(np.clip(x / scale, -3e38, 3e38)).to(q_type)
    k = torch.zeros((T // page + 1, 1, page, D), dtype=torch.float32)
    k[..., 3] = 1
    k = k.to({"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}[cache])
    seqs = T // tokens                       # of one token each, or one of all
    kv = L.KvCache(k.cuda(), k.clone().cuda())
    at = np.arange(T)
    table = np.tile(np.arange(T // page + 1), (seqs, 1))
    meta = L.lora_prepare_attn_meta(dev(np.arange(seqs + 1) * tokens), dev(np.full(seqs, T)), dev(table), kv, 1, T,
                                    max_q_len=tokens, causal=False, key_lo=dev(at), key_hi=dev(at + 1))
    lse = torch.empty((T, 1), device="cuda")
    out, _ = L.lora_attention(meta, q.cuda(), kv, scale=scale, cap=cap, lse=lse)
    x = q.double().numpy()[:, 0, 3] * float(np.float32(scale))
    want = float(np.float32(cap)) * np.tanh(x / float(np.float32(cap)))
    got = lse.cpu().double().numpy()[:, 0]
    # every operation on the score off by half a step or one, and tanh by 5 half steps of
    # 1 where it is at least a quarter: 32 half steps of the result
    bound = 32 * R.F32_HALF * np.abs(want) + np.finfo(np.float32).tiny
    assert np.all(np.abs(got - want) <= bound), (x[np.abs(got - want) > bound], got[np.abs(got - want) > bound])
    assert torch.equal(out[:, 0, 3].cpu(), torch.ones(T, dtype=q_type))


@pytest.mark.parametrize("cap", [1e4, 1e8, 1e30])
@pytest.mark.parametrize("cache", ["bf16", "f32", "e4m3"])
def test_cap_far_above_the_scores(L, cap, cache):
    """Such a cap changes nothing: the bounds are those without one."""
    b = R.Batch([1, 50, 2], [300, 120, 64], 8, 4, 128, 16, cache, seed=2)
    o, lse, _, _ = run(L, b, cap=cap)
    check(b, o, lse, b.reference())


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_memory_of_another_stream(L, raw):
    """With a stream given, metadata, outputs and workspaces that the call allocates are
    neither still in use on the current stream nor reused there while it runs."""
    b = R.Batch([1, 30, 1], [2000, 500, 700], 8, 2, 128, 16, "bf16", seed=1)
    d = Dev(L, b)
    want = L.lora_attention(d.meta(L), d.q, d.cache)
    need = L.lora_attention_workspace_bytes(d.meta(L))
    busy = torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    stream = s.cuda_stream if raw else s
    for size in (need, 1 << 16, 1 << 14):
        # the current stream: work that is still to write to memory it has freed
        for _ in range(20):
            busy.mul_(1.0001)
        held = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        del held
        # the other one: the call behind other work, and its memory freed at once
        with torch.cuda.stream(s):
            other = torch.ones((4096, 4096), device="cuda")
            for _ in range(20):
                other.mul_(1.0001)
        meta = d.meta(L, stream=stream)
        out = L.lora_attention(meta, d.q, d.cache, stream=stream)
        for _ in range(4):
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_append_of_more_rows_than_one_launch(L):
    """More tokens than a launch of 256 threads each may hold (2^24 - 1)."""
    T, D = (1 << 24) + 5, 8
    x = torch.zeros((T, 3 * D), dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, (1 << 24) - 1, 1 << 24, T - 1]
    x[rows] = torch.randn((len(rows), 3 * D), device="cuda").to(torch.bfloat16)
    slot = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    slot[rows] = torch.arange(len(rows), device="cuda")
    slot[[5, T - 3]] = -2                                   # bad
    k = torch.zeros((2, 1, 4, D), dtype=torch.bfloat16, device="cuda")
    v, q = torch.zeros_like(k), torch.full((T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lora_cache_append(x, L.KvCache(k, v), slot, q, num_bad=bad)
    assert int(bad) == 2
    assert torch.equal(k.view(-1, D), x[rows, D:2 * D]) and torch.equal(v.view(-1, D), x[rows, 2 * D:])
    assert torch.equal(q[rows], x[rows, :D]) and torch.all(q[[5, T - 3]] == 7)
    q[[5, T - 3]] = 0
    q[rows] = 0
    assert not q.any()


@pytest.mark.parametrize("groups", [False, True])
def test_tokens_without_sequences(L, groups):
    """A batch of no sequences: its tokens are outside every one, and not written."""
    b = R.Batch([1] * 5, [3] * 5, 4, 2, 64, 16, "bf16", seed=3)
    d = Dev(L, b)
    d.args = (dev(np.array([0])), dev(np.zeros(0)), torch.empty((0, 3), dtype=torch.int32, device="cuda"))
    if groups:
        d.kw.update(group_start=dev(np.array([0])), group_len=dev(np.zeros(0)))
    meta = d.meta(L, max_q_len=1, workspace=torch.full((1 << 20,), 0x5a, dtype=torch.uint8, device="cuda"))
    hold, lse = torch.full((5, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((5, 4), 5.0, device="cuda")
    L.lora_attention(meta, d.q, d.cache, hold, lse=lse)
    torch.cuda.synchronize()
    assert torch.all(hold == 9) and torch.all(lse == 5)
    t = meta.tensors()
    assert t["info"].tolist()[:6] == [0] * 6
    assert torch.equal(t["limits"].cpu(), torch.tensor([[0, 0, 0, -1]] * 5, dtype=torch.int32))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("q,kv", [([1] * 8, [5, 20, 33, 64, 150, 300, 700, 1500]), ([2, 4, 3], [90, 40, 600])])
def test_weights_of_few_rows(L, cache, q, kv):
    """Weights beyond bf16: an output that cancels is still right to its own rounding."""
    b = R.Batch(q, kv, 8, 2, 64, 16, cache, seed=12)
    o, lse, _, _ = run(L, b)
    out, rl, _, lse_tol = b.reference()
    b.v_store = b.v_store.float().abs().to(b.v_store.dtype)
    spread = b.reference()[0]                       # sum of weight * |v|
    # a weight: 2^-16 and twice its score's error (which the log-sum's bound holds), and as
    # many fp32 half steps as there are keys in a lane's sum; then one rounding
    w = 2.0 ** -16 + 2 * lse_tol[..., None] + max(kv) / 4 * R.F32_HALF
    tol = w * spread + R.BF16_HALF * (np.abs(out) + w * spread)
    check(b, o, lse, (out, rl, tol, lse_tol))
