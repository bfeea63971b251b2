"""lora_int8_matmul against exact integer sums: row counts from one to many, odd sizes,
ragged experts, strides, the largest sums, graphs and streams."""
import numpy as np
import pytest
import torch

import base_ref as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def L():
    import segmented_gather_rank_amd as lib
    return lib


def made(g, rows, d_in, d_out, experts=None, bias=False):
    byte = lambda *n: torch.randint(-127, 128, n, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    lead = () if experts is None else (experts,)
    x, xs = byte(rows, d_in), 0.01 + torch.rand(rows, generator=g, device="cuda")
    w, ws = byte(*lead, d_out, d_in), 1e-3 * torch.rand((*lead, d_out), generator=g, device="cuda")
    return x, xs, w, ws, torch.randn((*lead, d_out), generator=g, device="cuda") if bias else None


def dense(L, x, xs, w, ws, b, dtype, **kw):
    y = L.lora_int8_matmul(x, xs, L.Int8Weight(w, ws, bias=b), dtype=dtype, **kw)
    torch.cuda.synchronize()
    n = len(x)
    want, bound = R.int8_matmul(x, xs, w, ws, b, np.zeros(n, np.int64), np.arange(n), dtype)
    assert y.dtype == dtype
    R.near(y, want, bound, f"{tuple(x.shape)} x {tuple(w.shape)}")
    return y


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 32, 33, 64, 65, 100, 128, 129, 250, 257, 511])
@pytest.mark.parametrize("d_in,d_out", [(16, 8), (128, 16), (144, 40), (1008, 264), (2048, 128), (4112, 72)])
def test_dense(L, rows, d_in, d_out):
    g = torch.Generator("cuda").manual_seed(rows + d_in)
    args = made(g, rows, d_in, d_out, bias=rows % 2 == 0)
    for dtype in DTYPES:
        dense(L, *args, dtype)


@pytest.mark.parametrize("rows,d_in,d_out", [(300, 512, 1000), (513, 1152, 776), (1000, 256, 2056), (777, 4096, 520),
                                             (2049, 144, 256), (1, 14336, 4096), (16, 4096, 6144), (40, 2048, 4104), (256, 4096, 1024)])
def test_larger(L, rows, d_in, d_out):
    g = torch.Generator("cuda").manual_seed(rows)
    args = made(g, rows, d_in, d_out, bias=True)
    for dtype in DTYPES:
        dense(L, *args, dtype)


@pytest.mark.parametrize("rows", [1, 20, 300])
def test_largest_sums(L, rows):
    """The longest rows, of the largest magnitudes: sums next to 2^31, and of both signs."""
    d_in = 131056
    x = torch.full((rows, d_in), -128, dtype=torch.int8, device="cuda")
    w = torch.full((24, d_in), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    x[rows // 2, ::2] = 127
    one = torch.ones(rows, device="cuda")
    dense(L, x, one, w, torch.ones(24, device="cuda"), None, torch.float32)


@pytest.mark.parametrize("rows", [5, 70, 300])
def test_scales_that_are_not_finite(L, rows):
    """A row that could not be rounded (scale NaN) is NaN, the others are as they were; zeros stay zeros."""
    g = torch.Generator("cuda").manual_seed(rows)
    x, xs, w, ws, b = made(g, rows, 256, 64)
    xs[rows // 2] = torch.nan
    xs[0] = 0
    for dtype in DTYPES:
        y = dense(L, x, xs, w, ws, None, dtype)
        assert y[rows // 2].isnan().all() and (y[0] == 0).all() and not y[1:rows // 2].isnan().any()


@pytest.mark.parametrize("rows", [3, 100, 400])
def test_strides(L, rows):
    """Parts of wider matrices, on both sides of a wider output's other columns."""
    g = torch.Generator("cuda").manual_seed(rows)
    x, xs, w, ws, b = made(g, rows, 1200, 640, bias=True)
    for dtype in DTYPES:
        y = torch.full((rows, 400), 5.0, dtype=dtype, device="cuda")
        part = y[:, 16:16 + 264]
        wide, thin = x[:, 48:48 + 912], w[100:364, 128:128 + 912]
        dense(L, wide, xs, thin, ws[100:364].contiguous(), b[100:364].contiguous(), dtype, out=part)
        assert (y[:, :16] == 5).all() and (y[:, 280:] == 5).all()


def routed(T, topk, E, seed, skew=0.0):
    """Expert ids [T][topk], distinct in a row; with skew the first experts take most of them."""
    g = np.random.Generator(np.random.PCG64(seed))
    v = g.gumbel(size=(T, E)) - skew * np.arange(E)
    return np.argsort(-v, axis=1)[:, :topk].astype(np.int32)


def by_expert(L, T, topk, E, local, first, d_in, d_out, per_pair, dtype, skew=0.0, seed=0, bias=False):
    g = torch.Generator("cuda").manual_seed(seed)
    ids = routed(T, topk, E, seed, skew)
    emap = np.full(E, -1, np.int32)
    emap[first:first + local] = np.arange(local)
    expert = emap[ids].reshape(-1)
    x, xs, w, ws, b = made(g, T * topk if per_pair else T, d_in, d_out, local, bias)
    meta = L.lora_prepare_moe_meta(torch.from_numpy(ids).cuda(), torch.zeros(T, dtype=torch.int32, device="cuda"), 1, E, local,
                                   torch.from_numpy(emap).cuda())
    if per_pair:
        meta = meta.with_x_row_div(1)
    pairs = T * topk
    y = torch.full((pairs, d_out), 7.0, dtype=dtype, device="cuda")
    L.lora_int8_matmul(x, xs, L.Int8Weight(w, ws, bias=b), out=y, meta=meta)
    torch.cuda.synchronize()
    source = np.arange(pairs) if per_pair else np.arange(pairs) // topk
    want, bound = R.int8_matmul(x, xs, w, ws, b, expert, source, dtype)
    away = torch.from_numpy(expert < 0).cuda()
    assert (y[away] == 7).all()
    here = expert >= 0
    R.near(y[torch.from_numpy(here).cuda()], want[here], bound[here], "by expert")


@pytest.mark.parametrize("per_pair", [False, True])
@pytest.mark.parametrize("T,topk,E,local,first,d_in,d_out,skew", [
    (1, 1, 1, 1, 0, 64, 16, 0), (1, 8, 256, 256, 0, 512, 128, 0), (1, 2, 8, 1, 7, 144, 40, 0), (20, 2, 8, 8, 0, 1008, 264, 0),
    (256, 8, 64, 8, 8, 512, 72, 0), (600, 4, 6, 6, 0, 272, 520, 0), (333, 3, 16, 16, 0, 640, 136, 0.7),
    (1500, 2, 4, 3, 1, 256, 264, 0.5), (70, 1, 70, 70, 0, 128, 24, 0), (900, 1, 2, 1, 0, 384, 300 // 8 * 8, 2.0),
    (40, 8, 1000, 1000, 0, 64, 16, 0)])
def test_by_expert(L, T, topk, E, local, first, d_in, d_out, skew, per_pair):
    for dtype in DTYPES:
        by_expert(L, T, topk, E, local, first, d_in, d_out, per_pair, dtype, skew, seed=T + E, bias=T % 2 == 0)


def test_no_row_is_local(L):
    by_expert(L, 50, 2, 8, 2, 6, 128, 64, False, torch.bfloat16, skew=50.0, seed=1)


def test_metadata_by_slot(L):
    """Any metadata groups the rows: here one matrix for each slot, and rows without one."""
    g = torch.Generator("cuda").manual_seed(4)
    slots = torch.randint(-1, 5, (700,), generator=g, device="cuda", dtype=torch.int32)
    slots[:300] = 2
    x, xs, w, ws, b = made(g, 700, 528, 200, 5, True)
    y = torch.full((700, 200), 7.0, dtype=torch.float32, device="cuda")
    L.lora_int8_matmul(x, xs, L.Int8Weight(w, ws, bias=b), out=y, meta=L.lora_prepare_meta(slots, 5))
    expert = slots.cpu().numpy()
    want, bound = R.int8_matmul(x, xs, w, ws, b, expert, np.arange(700), torch.float32)
    here = expert >= 0
    R.near(y[slots >= 0], want[here], bound[here])
    assert (y[slots < 0] == 7).all()


def test_expert_stride_beyond_32_bits(L):
    """Experts far apart in one buffer: offsets past 2^31 and 2^32 bytes."""
    g = torch.Generator("cuda").manual_seed(9)
    stride = (1 << 32) // 3 // 16 * 16 + 16
    buf = torch.empty(3 * stride + 4096 * 128, dtype=torch.int8, device="cuda")
    w = buf.as_strided((4, 128, 256), (stride, 256, 1))
    w.copy_(torch.randint(-127, 128, (4, 128, 256), generator=g, device="cuda", dtype=torch.int8))
    slots = torch.randint(0, 4, (300,), generator=g, device="cuda", dtype=torch.int32)
    x, xs, _, _, _ = made(g, 300, 256, 8)
    ws = torch.rand((4, 128), generator=g, device="cuda")
    y = L.lora_int8_matmul(x, xs, L.Int8Weight(w, ws), meta=L.lora_prepare_meta(slots, 4), dtype=torch.float32)
    want, bound = R.int8_matmul(x, xs, w, ws, None, slots.cpu().numpy(), np.arange(300), torch.float32)
    R.near(y, want, bound)


def test_rows_beyond_32_bits(L):
    """x rows and y rows far apart: offsets past 2^32 bytes; the other columns are not touched."""
    g = torch.Generator("cuda").manual_seed(10)
    rows, far = 300, 1 << 24
    x, xs, w, ws, b = made(g, rows, 256, 64, bias=True)
    wide = torch.zeros((rows, far), dtype=torch.int8, device="cuda")
    wide[:, :256] = x
    out = torch.zeros((rows, far), dtype=torch.bfloat16, device="cuda")
    dense(L, wide[:, :256], xs, w, ws, b, torch.bfloat16, out=out[:, :64])
    assert int(out[:, 64:].count_nonzero()) == 0
    slots = torch.randint(-1, 3, (rows,), generator=g, device="cuda", dtype=torch.int32)
    slots[:150] = 1
    x3, _, w3, ws3, _ = made(g, rows, 256, 64, 3)
    y = torch.zeros((rows, 64), dtype=torch.float32, device="cuda")
    L.lora_int8_matmul(wide[:, :256], xs, L.Int8Weight(w3, ws3), out=y, meta=L.lora_prepare_meta(slots, 3))
    expert = slots.cpu().numpy()
    want, bound = R.int8_matmul(x, xs, w3, ws3, None, expert, np.arange(rows), torch.float32)
    R.near(y[slots >= 0], want[expert >= 0], bound[expert >= 0])


@pytest.mark.parametrize("T", [4, 200])
def test_two_graphs_and_a_stream(L, T):
    """Two captured graphs that share a workspace, replayed between eager calls, and a call on another stream."""
    g = torch.Generator("cuda").manual_seed(T)
    ids = torch.from_numpy(routed(T, 2, 6, T)).cuda()
    meta = L.lora_prepare_moe_meta(ids, torch.zeros(T, dtype=torch.int32, device="cuda"), 1, 6, 6)
    sets = []
    for seed in range(2):
        x, xs, w, ws, b = made(g, T, 512, 256, 6)
        sets.append((x, xs, L.Int8Weight(w, ws), torch.zeros((2 * T, 256), dtype=torch.bfloat16, device="cuda")))
    space = torch.empty(max(16, max(L.lora_int8_matmul_workspace_bytes(2 * T, s[2]) for s in sets)), dtype=torch.uint8, device="cuda")
    call = lambda s, **kw: L.lora_int8_matmul(s[0], s[1], s[2], out=s[3], meta=meta, workspace=space, **kw)  # noqa: E731
    want = []
    for s in sets:
        want.append(call(s).clone())
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(s)
    for _ in range(4):
        for s, graph, y in zip(sets, graphs, want):
            s[3].zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(s[3], y)
            assert torch.equal(call(s), y)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        sets[0][3].zero_()
        torch.cuda.synchronize()
        call(sets[0], stream=stream)
        side.synchronize()
        assert torch.equal(sets[0][3], want[0])


@pytest.mark.parametrize("T,used", [(1500, 3), (2000, 300), (4000, 9)])
def test_keys_beyond_256(L, T, used):
    """Several hundred keys, of which few hold many rows or many hold few."""
    g = torch.Generator("cuda").manual_seed(T)
    keys = 300 if used != 9 else 1023
    x, xs, w, ws, b = made(g, T, 272, 264, keys, True)
    of = torch.randperm(keys, generator=g, device="cuda")[:used].int()
    slots = of[torch.randint(0, used, (T,), generator=g, device="cuda")]
    slots[::7] = -1
    expert = slots.cpu().numpy()
    here = expert >= 0
    for dtype in DTYPES:
        y = torch.full((T, 264), 7.0, dtype=dtype, device="cuda")
        L.lora_int8_matmul(x, xs, L.Int8Weight(w, ws, bias=b), out=y, meta=L.lora_prepare_meta(slots, keys))
        want, bound = R.int8_matmul(x, xs, w, ws, b, expert, np.arange(T), dtype)
        R.near(y[slots >= 0], want[here], bound[here])
        assert (y[slots < 0] == 7).all()


def test_many_launches(L):
    """So many columns that a launch takes some experts only: each expert as a dense call of its own."""
    g = torch.Generator("cuda").manual_seed(3)
    experts, d_out = 11, 1 << 24
    x, xs, w, ws, _ = made(g, experts, 16, d_out, experts)
    slots = torch.arange(experts, device="cuda", dtype=torch.int32).flip(0).contiguous()
    y = L.lora_int8_matmul(x, xs, L.Int8Weight(w, ws), meta=L.lora_prepare_meta(slots, experts))
    for i in range(experts):
        e = experts - 1 - i
        assert torch.equal(y[i:i + 1], L.lora_int8_matmul(x[i:i + 1], xs[i:i + 1], L.Int8Weight(w[e], ws[e])))
    part = slice(d_out - 64, d_out)
    want, bound = R.int8_matmul(x, xs, w[:, part].contiguous(), ws[:, part].contiguous(), None, slots.cpu().numpy(), np.arange(experts),
                                torch.bfloat16)
    R.near(y[:, part], want, bound)


def test_two_threads(L):
    """Calls of every kernel at once from two threads, each on a stream of its own."""
    import threading
    g = torch.Generator("cuda").manual_seed(12)
    cases = []
    for rows, d_in, d_out in ((3, 256, 64), (200, 256, 640), (900, 256, 2048), (5000, 256, 4096)):
        x, xs, w, ws, b = made(g, rows, d_in, d_out, bias=True)
        weight = L.Int8Weight(w, ws, bias=b)
        cases.append((x, xs, weight, L.lora_int8_matmul(x, xs, weight)))
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                for x, xs, weight, want in cases:
                    y = L.lora_int8_matmul(x, xs, weight)
                    stream.synchronize()
                    if not torch.equal(y, want):
                        wrong.append(tuple(y.shape))

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_experts_side_by_side(L):
    """Experts whose rows lie between each other's, as a transposed [d_out][experts][d_in] holds them."""
    g = torch.Generator("cuda").manual_seed(13)
    for rows, d_in, d_out, experts in ((300, 272, 200, 3), (1200, 528, 264, 4), (20, 128, 40, 5)):
        x, xs, w, ws, _ = made(g, rows, d_in, d_out, experts)
        slots = torch.randint(0, experts, (rows,), generator=g, device="cuda", dtype=torch.int32)
        want, bound = R.int8_matmul(x, xs, w, ws, None, slots.cpu().numpy(), np.arange(rows), torch.float32)
        between = w.transpose(0, 1).contiguous().transpose(0, 1)
        assert between.stride() == (d_in, experts * d_in, 1)
        y = L.lora_int8_matmul(x, xs, L.Int8Weight(between, ws), meta=L.lora_prepare_meta(slots, experts), dtype=torch.float32)
        R.near(y, want, bound)


# d_in of 1, 2, 3, 4, 5, 6, 9 and 10 stages of 128 bytes, the last one whole or not
STAGES = [16, 144, 384, 512, 528, 656, 1040, 1280]


@pytest.mark.parametrize("d_in", STAGES)
@pytest.mark.parametrize("rows,d_out", [(1025, 3080), (2100, 3848)])
def test_dense_large_tiles(L, rows, d_out, d_in):
    """More than 768 tiles of 64 x 64: tiles of 128, and beyond 128 of 256 x 256 those."""
    g = torch.Generator("cuda").manual_seed(d_in)
    args = made(g, rows, d_in, d_out, bias=d_in % 32 == 0)
    for dtype in DTYPES:
        dense(L, *args, dtype)


def test_dense_more_tiles_than_workgroups(L):
    """306 tiles of 256 x 256, for one workgroup on each of 256 CUs."""
    g = torch.Generator("cuda").manual_seed(14)
    args = made(g, 4100, 1040, 4360, bias=True)
    for dtype in DTYPES:
        dense(L, *args, dtype)


@pytest.mark.parametrize("d_in", STAGES)
def test_by_expert_large_tiles(L, d_in):
    """More than 160 rows a segment: tiles of 256 x 256."""
    for per_pair, dtype in ((False, torch.bfloat16), (True, torch.float32)):
        by_expert(L, 1100, 2, 5, 4, 1, d_in, 520, per_pair, dtype, 0.2, seed=d_in, bias=True)


@pytest.mark.parametrize("T,topk,E,local,d_in,d_out,skew", [
    (2000, 2, 4, 4, 1040, 4360, 0.0),       # 306 tiles of 256
    (1000, 4, 40, 32, 528, 2200, 0.0),      # 576 items of 128: segments of more than 16 rows go to tiles, and some workgroups take two
    (1000, 4, 40, 32, 656, 2200, 0.12),     # the same with segments below 16 rows and above 128
    (500, 4, 40, 32, 1040, 2064, 0.0)])     # half a tile each
def test_by_expert_many_tiles(L, T, topk, E, local, d_in, d_out, skew):
    for per_pair, dtype in ((False, torch.bfloat16), (True, torch.float32)):
        by_expert(L, T, topk, E, local, 0, d_in, d_out, per_pair, dtype, skew, seed=T + d_in, bias=True)


def test_two_threads_in_every_kernel(L):
    """Two threads, each on a stream of its own, with calls that go to each kernel: dense ones of few rows, in tiles of 64, 128
    and 256, and by expert in those of few rows, 128 and 256."""
    import threading
    g = torch.Generator("cuda").manual_seed(15)
    cases = []
    for rows, d_out, experts in ((3, 64, 0), (200, 640, 0), (900, 4096, 0), (5000, 4096, 0), (40, 256, 8), (3300, 2200, 32), (1500, 520, 4)):
        x, xs, w, ws, b = made(g, rows, 272, d_out, experts or None, bias=True)
        expert, meta = np.zeros(rows, np.int64), None
        if experts:
            slots = torch.randint(0, experts, (rows,), generator=g, device="cuda", dtype=torch.int32)
            expert, meta = slots.cpu().numpy(), L.lora_prepare_meta(slots, experts)
        weight = L.Int8Weight(w, ws, bias=b)
        y = L.lora_int8_matmul(x, xs, weight, meta=meta)
        want, bound = R.int8_matmul(x, xs, w, ws, b, expert, np.arange(rows), y.dtype)
        R.near(y, want, bound, f"{rows} rows, {experts} experts")
        cases.append((x, xs, weight, meta, y))
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                for i, (x, xs, weight, meta, want) in enumerate(cases):
                    y = L.lora_int8_matmul(x, xs, weight, meta=meta)
                    stream.synchronize()
                    if not torch.equal(y, want):
                        wrong.append(i)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
