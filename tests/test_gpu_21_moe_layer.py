"""lora_moe_combine against the float64 form, and the operators of a MoE layer one after
the other, as a server runs them: routing, base products, delta, activation, weighted sum."""
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


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("added", ["no", "apart", "in_place"])
@pytest.mark.parametrize("T,K,E,local,width,gap", [(1, 1, 1, 1, 8, 0), (1, 8, 256, 32, 7168, 0), (5, 2, 8, 8, 2056, 8),
                                                   (70, 8, 64, 64, 520, 0), (33, 64, 64, 60, 72, 16), (9, 9, 12, 3, 4096, 0)])
def test_combine(L, T, K, E, local, width, gap, added, dtype):
    g = torch.Generator("cuda").manual_seed(T + K)
    host = torch.Generator().manual_seed(T)
    ids = torch.stack([torch.randperm(E, generator=host)[:K] for _ in range(T)]).int().cuda()
    emap = torch.randperm(E, generator=host).int().cuda()
    emap[emap >= local] = -1
    here = (emap[ids.long()] >= 0).cpu().numpy()
    y = torch.randn((T * K, width + gap), generator=g, device="cuda").to(dtype)[:, :width]
    y[torch.from_numpy(~here.reshape(-1)).cuda()] = torch.nan          # never written
    w = torch.rand((T, K), generator=g, device="cuda") - 0.3
    out = torch.full((T + 2, width + gap), 5.0, dtype=dtype, device="cuda")
    part = out[1:T + 1, :width]
    add = None
    if added != "no":
        add = torch.randn((T, width), generator=g, device="cuda").to(dtype)
    want, bound = R.combine(y, w, ids, here, add, dtype)
    if added == "in_place":
        part.copy_(add)
        add = part
    got = L.lora_moe_combine(y, w, ids, out=part, num_local_experts=local, expert_map=emap, add=add)
    R.near(got, want, bound)
    assert (out[0] == 5).all() and (out[T + 1] == 5).all() and (out[:, width:] == 5).all()


def test_combine_without_map(L):
    """Ids below the local count are local; ids out of range are nobody's, and their rows are not read."""
    ids = torch.tensor([[0, 5], [7, 1], [-1, 2], [9, 2147483647], [3, 3]], dtype=torch.int32, device="cuda")
    y = torch.arange(1, 11, device="cuda").float()[:, None].repeat(1, 16)
    w = torch.ones((5, 2), device="cuda")
    for kw, here in ((dict(num_experts=8, num_local_experts=4), ids < 4), (dict(num_experts=8), ids < 8), (dict(), ids < 2147483647)):
        here = (here & (ids >= 0)).cpu().numpy()
        z = y.clone()
        z[torch.from_numpy(~here.reshape(-1)).cuda()] = torch.nan
        want, bound = R.combine(z, w, ids, here, None, torch.float32)
        R.near(L.lora_moe_combine(z, w, ids, **kw), want, bound)
    # a map that names experts beyond the local ones: as the metadata counts them, bad and not local
    emap = torch.tensor([0, 1, 2, 3, -2, 4, -1, 9], dtype=torch.int32, device="cuda")
    here = ((ids >= 0) & (ids < 4)).cpu().numpy()
    want, bound = R.combine(y, w, ids, here, None, torch.float32)
    R.near(L.lora_moe_combine(y, w, ids, num_local_experts=4, expert_map=emap), want, bound)
    assert L.lora_moe_combine(y[:0], w[:0], ids[:0]).shape == (0, 16)


class Layer:
    """A MoE layer with 8-bit experts and adapters, of which this rank holds some."""

    def __init__(self, hidden=256, inter=192, E=16, local=6, topk=4, slots=3, rank=16, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        byte = lambda *n: torch.randint(-127, 128, n, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
        self.hidden, self.inter, self.E, self.local, self.topk, self.slots = hidden, inter, E, local, topk, slots
        self.bias = 0.1 * r(E)
        self.w13, self.s13 = byte(local, 2 * inter, hidden), 1e-3 * (0.5 + torch.rand((local, 2 * inter), generator=g, device="cuda"))
        self.w2, self.s2 = byte(local, hidden, inter), 1e-3 * (0.5 + torch.rand((local, hidden), generator=g, device="cuda"))
        self.a13 = [0.05 * r(slots, local, hidden, rank).bfloat16() for _ in range(2)]
        self.b13 = [0.05 * r(slots, local, rank, inter).bfloat16() for _ in range(2)]
        self.a2, self.b2 = 0.05 * r(slots, local, inter, rank).bfloat16(), 0.05 * r(slots, local, rank, hidden).bfloat16()
        self.emap = torch.full((E,), -1, dtype=torch.int32, device="cuda")
        self.emap[5:5 + local] = torch.arange(local, dtype=torch.int32, device="cuda")

    def handles(self, L):
        self.h13, self.h2 = L.Int8Weight(self.w13, self.s13), L.Int8Weight(self.w2, self.s2)
        self.routing = L.Routing(self.E, self.topk, score="sigmoid", bias=self.bias, num_groups=4, topk_groups=2, scale=2.0)
        return self

    def step(self, L, x, logits, slot, buffers):
        """One step; every intermediate is kept in `buffers` for the check."""
        b = buffers
        T, flat = len(x), lambda w: w.flatten(0, 1)  # noqa: E731
        L.lora_moe_route(logits, self.routing, topk_ids=b["ids"], weights=b["weights"])
        base = L.lora_prepare_moe_meta(b["ids"], b["nobody"], 1, self.E, self.local, self.emap, workspace=b["meta"])
        delta = L.lora_prepare_moe_meta(b["ids"], slot, self.slots, self.E, self.local, self.emap, workspace=b["meta_delta"])
        L.lora_quantize(x, q=b["xq"], scale=b["xs"])
        L.lora_int8_matmul(b["xq"], b["xs"], self.h13, out=b["gate_up"], meta=base)
        L.lora_apply(delta, x, [flat(a) for a in self.a13], [flat(w) for w in self.b13], [0, self.inter], b["gate_up"],
                     workspace=b["apply"])
        base, delta = base.with_x_row_div(1), delta.with_x_row_div(1)
        L.lora_quantize(b["gate_up"], q=b["aq"], scale=b["as"], activation="silu_mul", act=b["act"], meta=base)
        L.lora_int8_matmul(b["aq"], b["as"], self.h2, out=b["down"], meta=base)
        L.lora_apply(delta, b["act"], [flat(self.a2)], [flat(self.b2)], [0], b["down"], workspace=b["apply"])
        L.lora_moe_combine(b["down"], b["weights"], b["ids"], out=b["out"], num_local_experts=self.local, expert_map=self.emap,
                           add=x)

    def buffers(self, L, T):
        P, e = T * self.topk, lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        rows = dict(ids=e(T, self.topk, dtype=torch.int32), weights=e(T, self.topk, dtype=torch.float32),
                    nobody=torch.zeros(T, dtype=torch.int32, device="cuda"), xq=e(T, self.hidden, dtype=torch.int8),
                    xs=e(T, dtype=torch.float32), gate_up=e(P, 2 * self.inter), act=e(P, self.inter),
                    aq=e(P, self.inter, dtype=torch.int8), down=e(P, self.hidden), out=e(T, self.hidden),
                    meta=e(L.lora_moe_meta_workspace_bytes(T, self.topk, 1, self.local), dtype=torch.uint8),
                    meta_delta=e(L.lora_moe_meta_workspace_bytes(T, self.topk, self.slots, self.local), dtype=torch.uint8))
        rows["as"] = e(P, dtype=torch.float32)
        need = max(L.lora_apply_workspace_bytes(P, self.slots * self.local, d, n, 16, torch.bfloat16)
                   for d, n in ((self.hidden, 2), (self.inter, 1)))
        rows["apply"] = L.apply_workspace(need)
        return rows

    def check(self, x, logits, slot, b):
        """Every step's outputs from the step's own inputs, in float64."""
        T, K, f64 = len(x), self.topk, R.f64
        ids, weights = R.route(logits, K, "sigmoid", self.bias, 4, 2, 2, True, 2.0)
        assert (b["ids"].cpu().numpy() == ids).all()
        R.near(b["weights"], weights, np.abs(weights) * 2 * R.F32)
        expert = self.emap.cpu().numpy()[ids].reshape(-1)
        token = np.arange(T * K) // K
        here = np.nonzero(expert >= 0)[0]
        q, s = R.quantize(f64(x))
        assert (b["xq"].cpu().numpy() == q).all() and np.array_equal(b["xs"].cpu().numpy(), s)
        slots = slot.cpu().numpy()

        def delta(rows, v, A, B):
            """The adapters' part: their exact sum; u in float32 (its terms' size says how far off)."""
            out, size = np.zeros((len(rows), B.shape[-1])), np.zeros((len(rows), B.shape[-1]))
            A, B = f64(A), f64(B)
            for i, p in enumerate(rows):
                if slots[token[p]] >= 0:
                    a, w = A[slots[token[p]], expert[p]], B[slots[token[p]], expert[p]]
                    out[i] = v[i] @ a @ w
                    size[i] = np.abs(v[i]) @ np.abs(a) @ np.abs(w)
            return out, size

        bf = R.HALF[torch.bfloat16]
        base, _ = R.int8_matmul(b["xq"], b["xs"], self.w13, self.s13, None, expert, token, torch.bfloat16)
        parts = [delta(here, f64(x)[token[here]], self.a13[i], self.b13[i]) for i in range(2)]
        want = base[here] + np.concatenate([p[0] for p in parts], 1)
        size = np.concatenate([p[1] for p in parts], 1)
        # the base product and the sum are rounded to bf16, and the kernels may take u in bf16
        R.near(b["gate_up"][here], want, 2.02 * bf * (np.abs(base[here]) + np.abs(want)) + bf * size + 1e-6, "gate | up")
        a = R.silu_mul(b["gate_up"][here])
        R.near(b["act"][here], a, np.abs(a) * (bf + 110 * R.F32) + 1e-40, "act")
        m = np.abs(a).max(1)
        R.near(b["as"][here], m / 127, m / 127 * 112 * R.F32, "scale")
        assert (np.abs(f64(b["aq"])[here] - a * 127 / m[:, None]) <= 0.5 + 127 * 330 * R.F32).all()
        base, _ = R.int8_matmul(b["aq"], b["as"], self.w2, self.s2, None, expert, np.arange(T * K), torch.bfloat16)
        part, size = delta(here, f64(b["act"])[here], self.a2, self.b2)
        want = base[here] + part
        R.near(b["down"][here], want, 2.02 * bf * (np.abs(base[here]) + np.abs(want)) + bf * size + 1e-6, "down")
        want, bound = R.combine(b["down"], b["weights"], b["ids"].cpu(), (expert >= 0).reshape(T, K), x, torch.bfloat16)
        R.near(b["out"], want, bound, "out")


@pytest.mark.parametrize("T,kw", [(1, {}), (3, dict(local=1)), (50, {}), (400, dict(hidden=512, inter=136 // 16 * 16)),
                                  (900, dict(local=16 - 5, topk=2))])
def test_layer(L, T, kw):
    layer = Layer(seed=T, **kw).handles(L)
    g = torch.Generator("cuda").manual_seed(T)
    b = layer.buffers(L, T)
    for step in range(2):                            # the second on the first's buffers
        x = torch.randn((T, layer.hidden), generator=g, device="cuda").bfloat16()
        logits = torch.randn((T, layer.E), generator=g, device="cuda")
        slot = torch.randint(-1, layer.slots, (T,), generator=g, device="cuda", dtype=torch.int32)
        layer.step(L, x, logits, slot, b)
        torch.cuda.synchronize()
        layer.check(x, logits, slot, b)


def test_layer_captured(L):
    """The whole layer in a graph, replayed on new inputs between eager steps of another layer."""
    T = 40
    layer, other = Layer(seed=1).handles(L), Layer(seed=2).handles(L)
    g = torch.Generator("cuda").manual_seed(3)
    b, mine = layer.buffers(L, T), other.buffers(L, T)
    x = torch.randn((T, layer.hidden), generator=g, device="cuda").bfloat16()
    logits = torch.randn((T, layer.E), generator=g, device="cuda")
    slot = torch.randint(-1, layer.slots, (T,), generator=g, device="cuda", dtype=torch.int32)
    layer.step(L, x, logits, slot, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(L, x, logits, slot, b)
    for _ in range(4):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        logits.copy_(torch.randn(logits.shape, generator=g, device="cuda"))
        slot.copy_(torch.randint(-1, layer.slots, (T,), generator=g, device="cuda", dtype=torch.int32))
        graph.replay()
        other.step(L, x, logits, slot, mine)
        torch.cuda.synchronize()
        layer.check(x, logits, slot, b)
        other.check(x, logits, slot, mine)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("K", [1, 8, 20])
def test_combine_adds_last(L, K, in_place):
    """A row to add that is far larger than the sum: the sum is rounded at its own size, not at that of the row."""
    T, width = 5, 2056
    ids = torch.arange(K, device="cuda", dtype=torch.int32).expand(T, K).contiguous()
    w = torch.ones((T, K), device="cuda")
    add = torch.full((T, width), 2.0 ** 24, device="cuda")           # 1 is half a step there
    out = add.clone() if in_place else None
    got = L.lora_moe_combine(torch.ones((T * K, width), device="cuda"), w, ids, out=out, add=out if in_place else add)
    assert bool((got == 2.0 ** 24 + K // 2 * 2).all())               # halves go to the even neighbour
    g = torch.Generator("cuda").manual_seed(K)
    y, w = torch.randn((T * K, width), generator=g, device="cuda"), torch.rand((T, K), generator=g, device="cuda") - 0.3
    add = 1000 * torch.randn((T, width), generator=g, device="cuda")
    out = add.clone() if in_place else None
    local = np.ones((T, K), bool)
    want, _ = R.combine(y, w, ids, local, add, torch.float32)
    size, _ = R.combine(y.abs(), w.abs(), ids, local, None, torch.float32)
    got = L.lora_moe_combine(y, w, ids, out=out, add=out if in_place else add)
    # a product and a sum for each choice, off by a rounding of at most the terms' whole size; then one of the output's
    R.near(got, want, 2 * K * R.F32 * size * (1 + 1e-5) + R.F32 * np.abs(want) * (1 + 1e-5) + 1e-37)


def test_combine_many_launches(L):
    """More tokens than one launch takes: as the same tokens in two calls."""
    T, cut = (1 << 23) + 37, (1 << 23) - 5
    g = torch.Generator("cuda").manual_seed(2)
    y = torch.randn((2 * T, 8), generator=g, device="cuda").bfloat16()
    w = torch.rand((T, 2), generator=g, device="cuda")
    ids = torch.randint(0, 6, (T, 2), generator=g, device="cuda", dtype=torch.int32)
    out = L.lora_moe_combine(y, w, ids, num_experts=6, num_local_experts=4)
    for part, pairs in ((slice(0, cut), slice(0, 2 * cut)), (slice(cut, T), slice(2 * cut, 2 * T))):
        assert torch.equal(out[part], L.lora_moe_combine(y[pairs], w[part], ids[part], num_experts=6, num_local_experts=4))
    want, bound = R.combine(y[-100:], w[-50:], ids[-50:], (ids[-50:] < 4).cpu().numpy().reshape(-1, 2), None, torch.bfloat16)
    R.near(out[-50:], want, bound)
