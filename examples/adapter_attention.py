"""One attention layer of a multi-adapter server, from hidden states to attention
outputs: the adapters' delta into the packed q | k | v rows, rotation and append
to a paged cache, attention with the adapters' system prompts read once a group.

Keys and values carry their adapter's delta, so a cached prompt can be shared by
requests of one adapter only: here every adapter has a system prompt, and its
requests form a group.  Run it with ``python examples/adapter_attention.py``; it
checks every step's outputs against plain torch operations in float32.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import segmented_gather_rank_amd as L  # noqa: E402


class Layer:
    """The weights of the layer, the cache and its pages, and the requests' state."""

    def __init__(self, adapters=3, hidden=512, hq=8, hkv=2, dim=64, rank=16, pages=256, page=16, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        r = lambda *s: 0.05 * torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.hidden, self.hq, self.hkv, self.dim, self.page, self.adapters = hidden, hq, hkv, dim, page, adapters
        widths = [hq * dim, hkv * dim, hkv * dim]
        self.w = r(hidden, sum(widths)).bfloat16()
        self.a = [r(adapters, hidden, rank).bfloat16() for _ in widths]
        self.b = [r(adapters, rank, n).bfloat16() for n in widths]
        self.offsets = [0, widths[0], widths[0] + widths[1]]
        self.cache = L.KvCache(*(torch.zeros((pages, hkv, page, dim), dtype=torch.bfloat16, device="cuda") for _ in "kv"))
        self.free = list(range(pages))
        half = dim // 2
        angle = torch.arange(4096, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half) / half)
        self.table = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        self.rotation = L.Rotation(self.table)
        self.scale = 1 / math.sqrt(dim)
        self.rows = {}                                  # plain check: every request's q | k | v rows so far

    def step(self, requests, x, shared=None):
        """New tokens of some requests through the layer.  requests: dicts with
        "name", "slot" (adapter), "pages", "length" (tokens cached so far) and
        "new"; shared: [(requests in the group, shared keys)], in order."""
        new = [r["new"] for r in requests]
        T, dev = sum(new), "cuda"
        slots = torch.tensor([r["slot"] for r in requests for _ in range(r["new"])], dtype=torch.int32, device=dev)
        # base product (the caller's), then the delta of every token's adapter
        y = x @ self.w
        L.lora_apply(L.lora_prepare_meta(slots, self.adapters), x, self.a, self.b, self.offsets, y)
        pos, place = [], []
        for r in requests:
            for p in range(r["length"], r["length"] + r["new"]):
                if p // self.page == len(r["pages"]):
                    r["pages"].append(self.free.pop())
                pos.append(p)
                place.append(r["pages"][p // self.page] * self.page + p % self.page)
            r["length"] += r["new"]
        q = torch.empty((T, self.hq * self.dim), dtype=torch.bfloat16, device=dev)
        L.lora_cache_append(y, self.cache, torch.tensor(place, device=dev), q,
                            pos=torch.tensor(pos, dtype=torch.int32, device=dev), rotation=self.rotation)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        most = max(len(r["pages"]) for r in requests)
        groups = {}
        if shared:
            ends = [sum(n for n, _ in shared[:i + 1]) for i in range(len(shared))]
            groups = dict(group_start=ints([0] + ends), group_len=ints([keys for _, keys in shared]))
        meta = L.lora_prepare_attn_meta(
            ints([sum(new[:i]) for i in range(len(new) + 1)]), ints([r["length"] for r in requests]),
            ints([r["pages"] + [-1] * (most - len(r["pages"])) for r in requests]), self.cache, self.hq, T,
            max_q_len=max(new), **groups)
        out = L.lora_attention(meta, q, self.cache, scale=self.scale)
        return y, out.view(T, self.hq, self.dim)

    def check(self, requests, y, out):
        """Every new token against its request's whole history, in float32."""
        t = 0
        for r in requests:
            rows = self.rows.get(r["name"], self.rows.get(r.get("after"), torch.empty((0, y.shape[1]), device="cuda")))
            rows = torch.cat([rows, y[t:t + r["new"]].float()])
            self.rows[r["name"]] = rows
            n = len(rows)
            heads = rows.view(n, -1, self.dim)
            half = self.dim // 2
            cos, sin = self.table[:n, None, :half], self.table[:n, None, half:]
            a, b = heads[..., :half], heads[..., half:]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1).bfloat16().float()
            k = turned[:, self.hq:self.hq + self.hkv].repeat_interleave(self.hq // self.hkv, 1)
            v = heads[:, self.hq + self.hkv:].repeat_interleave(self.hq // self.hkv, 1)
            s = (turned[n - r["new"]:, :self.hq, None] * k.transpose(0, 1)[None]).sum(-1) * self.scale
            late = torch.arange(n, device="cuda")[None] > torch.arange(n - r["new"], n, device="cuda")[:, None]
            p = s.masked_fill(late[:, None], -math.inf).softmax(-1)
            want = (p[..., None] * v.transpose(0, 1)[None]).sum(2)
            got = out[t:t + r["new"]].float()
            # weights and result are each rounded to bf16 once
            bound = 2 * torch.finfo(torch.bfloat16).eps / 2 * (p[..., None] * v.transpose(0, 1).abs()[None]).sum(2) + 1e-4
            assert bool(((got - want).abs() <= bound).all()), f"{r['name']}: off by {(got - want).abs().max():.3e}"
            t += r["new"]


def main(adapters=3, per_adapter=4, prompt=80, decode=3):
    layer = Layer(adapters)
    g = torch.Generator("cuda").manual_seed(1)
    hidden = lambda n: torch.randn((n, layer.hidden), generator=g, device="cuda").bfloat16()  # noqa: E731

    # the adapters' system prompts, once each
    systems = [dict(name=f"system {s}", slot=s, pages=[], length=0, new=prompt + 16 * s) for s in range(adapters)]
    y, out = layer.step(systems, hidden(sum(r["new"] for r in systems)))
    layer.check(systems, y, out)

    # requests: the whole pages of their adapter's prompt are shared as they are
    requests, shared = [], []
    for s in systems:
        keys = s["length"] // layer.page * layer.page
        assert keys == s["length"], "prompts of whole pages here"
        shared.append((per_adapter, keys))
        requests += [dict(name=f"request {s['slot']}.{i}", after=s["name"], slot=s["slot"], pages=list(s["pages"]),
                          length=keys, new=5 + 11 * i) for i in range(per_adapter)]
    for step in range(1 + decode):
        y, out = layer.step(requests, hidden(sum(r["new"] for r in requests)), shared)
        layer.check(requests, y, out)
        for r in requests:
            r["new"] = 1
    print(f"{adapters} adapters, {len(requests)} requests, prompts of {[k for _, k in shared]} tokens: "
          f"{1 + decode} steps match")


if __name__ == "__main__":
    main()
