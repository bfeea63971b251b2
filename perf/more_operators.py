"""The base side of a layer whose adapters' delta the library adds: what is measured, and its plain form.

Four operators of a dense or MoE layer with 8-bit base weights:

* route: expert choices and their weights from a router's logits (softmax or sigmoid
  scores, a bias that decides but does not weigh, groups, renormalised weights);
* quantize: rows to 8-bit integers with one scale each, of a plain input or of the gated
  activation between an expert's two products;
* matmul: the product of 8-bit rows and weights with a scale for each token and channel,
  dense or by expert (rows grouped by metadata, some of them another rank's);
* combine: the weighted sum of a token's expert outputs.

A case is a dict of plain values.  Which experts the tokens choose comes from
``case["lens"]`` alone, up to the tokens' order, so the work of a case is known without
its data.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def _route(name, tokens, experts, topk, **kw):
    c = dict(op="route", name=name, tokens=tokens, experts=experts, topk=topk, score="softmax", bias=False, groups=1,
             topk_groups=1, renorm=True, dtype="f32", masked=0.0, scale=1.0)
    c.update(kw)
    return c


def _quantize(name, rows, width, **kw):
    """rows: tokens; with topk the rows are (token, choice) pairs of `experts` experts, `local` of them here."""
    c = dict(op="quantize", name=name, tokens=rows, width=width, act=False, dtype="bf16", topk=0, experts=0, local=0, lens=7)
    c.update(kw)
    return c


def _matmul(name, tokens, d_in, d_out, **kw):
    """per_pair: x has a row per (token, choice) pair (an expert's second product), else per token."""
    c = dict(op="matmul", name=name, tokens=tokens, d_in=d_in, d_out=d_out, dtype="bf16", topk=0, experts=0, local=0,
             per_pair=False, bias=False, lens=7)
    c.update(kw)
    return c


def _combine(name, tokens, width, **kw):
    c = dict(op="combine", name=name, tokens=tokens, width=width, topk=8, experts=256, local=256, dtype="bf16", add=False, lens=7)
    c.update(kw)
    return c


def listed():
    return [
        # the next token of a single user: latency alone
        _route("route_one", 1, 256, 8, score="sigmoid", bias=True, groups=8, topk_groups=4, scale=2.5),
        # a prefill batch through a router with balance bias and groups
        _route("route_groups_prefill", 17705, 256, 8, score="sigmoid", bias=True, groups=8, topk_groups=4, scale=2.5),
        # softmax router, bf16 logits, an odd number of experts, some of them masked for some tokens
        _route("route_softmax_odd", 4609, 60, 4, dtype="bf16", masked=0.1),
        # the prefill batch's hidden states before a dense 8-bit layer
        _quantize("quantize_prefill", 17705, 4096),
        # between the two expert products of a mixed step whose experts are all here
        _quantize("quantize_act_experts", 4608, 2048, act=True, topk=8, experts=256, local=256),
        # one token through q_proj: latency alone
        _matmul("matmul_one", 1, 4096, 4096),
        # 256 decode tokens through q | k | v, with its bias
        _matmul("matmul_decode", 256, 4096, 6144, bias=True),
        # the prefill batch through gate | up
        _matmul("matmul_prefill", 17705, 4096, 28672),
        # a decode step's 256 tokens through the gate | up of 32 local experts of 256
        _matmul("matmul_experts_decode", 256, 7168, 4096, topk=8, experts=256, local=32),
        # a mixed step's tokens through the down product of the same experts, ragged counts
        _matmul("matmul_experts_mixed", 4609, 2048, 7168, topk=8, experts=256, local=32, per_pair=True),
        # the decode step's weighted sum on one of 8 ranks
        _combine("combine_decode", 256, 7168, local=32),
        # a mixed step's weighted sum where every expert is local, added to the shared expert's output
        _combine("combine_mixed", 4608, 4096, add=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "quantize", "matmul", "matmul", "combine"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    lens = rng.randrange(1 << 30)
    experts, topk = rng.choice([(8, 2), (60, 4), (64, 6), (128, 8), (256, 8)])
    moe = dict(topk=topk, experts=experts, local=rng.choice([experts, max(1, experts // 8)]), lens=lens)
    if op == "route":
        groups, kept = rng.choice([(1, 1), (4, 2)])
        score = rng.choice(["softmax", "sigmoid"])
        c = _route("", _log(rng, 1, 17705), experts, topk, score=score, bias=rng.random() < 0.5, groups=groups,
                   topk_groups=kept, renorm=rng.random() < 0.7, dtype=dtype, masked=rng.choice([0.0, 0.0, 0.05]),
                   scale=rng.choice([1.0, 2.5]))
    elif op == "quantize":
        width = 16 * _log(rng, 4, 896)
        rows = _log(rng, 1, min(17705, 17705 * 4096 // width))
        c = _quantize("", rows, width, act=rng.random() < 0.5, dtype=dtype)
        if rng.random() < 0.4:
            c.update(moe, act=True, tokens=max(1, rows // (2 * topk)))
    elif op == "matmul":
        d_in, d_out = 16 * _log(rng, 8, 896), 8 * _log(rng, 8, 3584)
        if rng.random() < 0.5:
            tokens = _log(rng, 1, 17705)
            while 2 * tokens * d_in * d_out > 4e12 or tokens * d_out > 500_000_000:
                tokens = max(1, tokens // 2)
            c = _matmul("", tokens, d_in, d_out, dtype=dtype, bias=rng.random() < 0.3, lens=lens)
        else:
            while moe["local"] * d_in * d_out > 1_000_000_000:
                d_out = max(64, d_out // 16 * 8)
                if d_out == 64:
                    d_in = max(128, d_in // 32 * 16)
            tokens = _log(rng, 1, 4609)
            while tokens * topk * d_out > 300_000_000:
                tokens = max(1, tokens // 2)
            c = _matmul("", tokens, d_in, d_out, dtype=dtype, bias=rng.random() < 0.3, per_pair=rng.random() < 0.5, **moe)
    else:
        width = 8 * _log(rng, 8, 896)
        tokens = _log(rng, 1, 4608)
        while tokens * topk * width > 4608 * 8 * 4096:
            tokens = max(1, tokens // 2)
        c = _combine("", tokens, width, add=rng.random() < 0.5, dtype=dtype, **moe)
    del c["name"]
    return c


def _choices(c):
    """Expert ids [tokens][topk], every row distinct, some experts far more popular than others."""
    g = np.random.Generator(np.random.PCG64(c["lens"]))
    liking = g.normal(size=c["experts"]) * 0.7
    draws = liking + g.gumbel(size=(c["tokens"], c["experts"]))
    return np.argsort(-draws, axis=1)[:, :c["topk"]].astype(np.int32)


def work(case):
    c = case
    e = SIZE[c["dtype"]]
    if c["op"] == "route":
        return {"bytes": c["tokens"] * (c["experts"] * e + 8 * c["topk"]), "flops": 12 * c["tokens"] * c["experts"]}
    rows, hit = c["tokens"], 1
    if c["topk"]:                                  # the experts of this rank are the first ones
        ids = _choices(c)
        here = ids[ids < c["local"]]
        rows, hit = len(here), len(np.unique(here))
    if c["op"] == "quantize":
        # the row in (twice as wide where it holds gate | up), the bytes, the scale, the activation for the adapters
        return {"bytes": rows * (c["width"] * (e * (2 if c["act"] else 1) + 1 + (e if c["act"] else 0)) + 4),
                "flops": rows * c["width"] * (15 if c["act"] else 5) + 1}
    if c["op"] == "matmul":
        x_rows = rows if c["per_pair"] or not c["topk"] else len(np.unique(np.nonzero((ids < c["local"]).any(1))[0]))
        return {"bytes": x_rows * (c["d_in"] + 4) + hit * c["d_out"] * (c["d_in"] + 4) + rows * c["d_out"] * e,
                "flops": 2 * rows * c["d_in"] * c["d_out"]}
    return {"bytes": (rows + c["tokens"] * (2 if c["add"] else 1)) * c["width"] * e + 8 * c["tokens"] * c["topk"],
            "flops": 2 * rows * c["width"]}


# ------------------------------------------------------------------ inputs

def _inputs(c, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    dt = TYPES[c["dtype"]]
    s = dict(c)
    T = c["tokens"]
    if c["op"] == "route":
        s["logits"] = (1.5 * r(T, c["experts"])).to(dt)
        if c["masked"]:
            s["logits"][torch.rand((T, c["experts"]), generator=gen, device="cuda") < c["masked"]] = -math.inf
        s["bias_e"] = 0.05 * r(c["experts"]) if c["bias"] else None
        return s
    pairs = T
    if c["topk"]:
        order = torch.randperm(T, generator=gen, device="cuda")
        s["ids"] = torch.from_numpy(_choices(c)).cuda()[order].contiguous()
        pairs = T * c["topk"]
        s["expert_map"] = torch.arange(c["experts"], dtype=torch.int32, device="cuda")
        s["expert_map"][c["local"]:] = -1          # the other experts are other ranks'
        s["key"] = torch.where(s["ids"] < c["local"], s["ids"], -1).view(-1)
    if c["op"] == "quantize":
        # hidden states: most channels alike, a few far larger
        loud = 1 + 20 * (torch.rand(c["width"] * (2 if c["act"] else 1), generator=gen, device="cuda") < 0.004)
        s["x"] = (r(pairs, len(loud)) * loud).to(dt)
        s["q"] = torch.zeros((pairs, c["width"]), dtype=torch.int8, device="cuda")
        s["scale"] = torch.zeros(pairs, device="cuda")
        s["values"] = torch.zeros((pairs, c["width"]), dtype=torch.bfloat16, device="cuda")
        s["out"] = torch.zeros((pairs, c["width"]), dtype=dt, device="cuda") if c["act"] else None
    elif c["op"] == "matmul":
        rows = pairs if c["per_pair"] else T
        byte = lambda *n: torch.empty(n, dtype=torch.int8, device="cuda")  # noqa: E731
        # normal values whose largest is near 127, as quantised rows and channels hold
        s["x"] = byte(rows, c["d_in"])
        for a in range(0, rows, 8192):
            s["x"][a:a + 8192] = (32 * r(*s["x"][a:a + 8192].shape)).clamp_(-127, 127).round_()
        s["x_scale"] = 0.01 + 0.04 * torch.rand(rows, generator=gen, device="cuda")
        E = max(1, c["local"])
        s["w"] = byte(E, c["d_out"], c["d_in"])
        for e in range(E):
            s["w"][e] = (32 * r(c["d_out"], c["d_in"])).clamp_(-127, 127).round_()
        s["w_scale"] = 2e-4 + 6e-4 * torch.rand((E, c["d_out"]), generator=gen, device="cuda")
        s["bias_n"] = 0.5 * r(E, c["d_out"]) if c["bias"] else None
        s["y"] = torch.zeros((pairs, c["d_out"]), dtype=dt, device="cuda")
    else:
        s["rows"] = r(pairs, c["width"]).to(dt)
        s["rows"][s["key"] < 0] = math.nan         # another rank's: never written here
        s["weights"] = torch.rand((T, c["topk"]), generator=gen, device="cuda")
        s["weights"] /= s["weights"].sum(1, keepdim=True)
        s["shared"] = r(T, c["width"]).to(dt) if c["add"] else None
        s["out"] = torch.empty((T, c["width"]), dtype=dt, device="cuda")
    return s


def prepare(case, seed):
    c, s = case, _inputs(case, seed)
    if own:
        import segmented_gather_rank_amd as L
        T = c["tokens"]
        if c["op"] == "route":
            s["routing"] = L.Routing(c["experts"], c["topk"], score=c["score"], bias=s["bias_e"], num_groups=c["groups"],
                                     topk_groups=c["topk_groups"], renormalize=c["renorm"], scale=c["scale"])
            s["ids_out"] = torch.empty((T, c["topk"]), dtype=torch.int32, device="cuda")
            s["w_out"] = torch.empty((T, c["topk"]), device="cuda")
            return s
        s["meta"] = None
        if c["topk"] and c["op"] != "combine":
            # the step's rows by expert, kept for all of the layer's calls
            s["meta"] = L.lora_prepare_moe_meta(s["ids"], torch.zeros(T, dtype=torch.int32, device="cuda"), 1, c["experts"],
                                                c["local"], s["expert_map"])
            if c["op"] == "quantize" or c["per_pair"]:
                s["meta"] = s["meta"].with_x_row_div(1)
        if c["op"] == "matmul":
            s["handle"] = L.Int8Weight(s["w"], s["w_scale"], bias=s["bias_n"])
            s["ws"] = torch.empty(L.lora_int8_matmul_workspace_bytes(len(s["y"]), s["handle"]), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the pass

def run(state):
    s = state
    if own:
        import segmented_gather_rank_amd as L
    if s["op"] == "route":
        if own:
            return L.lora_moe_route(s["logits"], s["routing"], topk_ids=s["ids_out"], weights=s["w_out"])
        return _plain_route(s)
    if s["op"] == "quantize":
        if own:
            L.lora_quantize(s["x"], q=s["q"], scale=s["scale"], activation="silu_mul" if s["act"] else None, act=s["out"],
                            meta=s["meta"])
        else:
            _plain_quantize(s)
        # 8-bit storage is handed on as the values it stands for
        torch.mul(s["q"], s["scale"][:, None], out=s["values"])
        return s["values"], s["scale"], s["out"]
    if s["op"] == "matmul":
        if own:
            return L.lora_int8_matmul(s["x"], s["x_scale"], s["handle"], out=s["y"], meta=s["meta"], workspace=s["ws"])
        return _plain_matmul(s)
    if own:
        return L.lora_moe_combine(s["rows"], s["weights"], s["ids"], out=s["out"], num_local_experts=s["local"],
                                  expert_map=s["expert_map"], add=s["shared"])
    return _plain_combine(s)


def _plain_route(s):
    """Scores, biased scores, groups, then a stable sort; in 64 bits, since near scores decide the choice."""
    x = s["logits"].double()
    T, E = x.shape
    if s["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-x))
    choice = score if s["bias_e"] is None else score + s["bias_e"].double()
    choice = torch.where(x == -math.inf, x, choice)
    if s["groups"] > 1:
        by_group = choice.view(T, s["groups"], -1)
        rank = by_group.sort(2, descending=True).values[..., :2].sum(2)
        best = rank.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        kept = torch.zeros((T, s["groups"]), dtype=torch.bool, device="cuda").scatter_(1, best, True)
        # dropped groups go behind masked experts of the kept ones
        order = torch.where(kept[..., None], by_group.clamp_min(-1e300), -math.inf).view(T, E)
    else:
        order = choice
    ids = order.sort(dim=1, descending=True, stable=True).indices[:, :s["topk"]]
    w = score.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.int(), (w * s["scale"]).float()


def _plain_quantize(s):
    """The activation in 32 bits, the largest of each row, and the rounding in 64 (values halfway between two steps)."""
    v = s["x"].float()
    if s["act"]:
        gate, up = v[:, :s["width"]], v[:, s["width"]:]
        v = gate / (1 + torch.exp(-gate)) * up
    top = v.abs().amax(1).double()
    q = torch.round(127 * v.double() / torch.where(top > 0, top, torch.ones_like(top))[:, None]).to(torch.int8)
    scale = (top / 127).float()
    if s["topk"]:
        here = s["key"] >= 0
        s["q"].copy_(torch.where(here[:, None], q, s["q"]))
        s["scale"].copy_(torch.where(here, scale, s["scale"]))
        s["out"].copy_(torch.where(here[:, None], v, s["out"].float()))
    else:
        s["q"].copy_(q)
        s["scale"].copy_(scale)
        if s["act"]:
            s["out"].copy_(v)


def _plain_matmul(s):
    """Products in 32 bits; by expert, the rows are laid out expert by expert first."""
    x, w, xs = s["x"], s["w"], s["x_scale"]
    if not s["topk"]:
        y = torch.matmul(x.float(), w[0].float().t()) * xs[:, None] * s["w_scale"]
        s["y"].copy_(y if s["bias_n"] is None else y + s["bias_n"])
        return s["y"]
    E = s["local"]
    pair = torch.nonzero(s["key"] >= 0).squeeze(1)
    if not len(pair):
        return s["y"]
    key = s["key"][pair].long()
    count = (key[:, None] == torch.arange(E, device="cuda")).sum(0)
    pair, key = pair[key.argsort(stable=True)], key.sort().values
    place = torch.arange(len(pair), device="cuda") - (count.cumsum(0) - count)[key]
    source = pair if s["per_pair"] else pair // s["topk"]
    laid = torch.zeros((E, int(count.max()), x.shape[1]), device="cuda")
    laid[key, place] = x[source].float()
    y = torch.bmm(w.float(), laid.transpose(1, 2).contiguous())            # [E][d_out][rows]
    y = y.transpose(1, 2)[key, place] * xs[source][:, None] * s["w_scale"][key]
    s["y"][pair] = (y if s["bias_n"] is None else y + s["bias_n"][key]).to(s["y"].dtype)
    return s["y"]


def _plain_combine(s):
    T, K = s["ids"].shape
    here = (s["key"] >= 0).view(T, K, 1)
    rows = torch.where(here, s["rows"].view(T, K, -1).float(), torch.zeros((), device="cuda"))
    out = (rows * s["weights"][..., None]).sum(1)
    s["out"].copy_(out + s["shared"].float() if s["add"] else out)
    return s["out"]


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    c, s = case, _inputs(case, seed)
    f64 = torch.float64
    if c["op"] == "route":
        ids, w = [], []
        for x in s["logits"].to(f64).split(512):
            n, E = x.shape
            p = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
            ch = (p + s["bias_e"].to(f64) if c["bias"] else p).masked_fill(x.isinf(), -math.inf)
            e = torch.arange(E, device="cuda")

            def places(v):                         # how many entries come before each: larger ones, and equal ones to its left
                i = torch.arange(v.shape[1], device="cuda")
                left = i[:, None] < i[None, :]     # [f][e]: f stands left of e
                return ((v[:, :, None] > v[:, None, :]) | ((v[:, :, None] == v[:, None, :]) & left)).sum(1)

            if c["groups"] > 1:
                g = e // (E // c["groups"])
                two = torch.stack([ch[:, g == i].topk(2).values.sum(1) for i in range(c["groups"])], 1)
                ch = ch.clamp_min(-1e250).masked_fill((places(two) >= c["topk_groups"])[:, g], -math.inf)
            at = places(ch)
            chosen = torch.stack([(at == j).to(f64).argmax(1) for j in range(c["topk"])], 1)
            v = torch.take_along_dim(p, chosen, 1)
            w.append(v * c["scale"] / (v.sum(1, keepdim=True) if c["renorm"] else 1))
            ids.append(chosen.int())
        return torch.cat(ids), torch.cat(w)
    if c["op"] == "quantize":
        values, scales, outs = s["values"].to(f64), s["scale"].to(f64), None if s["out"] is None else s["out"].to(f64)
        live = torch.nonzero(s["key"] >= 0).squeeze(1) if c["topk"] else torch.arange(c["tokens"], device="cuda")
        for at in live.split(2048):
            v = s["x"][at].to(f64)
            if c["act"]:
                v = torch.nn.functional.silu(v[:, :c["width"]]) * v[:, c["width"]:]
                outs[at] = v
            scales[at] = v.abs().amax(1) / 127
            step = scales[at][:, None].clamp_min(1e-300)
            low = torch.floor(v / step)
            part = v / step - low
            odd = low.remainder(2)                 # halfway: to the even neighbour
            values[at] = (low + ((part > 0.5) | ((part == 0.5) & (odd == 1)))) * step
        return values, scales, outs
    if c["op"] == "matmul":
        y = s["y"].to(f64)
        for e in range(max(1, c["local"])):
            at = torch.nonzero(s["key"] == e).squeeze(1) if c["topk"] else torch.arange(c["tokens"], device="cuda")
            w = s["w"][e].to(f64) * s["w_scale"][e].to(f64)[:, None]
            for part in at.split(4096):
                i = part // c["topk"] if c["topk"] and not c["per_pair"] else part
                y[part] = (s["x"][i].to(f64) * s["x_scale"][i].to(f64)[:, None]) @ w.t()
                if c["bias"]:
                    y[part] += s["bias_n"][e].to(f64)
        return y
    T, K = s["ids"].shape
    out = s["shared"].to(f64).clone() if c["add"] else torch.zeros((T, c["width"]), dtype=f64, device="cuda")
    for j in range(K):
        t = torch.nonzero(s["ids"][:, j] < c["local"]).squeeze(1)
        out[t] += s["weights"][t, j].to(f64)[:, None] * s["rows"][t * K + j].to(f64)
    return out
