"""Attention next to the adapters' q/k/v delta: what is measured, and its plain form.

Three operators that follow a layer's q/k/v projection (base product plus
adapter delta, packed as q | k | v in one row per token):

* append: q and k are rotated by their positions (one or three axes), q goes to
  a buffer of its own, k and v go into the pages of a cache (bf16, fp32 or e4m3);
* attention: every query row against the cached keys of its sequence, decode and
  prefill mixed in one batch, causal or not, with a sliding window, a prefix or
  document mask, a tanh cap on the scores, a bias linear in the distance;
* prefix: the same for batches whose sequences share leading keys (requests of
  one adapter with one system prompt), whose keys are read once per group.

A case is a dict of plain values.  Lengths come from ``case["lens"]`` alone, so
the work of a case is known without its data.
"""
import math
import random

import numpy as np
import torch

own = False

HEADS = [(32, 8), (16, 16), (28, 4), (8, 1), (24, 8)]
DIMS = [64, 128, 96, 256]
PAGES = [16, 32, 64]
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}


# ------------------------------------------------------------------ cases

def _append(name, tokens, **kw):
    c = dict(op="append", name=name, tokens=tokens, hq=32, hkv=8, d=128, rot=128, page=16, dtype="bf16",
             cache="bf16", axes=1, interleaved=False, hold="heads", positions=32768)
    c.update(kw)
    return c


def _attend(name, decode, prefill, op="attention", **kw):
    """decode: (sequences, fewest keys, most keys), one query token each;
    prefill: (sequences, fewest queries, most queries, most keys before them)."""
    c = dict(op=op, name=name, n_dec=decode[0], dec_lo=decode[1], dec_hi=decode[2], n_pre=prefill[0],
             pre_lo=prefill[1], pre_hi=prefill[2], past=prefill[3], hq=32, hkv=8, d=128, page=16, dtype="bf16",
             cache="bf16", causal=True, window=0, prefix_mask=False, docs=False, cap=0.0, slopes=False,
             hold="heads", groups=0, shared=0, lens=7)
    c.update(kw)
    return c


def listed():
    return [
        # one token of one sequence: latency alone
        _append("append_one", 1),
        # the mixed q/k/v batch: 512 decode tokens and 4 prompts of 1024
        _append("append_mixed", 4608),
        # image tokens with time, height and width positions into an 8-bit cache, odd count
        _append("append_three_axes_e4m3", 4097, hq=28, hkv=4, axes=3, cache="e4m3", page=32),
        # a prefill batch, interleaved pairs over half the head, pages of whole token rows
        _append("append_prefill", 17705, interleaved=True, rot=64, hold="tokens"),
        # a single user's next token
        _attend("decode_one", (1, 1000, 1000), (0, 0, 0, 0)),
        # a decode batch of a chat service, ragged contexts
        _attend("decode_batch", (256, 64, 6000), (0, 0, 0, 0)),
        # long contexts in an 8-bit cache with capped scores
        _attend("decode_long_e4m3_cap", (24, 30000, 65000), (0, 0, 0, 0), cache="e4m3", cap=50.0, page=64),
        # the mixed batch: 512 decode tokens and 4 prompts of 1024, distance bias, a sliding window
        _attend("mixed_window_bias", (512, 1, 2000), (4, 1024, 1024, 0), window=1024, slopes=True),
        # one long prompt, causal
        _attend("prefill_long", (0, 0, 0, 0), (1, 16384, 16384, 0)),
        # packed documents with padding rows that see nothing, prefix mask, odd head size, one head per key head
        _attend("prefill_documents", (0, 0, 0, 0), (5, 300, 2500, 129), hq=16, hkv=16, d=96, docs=True,
                prefix_mask=True, hold="tokens"),
        # four adapters, each with its own system prompt, 32 requests of each in decode
        _attend("prefix_adapters", (128, 20, 1500), (0, 0, 0, 0), op="prefix", groups=4, shared=8192),
        # one short prompt shared by few requests, some still in prefill
        _attend("prefix_few", (5, 1, 300), (2, 40, 90, 200), op="prefix", groups=1, shared=2000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hq, hkv = rng.choice(HEADS)
    d = rng.choice(DIMS)
    op = rng.choice(["append", "attention", "attention", "prefix"])
    dtype = "f32" if rng.random() < 0.12 else "bf16"
    cache = "f32" if dtype == "f32" else rng.choice(["bf16", "bf16", "e4m3"])
    kw = dict(hq=hq, hkv=hkv, d=d, page=rng.choice(PAGES), dtype=dtype, cache=cache,
              hold=rng.choice(["heads", "tokens"]))
    if op == "append":
        c = _append("", _log(rng, 1, 17705), **kw)
        c.update(rot=rng.choice([d, d // 2]), axes=rng.choice([1, 3]), interleaved=rng.random() < 0.5)
    else:
        kw.update(window=rng.choice([0, 0, _log(rng, 16, 4096)]), cap=rng.choice([0.0, 0.0, 30.0]),
                  slopes=rng.random() < 0.3, prefix_mask=rng.random() < 0.2, lens=rng.randrange(1 << 30))
        keys = (32 if dtype == "f32" else 256) * 1024 * 2048 // (hkv * d * 4)   # of all sequences together
        n = _log(rng, 1, 256)
        most = _log(rng, 8, max(8, min(32768, keys // n)))
        dec = (n, max(1, most // rng.choice([1, 4, 100])), most)
        pre = (0, 0, 0, 0)
        if rng.random() < 0.5:
            m = rng.choice([1, 2, 5])
            q = _log(rng, 2, 1000 if dtype == "f32" else 4000)
            pre = (m, max(1, q // 3), q, rng.choice([0, 0, 777]))
            if rng.random() < 0.3:
                dec = (0, 0, 0)
        if op == "prefix":
            g = rng.choice([1, 2, 4])
            kw.update(groups=g, shared=_log(rng, 32, 16384 if dtype == "bf16" else 2048))
            dec = (max(dec[0], g), max(1, dec[1]), max(1, dec[2]))
        elif rng.random() < 0.3:
            kw.update(docs=True)
        c = _attend("", dec, pre, op=op, **kw)
    del c["name"]
    return c


def _lengths(c):
    """Query tokens and keys of every sequence, and the sequences of every group."""
    r = random.Random(c["lens"])
    q = [1] * c["n_dec"]
    own_keys = [r.randint(c["dec_lo"], c["dec_hi"]) for _ in q]
    for _ in range(c["n_pre"]):
        n = r.randint(c["pre_lo"], c["pre_hi"])
        q.append(n)
        own_keys.append(n + r.randint(0, c["past"]))
    start, shared = [], []
    if c["groups"]:
        # groups of consecutive sequences; the keys that a group shares fill whole pages
        cuts = [len(q) * g // c["groups"] for g in range(c["groups"] + 1)]
        start = cuts
        shared = [max(1, c["shared"] * (2 + g % 3) // 4 // c["page"]) * c["page"] for g in range(c["groups"])]
        for g in range(c["groups"]):
            for n in range(cuts[g], cuts[g + 1]):
                own_keys[n] += shared[g]
    return q, own_keys, start, shared


def _limits(c, q, kv, n):
    """[lo, hi) of the keys that every query row of sequence n sees, and the
    arrays (document bounds, prefix length) that say so."""
    p = np.arange(kv[n] - q[n], kv[n])
    r = random.Random(c["lens"] * 7919 + n)
    lo, hi = np.zeros(q[n], np.int64), (p + 1 if c["causal"] else np.full(q[n], kv[n]))
    prefix, doc_lo, doc_hi = 0, np.zeros(q[n], np.int64), np.full(q[n], kv[n])
    if c["window"]:
        lo = np.maximum(lo, p + 1 - c["window"])
    if c["prefix_mask"]:
        prefix = r.randint(0, kv[n])
        hi = np.maximum(hi, prefix)
    if c["docs"]:
        at = 0
        while at < kv[n]:
            end = min(kv[n], at + r.randint(1, max(2, kv[n] // 3)))
            rows = (p >= at) & (p < end)
            doc_lo[rows], doc_hi[rows] = at, end
            if end - at >= 4:                      # the last row of a document is padding
                doc_hi[p == end - 1] = at
            at = end
    lo, hi = np.maximum(lo, doc_lo), np.minimum(np.minimum(hi, doc_hi), kv[n])
    return lo, np.maximum(lo, hi), prefix, doc_lo, doc_hi


def work(case):
    c = case
    e, b = SIZE[c["dtype"]], SIZE[c["cache"]]
    if c["op"] == "append":
        rows = c["tokens"] * c["d"]
        return {"bytes": rows * e * (2 * c["hq"] + 2 * c["hkv"]) + rows * b * 2 * c["hkv"] + c["tokens"] * c["rot"] * 4,
                "flops": 3 * c["tokens"] * c["rot"] * (c["hq"] + c["hkv"])}
    q, kv, start, shared = _lengths(c)
    pairs = keys = 0
    group = {n: g for g in range(c["groups"]) for n in range(start[g], start[g + 1])}
    low = {}
    for n in range(len(q)):
        lo, hi, *_ = _limits(c, q, kv, n)
        see = hi > lo
        if not see.any():
            continue
        pairs += int((hi - lo).sum())
        first, last, sh = int(lo[see].min()), int(hi.max()), shared[group[n]] if n in group else 0
        keys += max(0, last - max(first, sh))
        if sh and first < sh:
            low[group[n]] = min(low.get(group[n], sh), first)
    keys += sum(shared[g] - at for g, at in low.items())
    return {"bytes": keys * c["hkv"] * c["d"] * 2 * b + 2 * sum(q) * c["hq"] * c["d"] * e,
            "flops": 4 * pairs * c["hq"] * c["d"]}


# ------------------------------------------------------------------ inputs

def _store(x, kind):
    return x.clamp(-448, 448).to(TYPES[kind]) if kind == "e4m3" else x.to(TYPES[kind])


def _pages(c, n, gen):
    """Keys or values of n pages, indexed [page][head][position][dim]."""
    shape = (n, c["hkv"], c["page"], c["d"])
    if c["hold"] == "tokens":                      # a page holds whole token rows
        shape = (n, c["page"], c["hkv"], c["d"])
    x = torch.empty(shape, dtype=TYPES[c["cache"]], device="cuda")
    for i in range(0, n, 4096):
        x[i:i + 4096] = _store(torch.randn(x[i:i + 4096].shape, generator=gen, device="cuda"), c["cache"])
    return x.transpose(1, 2) if c["hold"] == "tokens" else x


def _inputs(c, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    host = random.Random(seed)
    s = dict(c)
    scales = [2.0 ** host.randint(-3, -1) for _ in range(2 * c["hkv"])] if c["cache"] == "e4m3" else [1.0] * 2 * c["hkv"]
    s["k_scale"] = torch.tensor(scales[:c["hkv"]], device="cuda")
    s["v_scale"] = torch.tensor(scales[c["hkv"]:], device="cuda")
    if c["op"] == "append":
        T, D = c["tokens"], c["d"]
        s["qkv"] = torch.randn((T, (c["hq"] + 2 * c["hkv"]) * D), generator=gen, device="cuda").to(TYPES[c["dtype"]])
        n = (T + T // 8) // c["page"] + 1
        s["slot"] = torch.randperm(n * c["page"], generator=gen, device="cuda")[:T]
        if T > 8:                                  # some tokens are not kept
            s["slot"][5::97] = -1
        s["pos"] = torch.randint(0, c["positions"], (c["axes"], T), generator=gen, device="cuda", dtype=torch.int32)
        # the table of a user's program: cosines, then sines, of position times frequency
        half = c["rot"] // 2
        freq = 500000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        angle = torch.arange(c["positions"], dtype=torch.float64)[:, None] * freq
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        s["sections"] = [half] if c["axes"] == 1 else [half - 2 * (half // 3), half // 3, half // 3]
        s["k"], s["v"] = _pages(c, n, gen), _pages(c, n, gen)
        s["q_out"] = torch.empty((T, c["hq"] * D), dtype=TYPES[c["dtype"]], device="cuda")
        return s

    q, kv, start, shared = _lengths(c)
    N, T, page = len(q), sum(q), c["page"]
    need = [-(-k // page) for k in kv]
    group = {n: g for g in range(c["groups"]) for n in range(start[g], start[g + 1])}
    total = sum(need) - sum((start[g + 1] - start[g] - 1) * shared[g] // page for g in range(c["groups"]) if start[g + 1] > start[g])
    ids = torch.randperm(total + 3, generator=gen, device="cuda").cpu().numpy()
    table = np.full((N, max(need)), -1, np.int32)
    at = 0
    for n in range(N):
        lead = 0
        if n in group and n > start[group[n]]:     # the group's pages, then its own
            lead = shared[group[n]] // page
            table[n, :lead] = table[start[group[n]], :lead]
        table[n, lead:need[n]] = ids[at:at + need[n] - lead]
        at += need[n] - lead
    limits = [_limits(c, q, kv, n) for n in range(N)]
    dev = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    s.update(q_len=q, kv_len=kv, q_start=dev(np.concatenate([[0], np.cumsum(q)])), kv=dev(kv), table=dev(table),
             group_start=dev(start) if start else None, group_len=dev(shared) if start else None, scale=1.0 / math.sqrt(c["d"]))
    s["prefix_len"] = dev([m[2] for m in limits]) if c["prefix_mask"] else None
    s["key_lo"] = dev(np.concatenate([m[3] for m in limits])) if c["docs"] else None
    s["key_hi"] = dev(np.concatenate([m[4] for m in limits])) if c["docs"] else None
    s["slope"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / c["hq"]) for h in range(c["hq"])], device="cuda") if c["slopes"] else None
    s["k"], s["v"] = _pages(c, total + 3, gen), _pages(c, total + 3, gen)
    s["q"] = (1.5 * torch.randn((T, c["hq"], c["d"]), generator=gen, device="cuda")).to(TYPES[c["dtype"]])
    return s


def prepare(case, seed):
    c, s = case, _inputs(case, seed)
    if own:
        import segmented_gather_rank_amd as L
        scales = (s["k_scale"], s["v_scale"]) if c["cache"] == "e4m3" else ()
        s["handle"] = L.KvCache(s["k"], s["v"], *scales)
        if c["op"] == "append":
            s["rotation"] = L.Rotation(s["table"], sections=s["sections"], interleaved=c["interleaved"])
            return s
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], device="cuda")
        # the step's plan, kept for all of its layers
        s["meta"] = L.lora_prepare_attn_meta(
            s["q_start"], s["kv"], s["table"], s["handle"], c["hq"], len(s["q"]), max_q_len=max(s["q_len"]),
            causal=c["causal"], window=c["window"], prefix_len=s["prefix_len"], key_lo=s["key_lo"],
            key_hi=s["key_hi"], group_start=s["group_start"], group_len=s["group_len"])
        s["ws"] = torch.empty(L.lora_attention_workspace_bytes(s["meta"]), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the pass

def run(state):
    s = state
    if s["op"] == "append":
        if own:
            import segmented_gather_rank_amd as L
            L.lora_cache_append(s["qkv"], s["handle"], s["slot"], s["q_out"], pos=s["pos"], rotation=s["rotation"])
        else:
            _plain_append(s)
        if s["cache"] == "e4m3":
            # 8-bit storage is handed on as the values it stands for (the scales are powers of two)
            up = lambda x, f: x.to(torch.bfloat16) * f.to(torch.bfloat16)[:, None, None]  # noqa: E731
            return s["q_out"], up(s["k"], s["k_scale"]), up(s["v"], s["v_scale"])
        return s["q_out"], s["k"], s["v"]
    if own:
        import segmented_gather_rank_amd as L
        return L.lora_attention(s["meta"], s["q"], s["handle"], s["out"], scale=s["scale"], cap=s["cap"],
                                slopes=s["slope"], lse=s["lse"], workspace=s["ws"])
    return _plain_attention(s)


def _plain_append(s):
    """The rotation pair by pair, then a copy to every token's place."""
    T, D, hq, hkv, half = s["tokens"], s["d"], s["hq"], s["hkv"], s["rot"] // 2
    axis = torch.tensor([a for a, n in enumerate(s["sections"]) for _ in range(n)], device="cuda")
    pos = s["pos"].long()[axis].t()                                        # [T][half]
    pair = torch.arange(half, device="cuda")
    cos, sin = s["table"][pos, pair][:, None], s["table"][pos, half + pair][:, None]
    x = s["qkv"].float().view(T, hq + 2 * hkv, D)
    rotated = x[:, :hq + hkv].clone()
    if s["interleaved"]:
        a, b = x[:, :hq + hkv, 0:2 * half:2], x[:, :hq + hkv, 1:2 * half:2]
        rotated[..., 0:2 * half:2], rotated[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[:, :hq + hkv, :half], x[:, :hq + hkv, half:2 * half]
        rotated[..., :half], rotated[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
    s["q_out"].copy_(rotated[:, :hq].reshape(T, hq * D))
    keep = s["slot"] >= 0
    at = s["slot"][keep]
    page, off = at // s["page"], at % s["page"]
    # [token][head][dim] into [page, :, position]
    s["k"][page, :, off] = _store(rotated[keep, hq:] / s["k_scale"][:, None], s["cache"])
    s["v"][page, :, off] = _store(x[keep, hq + hkv:] / s["v_scale"][:, None], s["cache"])


def _plain_attention(s):
    """Sequence by sequence and in blocks of query rows: scores, cap, bias, mask, softmax, product."""
    T, hq, hkv, D, G = sum(s["q_len"]), s["hq"], s["hkv"], s["d"], s["hq"] // s["hkv"]
    out = torch.empty_like(s["q"])
    lse = torch.empty((T, hq), device="cuda")
    t0 = 0
    for n, (m, kn) in enumerate(zip(s["q_len"], s["kv_len"])):
        ids = s["table"][n, :-(-kn // s["page"])].long()
        k = (s["k"][ids].float() * s["k_scale"][:, None, None]).transpose(0, 1).reshape(hkv, -1, D)[:, :kn]
        v = (s["v"][ids].float() * s["v_scale"][:, None, None]).transpose(0, 1).reshape(hkv, -1, D)[:, :kn]
        j = torch.arange(kn, device="cuda")
        block = max(1, (1 << 28) // (kn * hq))
        for a in range(0, m, block):
            b = min(m, a + block)
            rows = slice(t0 + a, t0 + b)
            p = torch.arange(kn - m + a, kn - m + b, device="cuda")[:, None]
            hi = p + 1 if s["causal"] else torch.full_like(p, kn)
            lo = torch.zeros_like(p)
            if s["prefix_len"] is not None:
                hi = torch.maximum(hi, s["prefix_len"][n].long())
            if s["window"]:
                lo = p + 1 - s["window"]
            if s["key_lo"] is not None:
                lo = torch.maximum(lo, s["key_lo"][rows, None].long())
                hi = torch.minimum(hi, s["key_hi"][rows, None].long())
            see = (j >= lo) & (j < hi)                                     # [rows][keys]
            q = s["q"][rows].float().view(b - a, hkv, G, D).permute(1, 0, 2, 3).reshape(hkv, -1, D)
            x = torch.matmul(q, k.transpose(1, 2).contiguous()).view(hkv, b - a, G, kn) * s["scale"]
            if s["cap"]:
                x = s["cap"] * torch.tanh(x / s["cap"])
            if s["slope"] is not None:
                x = x - s["slope"].view(hkv, 1, G, 1) * (p - j).abs().float()[None, :, None, :]
            x = x.masked_fill(~see[None, :, None, :], -math.inf)
            top = x.amax(-1, keepdim=True)
            top = torch.where(top == -math.inf, torch.zeros_like(top), top)
            w = torch.exp(x - top)
            total = w.sum(-1, keepdim=True)
            o = torch.matmul(w.view(hkv, -1, kn), v).view(hkv, b - a, G, D)
            o = torch.where(total > 0, o / total, torch.zeros_like(o))
            out[rows] = o.permute(1, 0, 2, 3).reshape(b - a, hq, D).to(out.dtype)
            lse[rows] = (top + torch.log(total)).squeeze(-1).permute(1, 0, 2).reshape(b - a, hq)
        t0 += m
    return out, lse


# ------------------------------------------------------------------ in 64 bits

def _grid8(x):
    """x (float64) rounded to the nearest e4m3 value, ties to even, saturating at 448."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -40))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    f64 = torch.float64
    ks, vs = s["k_scale"].to(f64), s["v_scale"].to(f64)
    if c["op"] == "append":
        T, D, hq, hkv, half = c["tokens"], c["d"], c["hq"], c["hkv"], c["rot"] // 2
        qkv = s["qkv"].to(f64).view(T, -1, D)
        # every pair as one complex number, turned by its angle
        re = list(range(0, 2 * half, 2)) if c["interleaved"] else list(range(half))
        im = [i + (1 if c["interleaved"] else half) for i in re]
        first = np.cumsum([0] + s["sections"])
        for h in range(hq + hkv):
            z = torch.complex(qkv[:, h, re], qkv[:, h, im])
            for a in range(c["axes"]):
                w = s["table"][s["pos"][a].long()].to(f64)
                i, e = int(first[a]), int(first[a + 1])
                z[:, i:e] *= torch.complex(w[:, i:e], w[:, half + i:half + e])
            qkv[:, h, re], qkv[:, h, im] = z.real, z.imag
        k, v = s["k"].to(f64) * ks[:, None, None], s["v"].to(f64) * vs[:, None, None]
        for x, f, h0 in ((k, ks, hq), (v, vs, hq + hkv)):
            new = qkv[:, h0:h0 + hkv]
            new = _grid8(new / f[:, None]) * f[:, None] if c["cache"] == "e4m3" else new
            flat = x.permute(0, 2, 1, 3).reshape(-1, hkv, D).clone()
            keep = s["slot"] >= 0
            flat[s["slot"][keep]] = new[keep]
            x.copy_(flat.view(x.shape[0], x.shape[2], hkv, D).permute(0, 2, 1, 3))
        return qkv[:, :hq].reshape(T, hq * D), k, v

    q_len, kv_len, _, _ = _lengths(c)
    hq, hkv, D, G = c["hq"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    out = torch.zeros((sum(q_len), hq, D), dtype=f64, device="cuda")
    lse = torch.full((sum(q_len), hq), -math.inf, dtype=f64, device="cuda")
    t0 = 0
    for n in range(len(q_len)):
        lo, hi, *_ = _limits(c, q_len, kv_len, n)
        ids = s["table"][n, :-(-kv_len[n] // c["page"])].long()
        j = torch.arange(kv_len[n], device="cuda")
        lo, hi = torch.tensor(lo, device="cuda"), torch.tensor(hi, device="cuda")
        heads = range(hkv)
        step = max(1, (1 << 27) // (kv_len[n] * G))
        for h in heads:
            kh = s["k"][ids, h].reshape(-1, D)[:kv_len[n]].to(f64) * ks[h]
            vh = s["v"][ids, h].reshape(-1, D)[:kv_len[n]].to(f64) * vs[h]
            for a in range(0, q_len[n], step):
                r = torch.arange(a, min(q_len[n], a + step), device="cuda")
                x = s["q"][t0 + r, h * G:(h + 1) * G].to(f64).reshape(-1, D) @ kh.t() / math.sqrt(D)
                x = x.view(len(r), G, -1)
                x = c["cap"] * torch.tanh(x / c["cap"]) if c["cap"] else x
                gap = (r + kv_len[n] - q_len[n])[:, None] - j
                if c["slopes"]:
                    x = x - gap.abs()[:, None] * s["slope"][h * G:(h + 1) * G].to(f64)[:, None]
                hide = (j < lo[r][:, None]) | (j >= hi[r][:, None])
                x = x.masked_fill(hide[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                w = torch.where(z.isinf()[..., None], torch.zeros_like(x), torch.exp(x - z[..., None]))
                out[t0 + r, h * G:(h + 1) * G] = (w.reshape(-1, kv_len[n]) @ vh).view(len(r), G, D)
                lse[t0 + r, h * G:(h + 1) * G] = z
        t0 += q_len[n]
    return out, lse
