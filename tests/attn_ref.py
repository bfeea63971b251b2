"""Plain float64 attention and cache append (numpy), written from the formulas in
the C header, and the error bounds that follow from the kernels' roundings."""
from __future__ import annotations

import math

import numpy as np
import torch

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2
F32_HALF = torch.finfo(torch.float32).eps / 2


def e4m3_round(x):
    """float64 -> nearest e4m3 value (ties to even, saturating; NaN stays)."""
    x = np.asarray(x, np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -40))), -6)
        step = 2.0 ** (e - 3)
        r = np.clip(np.where(np.isinf(x), np.sign(x) * 448.0, np.round(x / step) * step), -448, 448)
    return np.where(np.isnan(x), np.nan, r)


def append(qkv, hq, hkv, D, offsets, slot, k, v, k_scale=None, v_scale=None, table=None, pos=None, rot=0,
           interleaved=False, sections=None, e4m3=False, page_size=16):
    """Returns (q rows, k, v, bad count) in float64; k, v: [page][head][pos][dim]
    copies holding the values that stored numbers stand for divided by nothing
    (e4m3: the stored numbers themselves, before the scale)."""
    qkv = qkv.astype(np.float64)
    T = qkv.shape[0]
    q_out = np.full((T, hq * D), np.nan)
    k, v = k.astype(np.float64).copy(), v.astype(np.float64).copy()
    pages = k.shape[0]
    bad = 0
    for t in range(T):
        s = int(slot[t])
        is_bad = s < -1 or s >= pages * page_size
        if table is not None:
            is_bad |= any(not 0 <= int(pos[x][t]) < len(table) for x in range(len(pos)))
        if is_bad:
            bad += 1
            continue
        heads = [qkv[t, offsets[0] + h * D: offsets[0] + (h + 1) * D].copy() for h in range(hq)]
        heads += [qkv[t, offsets[1] + h * D: offsets[1] + (h + 1) * D].copy() for h in range(hkv)]
        if table is not None:
            half = rot // 2
            bounds = np.cumsum(sections)
            for x in heads:
                src = x.copy()
                for j in range(half):
                    ax = int(np.searchsorted(bounds, j, side="right"))
                    c, n = float(table[pos[ax][t]][j]), float(table[pos[ax][t]][half + j])
                    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
                    x[a], x[b] = src[a] * c - src[b] * n, src[b] * c + src[a] * n
        for h in range(hq):
            q_out[t, h * D:(h + 1) * D] = heads[h]
        if s >= 0:
            p, i = divmod(s, page_size)
            for h in range(hkv):
                vv = qkv[t, offsets[2] + h * D: offsets[2] + (h + 1) * D]
                ks = 1.0 if k_scale is None else float(k_scale[h])
                vs = 1.0 if v_scale is None else float(v_scale[h])
                k[p, h, i], v[p, h, i] = heads[hq + h] / ks, vv / vs
                if e4m3:
                    v[p, h, i] = e4m3_round(np.float32(vv) / np.float32(vs))
    return q_out, k, v, bad


class Batch:
    """A batch of sequences with random lengths, pages and contents."""

    def __init__(self, q_len, kv_len, hq, hkv, D, page, cache="bf16", layout="heads", seed=0, spare=3,
                 causal=True, window=0, prefix_len=None, key_lo=None, key_hi=None, groups=None, group_len=None):
        r = np.random.Generator(np.random.PCG64(seed))
        self.rng = r
        self.q_len, self.kv_len, self.hq, self.hkv, self.D, self.page = list(q_len), list(kv_len), hq, hkv, D, page
        self.cache, self.causal, self.window = cache, causal, window
        self.prefix_len, self.key_lo, self.key_hi = prefix_len, key_lo, key_hi
        self.groups, self.group_len = groups, group_len     # starts (with the end), lengths
        self.N, self.T = len(self.q_len), int(sum(self.q_len))
        self.q_start = np.concatenate([[0], np.cumsum(self.q_len)]).astype(np.int32)
        need = [-(-n // page) for n in self.kv_len]
        self.pages = sum(need) + spare
        ids = r.permutation(self.pages)
        self.table = np.full((self.N, max(need + [0]) + 1), -7, np.int32)
        at = 0
        for n in range(self.N):
            self.table[n, :need[n]] = ids[at:at + need[n]]
            at += need[n]
        shape = (self.pages, hkv, page, D) if layout == "heads" else (self.pages, page, hkv, D)
        dt = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}[cache]
        mk = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))  # noqa: E731
        self.k_store, self.v_store = mk(*shape).to(dt), mk(*shape).to(dt)
        self.layout = layout
        self.k_scale = self.v_scale = None
        if cache == "e4m3":
            self.k_scale = torch.from_numpy(r.uniform(0.5, 2, hkv).astype(np.float32))
            self.v_scale = torch.from_numpy(r.uniform(0.5, 2, hkv).astype(np.float32))
        self.q_dtype = torch.float32 if cache == "f32" else torch.bfloat16
        self.q = mk(self.T, hq, D).to(self.q_dtype)
        if groups:
            self.share()

    def share(self):
        """Every member of a group gets the group's keys: the same numbers in its
        own pages up to the last whole shared one, which it takes as they are."""
        k, v = self.views()
        for g in range(len(self.group_len)):
            first = self.groups[g]
            for n in range(first + 1, self.groups[g + 1]):
                for i in range(self.group_len[g]):
                    a, b = self.table[first, i // self.page], self.table[n, i // self.page]
                    k[b, :, i % self.page], v[b, :, i % self.page] = k[a, :, i % self.page], v[a, :, i % self.page]

    def views(self):
        if self.layout == "heads":
            return self.k_store, self.v_store
        return self.k_store.transpose(1, 2), self.v_store.transpose(1, 2)

    def limits(self, n, i):
        kv, t = self.kv_len[n], int(self.q_start[n]) + i
        p = kv - self.q_len[n] + i
        lo = max(0, p + 1 - self.window if self.window else 0, int(self.key_lo[t]) if self.key_lo is not None else 0)
        hi = p + 1 if self.causal else kv
        if self.prefix_len is not None:
            hi = max(hi, int(self.prefix_len[n]))
        if self.key_hi is not None:
            hi = min(hi, int(self.key_hi[t]))
        hi = min(hi, kv)
        return (lo, hi, p) if hi > lo else (0, 0, p)

    def reference(self, scale=None, cap=0.0, slopes=None, bad_seqs=()):
        """out, lse and the bounds of their errors, float64."""
        D, G = self.D, self.hq // self.hkv
        scale = D ** -0.5 if scale is None else scale
        kk, vv = (x.to(torch.float64).numpy() for x in self.views())
        q = self.q.to(torch.float64).numpy()
        out = np.zeros((self.T, self.hq, D))
        lse = np.full((self.T, self.hq), -np.inf)
        out_tol, lse_tol = np.zeros_like(out), np.zeros_like(lse)
        w_half = F32_HALF * 4 if self.cache == "f32" else BF16_HALF
        o_half = F32_HALF if self.cache == "f32" else BF16_HALF
        for n in range(self.N):
            if n in bad_seqs:
                continue
            pages = self.table[n]
            for i in range(self.q_len[n]):
                lo, hi, p = self.limits(n, i)
                j = np.arange(lo, hi)
                ids = pages[j // self.page]
                j, ids = j[(ids >= 0) & (ids < self.pages)], ids[(ids >= 0) & (ids < self.pages)]
                if len(j) == 0:
                    continue
                t = int(self.q_start[n]) + i
                for h in range(self.hq):
                    kh = h // G
                    K = kk[ids, kh, j % self.page] * (1.0 if self.k_scale is None else float(self.k_scale[kh]))
                    V = vv[ids, kh, j % self.page] * (1.0 if self.v_scale is None else float(self.v_scale[kh]))
                    x = (K @ q[t, h]) * scale
                    size = np.abs(K) @ np.abs(q[t, h]) * abs(scale)
                    if cap:
                        x = cap * np.tanh(x / cap)
                    if slopes is not None:
                        bias = float(slopes[h]) * np.abs(p - j)
                        x, size = x - bias, size + bias
                    with np.errstate(invalid="ignore"):
                        m = x.max()
                        w = np.exp(x - m)
                    s = w.sum()
                    lse[t, h] = m + math.log(s) if s > 0 else m
                    with np.errstate(invalid="ignore"):
                        out[t, h] = (w / s) @ V
                        spread = (w / s) @ np.abs(V)
                    # a score: D products in fp32, then a handful of operations on it
                    x_err = (D + 8) * F32_HALF * 2 * np.nan_to_num(size, posinf=0).max() + cap * 4 * F32_HALF + 8 * F32_HALF
                    lse_tol[t, h] = x_err + 8 * F32_HALF * (1 + abs(lse[t, h]))
                    out_tol[t, h] = (w_half + 2 * x_err + (8 + math.log2(len(j) + 1)) * 2 * F32_HALF) * spread \
                        + o_half * (np.abs(out[t, h]) + spread * (w_half + 2 * x_err))
        return out, lse, out_tol, lse_tol
