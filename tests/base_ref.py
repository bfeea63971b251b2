"""The base side's operators in float64 on the CPU, from their definitions, and the error
bounds that their roundings give."""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # a rounding's largest relative error
F32 = 2.0 ** -24


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def first_places(v, n):
    """Indices of the n largest of a row, equal values by ascending index; NaN as -inf."""
    v = np.where(np.isnan(v), -np.inf, v)
    return np.argsort(-v, kind="stable")[:n]


def route(logits, topk, score, bias=None, groups=1, kept=1, group_top=2, renorm=True, scale=1.0):
    """ids [T][topk] and weights [T][topk] (float64)."""
    x = f64(logits)
    T, E = x.shape
    ids, weights = np.zeros((T, topk), np.int64), np.zeros((T, topk))
    for t in range(T):
        masked = np.isnan(x[t]) | (x[t] == -np.inf)
        live = np.where(masked, -np.inf, x[t])
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "sigmoid":
                s = np.where(masked, 0.0, 1 / (1 + np.exp(-live)))
                whole = 1.0
            else:
                s = np.where(masked, 0.0, np.where(live == live.max(), 1.0, np.exp(live - live.max())))
                whole = s.sum()
        c = s / whole if whole > 0 else s
        if bias is not None:
            c = c + f64(bias)
        c = np.where(masked | np.isnan(c), -np.inf, c)
        order = c if bias is not None else live
        allowed = np.arange(E)
        if groups > 1 and kept < groups:
            by_group = (c if bias is not None or group_top > 1 else live).reshape(groups, -1)
            rank = -np.sort(-by_group, axis=1)[:, :group_top].sum(1)
            best = first_places(rank, kept)
            allowed = np.concatenate([np.arange(g * (E // groups), (g + 1) * (E // groups)) for g in sorted(best)])
        chosen = allowed[first_places(order[allowed], topk)]
        ids[t] = chosen
        whole = s[chosen].sum() if renorm else whole
        weights[t] = s[chosen] / whole * scale if whole > 0 else 0.0
        if np.isnan(x[t]).any():
            weights[t] = np.nan
    return ids, weights


def silu_mul(x):
    """The gated activation of gate | up, float64."""
    v = f64(x)
    gate, up = np.split(v, 2, axis=1)
    with np.errstate(over="ignore", invalid="ignore"):
        return gate / (1 + np.exp(-gate)) * up


def quantize(v):
    """Integers and scales of rows (float64 holding float32 values)."""
    q, scale = np.zeros(v.shape, np.int64), np.zeros(len(v), np.float32)
    for i, r in enumerate(v):
        m = np.abs(r).max()
        if not np.isfinite(r).all():
            scale[i] = np.nan
        elif m > 0:
            # 127 r has at most 31 bits: the quotient is rounded once, and lies on a half only where the real one does
            q[i] = np.rint(127 * r / m)
            scale[i] = np.float32(m) / np.float32(127)
    return q, scale


def int8_matmul(x, xs, w, ws, bias, expert, source, dtype):
    """y [rows][d_out] and its bound; expert -1: NaN (not written)."""
    x, w = f64(x), f64(w)                            # sums stay below 2^31: exact
    w = w.reshape((-1,) + w.shape[-2:])
    xs, ws = f64(xs), f64(ws).reshape(len(w), -1)
    b = None if bias is None else f64(bias).reshape(len(w), -1)
    y = np.full((len(expert), w.shape[1]), np.nan)
    bound = np.zeros_like(y)
    for e in np.unique(expert[expert >= 0]):
        rows = np.nonzero(expert == e)[0]
        sums = x[source[rows]] @ w[e].T
        p = sums * xs[source[rows], None] * ws[e]
        y[rows] = p if b is None else p + b[e]
        # in float32: the sum, the scales' product, their product, the bias; then y's own
        bound[rows] = 4 * F32 * (np.abs(p) + np.abs(y[rows])) + HALF[dtype] * np.abs(y[rows]) * (1 + 8 * F32) + 1e-37
    return y, bound


def combine(y, weights, ids, local, add, dtype):
    """out [T][width] and its bound; local: whether each id is."""
    T, K = ids.shape
    rows, w = f64(y).reshape(T, K, -1), f64(weights)
    size = np.zeros((T, rows.shape[2])) if add is None else np.abs(f64(add))
    out = np.zeros_like(size) if add is None else f64(add)
    for j in range(K):
        at = local[:, j]
        out[at] += w[at, j, None] * rows[at, j]
        size[at] += np.abs(w[at, j, None] * rows[at, j])
    # every term and every sum rounded once in float32
    return out, (K + 2) * F32 * size + HALF[dtype] * np.abs(out) * (1 + 2 * (K + 2) * F32) + 1e-37


def near(got, want, bound, what=""):
    got = f64(got)
    # a bound that is near a rounding border may fall to either side: one more of the float64's own errors
    bad = ~(np.abs(got - want) <= bound * (1 + 1e-6))
    bad &= ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]!r} for {want[bad][0]!r}, bound {bound[bad][0] if np.ndim(bound) else bound}")
