"""The grouped-product operators written out in 64 bits with numpy, one token and one group at a
time, and the error bounds of their 32- and 16-bit arithmetic."""
import numpy as np

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # half the spacing of the type's numbers
# one term of a 32-bit sum: the multiply-add units round to nearest (2^-24), the matrix units may cut
# off (2^-23); two roundings per term are allowed for
SUM = 2.0 ** -22


TINY = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}  # half a spacing below the type's normal range (f16's reaches into use)


def rounding(dtype, v):
    """The most that rounding v to the type changes it."""
    return np.maximum(U[dtype] * np.abs(v), TINY[dtype])


def scores(logits, score):
    l = np.asarray(logits, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    l = np.minimum(l, np.finfo(np.float32).max)
    s = np.zeros_like(l)
    for t in range(l.shape[0]):
        ok = l[t] > -np.inf
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s[t, ok] = 1.0 / (1.0 + np.exp(-l[t, ok]))
        elif ok.any():
            e = np.exp(l[t, ok] - l[t, ok].max())
            s[t, ok] = e / e.sum()
    return l, s


def route(logits, top_k, bias=None, score="softmax", groups=1, groups_kept=1, group_score="max", renormalise=True,
          scale=1.0):
    """ids, weights, and the smallest difference between two unequal values that were compared."""
    l, s = scores(logits, score)
    tokens, experts = l.shape
    ids = np.full((tokens, top_k), -1, np.int64)
    weights = np.zeros((tokens, top_k))
    gap = np.inf

    def closest(v):
        v = np.unique(np.round([x for x in v if np.isfinite(x)], 14))
        return np.diff(v).min() if len(v) > 1 else np.inf

    for t in range(tokens):
        c = l[t] if bias is None else np.where(l[t] > -np.inf, s[t] + np.asarray(bias, np.float64), -np.inf)
        per = experts // groups
        usable = list(range(experts))
        if groups_kept < groups:
            by = s[t] if bias is None and group_score == "top2" else c
            val = []
            for g in range(groups):
                m = sorted((by[e] for e in range(g * per, (g + 1) * per) if c[e] > -np.inf), reverse=True)
                val.append(-np.inf if not m else sum(m[:2]) if group_score == "top2" else m[0])
            gap = min(gap, closest(val))
            kept = sorted(range(groups), key=lambda g: (-np.round(val[g], 14), g))[:groups_kept]
            usable = [e for g in kept for e in range(g * per, (g + 1) * per)]
        if bias is not None:
            gap = min(gap, closest(c))
        best = sorted((e for e in usable if c[e] > -np.inf), key=lambda e: (-np.round(c[e], 14), e))[:top_k]
        best.sort()
        w = s[t, best]
        if renormalise:
            w = w / w.sum() if len(w) and w.sum() > 0 else 0 * w
        ids[t, :len(best)], weights[t, :len(best)] = best, w * scale
    return ids, weights, gap


def route_grad(logits, ids, grad, score, renormalise, scale):
    _, s = scores(logits, score)
    out = np.zeros_like(s)
    for t in range(s.shape[0]):
        at = [e for e in ids[t] if e >= 0]
        if not at:
            continue
        d = np.asarray(grad, np.float64)[t, :len(at)] * scale
        if renormalise:
            total = s[t, at].sum()
            d = (d - (d * s[t, at]).sum() / total) / total if total > 0 else 0 * d
        full = np.zeros(s.shape[1])
        full[at] = d
        out[t] = full * s[t] * (1 - s[t]) if score == "sigmoid" else s[t] * (full - (full * s[t]).sum())
    return out


def transpose(ids, groups):
    flat = np.asarray(ids).reshape(-1)
    order = [i for g in range(groups) for i in np.nonzero(flat == g)[0]]
    offsets = np.concatenate([[0], np.cumsum([(flat == g).sum() for g in range(groups)])])
    position = np.full(flat.shape, -1)
    position[order] = np.arange(len(order))
    order = np.array(order + [-1] * (len(flat) - len(order)))
    return offsets, order, position.reshape(np.asarray(ids).shape)


def product(x, w, ids, offsets, order):
    """y and the sum of absolute products of each element."""
    k = ids.shape[1]
    y = np.zeros((ids.size, w.shape[1]))
    mag = np.zeros_like(y)
    for g in range(w.shape[0]):
        p = slice(offsets[g], offsets[g + 1])
        rows = x[order[p] // k]
        y[p], mag[p] = rows @ w[g].T, np.abs(rows) @ np.abs(w[g]).T
    return y, mag
