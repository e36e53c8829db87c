"""Routing from logits in float64 numpy, by its definition (test helper):
one token at a time, comparisons in Python's order."""
import numpy as np


def scores(row, score):
    x = np.asarray(row, dtype=np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        if np.all(x == -np.inf):
            return np.zeros_like(x)
        z = np.exp(x - np.fmax.reduce(x))   # one NaN makes the sum, and every score, NaN
        return z / z.sum()


def _order(values):
    """Indices by descending value, NaN last, ties to the lower index."""
    v = [(-np.inf if np.isnan(x) else float(x), 0 if np.isnan(x) else 1) for x in values]
    return sorted(range(len(v)), key=lambda i: (-v[i][1], -v[i][0] if v[i][1] else 0.0, i))


def choose(row, k, o, bias):
    s = scores(row, o.score)
    with np.errstate(all="ignore"):
        c = (s + (np.asarray(bias, np.float64) if bias is not None else 0.0)).astype(np.float32)
        E, G = len(c), o.groups
        allowed = set(range(E))
        if o.top_groups < G:
            per = E // G
            vals = []
            for g in range(G):
                mine = [c[g * per + i] for i in _order(c[g * per:(g + 1) * per])]
                vals.append(np.float32(mine[0] + mine[1]) if o.group_score == "top2" and per > 1 else mine[0])
            best = _order(vals)[:o.top_groups]
            allowed = {g * per + i for g in best for i in range(per)}
    idx = [e for e in _order(c) if e in allowed][:k]
    w = s[idx]
    if o.renorm:
        t = 0.0
        for v in w:
            t = t + v
        w = np.zeros_like(w) if t == 0 else w / t
    return idx, w * o.scale


def route(logits, k, o, bias=None):
    got = [choose(r, k, o, bias) for r in logits]
    idx = np.array([g[0] for g in got], dtype=np.int32)
    w = np.array([g[1] for g in got])
    flat = idx.ravel()
    offsets = np.zeros(logits.shape[1] + 1, dtype=np.int32)
    offsets[1:] = np.cumsum(np.bincount(flat, minlength=logits.shape[1]))
    return idx, w, offsets, np.argsort(flat, kind="stable").astype(np.int32)


def weights(row, idx, o):
    """The chosen experts' weights as a function of the logits (idx fixed)."""
    w = scores(row, o.score)[idx]
    return (w / w.sum() if o.renorm else w) * o.scale


def dlogits(logits, idx, dw, o):
    """The gradient by its formula."""
    out = np.zeros(logits.shape)
    for t, row in enumerate(logits):
        s = scores(row, o.score)
        w = s[idx[t]]
        d = np.asarray(dw[t], np.float64) * o.scale
        if o.renorm:
            total = w.sum()
            d = (d - (d * w).sum() / total) / total if total else np.zeros_like(d)
        ds = np.zeros_like(s)
        np.add.at(ds, idx[t], d)
        out[t] = ds * s * (1 - s) if o.score == "sigmoid" else s * (ds - (ds * s).sum())
    return out
