"""Routing and its gradient in float64 numpy over whole batches (test helper).

The gradient is written with the weights themselves: a slot's score has the
gradient ds_j, and p_j = ds_j s_j is scale dw_j s_j, or with renormalised
weights w_j = s_j / S

    p_j = scale w_j (dw_j - sum_i dw_i w_i),

which divides nothing but a score by the sum of the scores, so it stays finite
where S is so small that 1 / S is not.  Then dl_e = p_e (1 - s_e) for sigmoid
scores and p_e - s_e sum_j p_j for softmax, where the sum is 0 if the weights
are renormalised (they add up to 1)."""
import numpy as np


def scores(x, score):
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        m = np.fmax.reduce(x, axis=1, keepdims=True)
        z = np.where(x == -np.inf, 0.0, np.exp(x - m))
        total = z.sum(1, keepdims=True)
        return np.where(total == 0, 0.0, z / total)


def dlogits(x, idx, dw, o):
    T, E = x.shape
    s, t = scores(x, o.score), np.arange(T)[:, None]
    on = (idx >= 0) & (idx < E)
    e = np.where(on, idx, 0)
    with np.errstate(all="ignore"):
        sc = np.where(on, s[t, e], 0.0)
        d = np.where(on, np.asarray(dw, np.float64) * o.scale, 0.0)
        if o.renorm:
            total = sc.sum(1, keepdims=True)
            w = np.where(total == 0, 0.0, sc / total)
            p = w * (d - (d * w).sum(1, keepdims=True))
        else:
            p = d * sc
        out = np.zeros((T, E))
        np.add.at(out, (np.broadcast_to(t, idx.shape)[on], idx[on]), p[on])
        if o.score == "sigmoid":
            return out * (1.0 - s)
        # the rest of a row's sum of p is 0 under renorm; a NaN score keeps its row NaN
        return out - s * (0.0 if o.renorm else p.sum(1, keepdims=True))


def chosen_softmax(x, idx, dw, o):
    """Weights and gradient of the chosen logits where softmax weights are
    renormalised, from these logits alone: (w [T, k], p [T, k])."""
    z = np.take_along_axis(np.asarray(x, np.float64), idx, 1)
    w = np.exp(z - z.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    d = np.asarray(dw, np.float64)
    return w * o.scale, o.scale * w * (d - (d * w).sum(1, keepdims=True))


def route(x, k, o, bias=None):
    """Indices, weights, offsets and rows of finite logits, without groups or
    with a group's value its largest choice value."""
    s = scores(x, o.score)
    T, E = s.shape
    c = (s + (0.0 if bias is None else np.asarray(bias, np.float64))).astype(np.float32)
    if o.top_groups < o.groups:
        per = c.reshape(T, o.groups, -1)
        best = np.argsort(-per.max(2), axis=1, kind="stable")[:, :o.top_groups]
        shut = np.ones((T, o.groups), bool)
        np.put_along_axis(shut, best, False, 1)
        c = np.where(shut[:, :, None], -np.inf, per).reshape(T, E)
    idx = np.argsort(-c, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(s, idx, 1)
    w = (w / w.sum(1, keepdims=True) if o.renorm else w) * o.scale
    flat = idx.ravel()
    off = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    return idx, w, off, np.argsort(flat, kind="stable")
