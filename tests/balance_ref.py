"""The router's balance losses and their gradient in float64 numpy (test
helper)."""
import numpy as np


def probabilities(x, score):
    """(p, softmax, logsumexp, 1 - sigmoid) of logits x [T, E]; zeros for a
    token of -inf alone."""
    x = np.asarray(x, np.float64)
    m = x.max(1, keepdims=True)
    m = np.where(m == -np.inf, 0, m)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        z = np.exp(x - m)
        total = z.sum(1, keepdims=True)
        soft = np.where(total == 0, 0, z / total)
        lse = np.where(total == 0, 0, m + np.log(total))[:, 0]
        if score == "softmax":
            return soft, soft, lse, np.ones_like(x)
        # log sigmoid, relative to the token's largest
        s = np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))
        top = s.max(1, keepdims=True)
        z = np.exp(s - np.where(top == -np.inf, 0, top))
        total = z.sum(1, keepdims=True)
        return np.where(total == 0, 0, z / total), soft, lse, 1 / (1 + np.exp(x))


def tokens_of(T, mask, offsets):
    """Each sequence's tokens."""
    live = np.ones(T, bool) if mask is None else np.asarray(mask)
    cuts = [0, T] if offsets is None else np.clip(np.asarray(offsets), 0, T)
    return [np.nonzero(live[a:b])[0] + a for a, b in zip(cuts[:-1], cuts[1:])]


def balance(x, idx, score, mask=None, offsets=None):
    """(losses [2], counts, prob, tokens)."""
    (T, E), k = x.shape, idx.shape[1]
    p, _, lse, _ = probabilities(x, score)
    seqs = tokens_of(T, mask, offsets)
    counts = np.array([[(idx[t] == e).sum() for e in range(E)] for t in seqs])
    prob = np.array([p[t].mean(0) if len(t) else np.zeros(E) for t in seqs])
    n = np.array([len(t) for t in seqs])
    each = [E * (c / (k * m) * q).sum() for c, q, m in zip(counts, prob, n) if m]
    z = [(lse[t] ** 2).sum() for t in seqs]
    return np.array([np.mean(each) if each else 0, sum(z) / max(n.sum(), 1)]), counts, prob, n


def gradient(x, idx, score, dlosses, mask=None, offsets=None):
    (T, E), k = x.shape, idx.shape[1]
    p, soft, lse, rest = probabilities(x, score)
    seqs = tokens_of(T, mask, offsets)
    _, counts, _, n = balance(x, idx, score, mask, offsets)
    d = np.zeros((T, E))
    for t, c, m in zip(seqs, counts, n):
        if m:
            f = dlosses[0] * E * c / (k * m * m * (n > 0).sum())
            g = p[t] * (f - (f * p[t]).sum(1, keepdims=True))
            d[t] = g * rest[t] + 2 * dlosses[1] / n.sum() * lse[t][:, None] * soft[t]
    return d
