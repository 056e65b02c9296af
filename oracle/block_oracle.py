"""FP64 restatement of the operators round the routed layer: norms with gate and
residual, the product with its epilogue, the balance loss and its gradient.
Shares no code with the library."""
import math

import numpy as np

_ERF = np.vectorize(math.erf, otypes=[np.float64])


def norm(v, w, b=None, kind="rms", eps=1e-6, offset=0.0):
    """Rows of v; returns (y, 1 / sqrt(mean square or variance + eps) [T][1])."""
    v = np.asarray(v, np.float64)
    with np.errstate(all="ignore"):
        if kind == "layer":
            v = v - v.mean(1, keepdims=True)
        r = 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
        y = v * r * (np.asarray(w, np.float64) + offset)
        if b is not None:
            y = y + np.asarray(b, np.float64)
    return y, r


def gate_of(gate, T, H):
    """A gate [T], [H], [T][H] or None as something that multiplies [T][H]; a float32 vector is per token."""
    if gate is None:
        return np.ones((1, 1))
    g = np.asarray(gate, np.float64)
    if g.ndim == 2:
        return g
    return g[:, None] if gate.dtype == np.float32 else g[None, :]


def residual(branch, res, gate=None, scale=1.0, rscale=1.0, post=None):
    """h, and the sum of its terms' magnitudes; post: settings of norm() for the branch."""
    a = np.asarray(branch, np.float64)
    T, H = a.shape
    if post is not None:
        a, _ = norm(a, **post)
    a = scale * gate_of(gate, T, H) * a
    r = rscale * np.asarray(res, np.float64) if res is not None else np.zeros_like(a)
    return r + a, np.abs(r) + np.abs(a)


def act(name, v):
    with np.errstate(all="ignore"):
        if name == "relu":
            return np.where(np.isnan(v), v, np.maximum(v, 0.0))
        sig = np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))
        if name == "sigmoid":
            return sig
        if name == "silu":
            return v * sig
        if name == "gelu":
            return 0.5 * v * (1.0 + _ERF(v / math.sqrt(2.0)))
        if name == "gelu_tanh":
            return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def linear(x, w, bias=None, name="none", res=None):
    """y, and sum |terms| of the product with |bias|."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    v, a = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        v, a = v + np.asarray(bias, np.float64), a + np.abs(np.asarray(bias, np.float64))
    y = act(name, v)
    return (y if res is None else y + np.asarray(res, np.float64)), a


def probabilities(l, score):
    """p [T][E], good [T], 1 - sigmoid(l) (or 1) of logits l; bad rows' p are 0."""
    l = np.asarray(l, np.float64)
    good = ~(np.isnan(l).any(1) | (l == np.inf).any(1)) & (l > -np.inf).any(1)
    p, rest = np.zeros(l.shape), np.ones(l.shape)
    for t in np.flatnonzero(good):
        if score == "softmax":
            e = np.exp(l[t] - l[t].max())
        else:  # log sigmoid(l) = min(l, 0) - log(1 + e^-|l|), so that no row vanishes
            ls = np.minimum(l[t], 0.0) - np.log1p(np.exp(-np.abs(l[t])))
            e = np.exp(ls - ls.max())
            rest[t] = -np.expm1(ls)
        p[t] = e / e.sum()
    return p, good, rest


def balance(l, ids, offsets, k, score="softmax", coef=1.0):
    """counts, tokens, mean, loss."""
    T, E = l.shape
    p, good, _ = probabilities(l, score)
    off = [0, T] if offsets is None else list(offsets)
    S = len(off) - 1
    counts, tokens, mean = np.zeros((S, E), np.int64), np.zeros(S, np.int64), np.zeros((S, E))
    parts = []
    for s in range(S):
        a, b = off[s], off[s + 1]
        for e in np.asarray(ids[a:b]).ravel():
            if 0 <= e < E:
                counts[s, e] += 1
        tokens[s] = good[a:b].sum()
        if tokens[s]:
            mean[s] = p[a:b].sum(0) / tokens[s]
            parts.append((E * counts[s] / (k * tokens[s]) * mean[s]).sum())
    return counts, tokens, mean, coef * (sum(parts) / len(parts) if parts else 0.0)


def balance_grad(l, offsets, k, counts, tokens, score="softmax", coef=1.0, grad=1.0):
    """d loss / d l [T][E], the magnitude its terms have, and which rows are of a sequence."""
    T, E = l.shape
    p, good, rest = probabilities(l, score)
    off = [0, T] if offsets is None else list(offsets)
    live = sum(1 for n in tokens if n > 0)
    d, m, inside = np.zeros((T, E)), np.zeros((T, E)), np.zeros(T, bool)
    for s in range(len(off) - 1):
        for t in range(off[s], off[s + 1]):
            inside[t] = True
            if good[t]:
                f = E * np.asarray(counts[s], np.float64) / (k * tokens[s])
                c = grad * coef / (live * tokens[s]) * p[t] * rest[t]
                dot = (f * p[t]).sum()
                d[t], m[t] = c * (f - dot), np.abs(c) * (f + dot)
    return d, m, inside
