"""Float64 definitions of the operators around the grouped GEMMs: layer norm,
routing to experts, token permutation, gated activation.  Plain numpy, arrays
of float64 in and out; gradients from the formulas (the tests check them
against differences)."""

import numpy as np

RENORM_EPS = 1e-20


# ------------------------------------------------------------------ layer norm

def layer_norm(x, weight=None, bias=None, eps=1e-5):
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = 1.0 / np.sqrt(var + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd):
    xh = (x - mean[:, None]) * rstd[:, None]
    a = dy if weight is None else dy * weight
    dx = rstd[:, None] * (a - a.mean(1, keepdims=True) - xh * (a * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


# --------------------------------------------------------------------- routing

def scores(logits, score):
    with np.errstate(over="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-logits))
        top = logits.max(1, keepdims=True)
        e = np.exp(logits - np.where(np.isneginf(top), 0.0, top))
        total = e.sum(1, keepdims=True)
        return e / np.where(total == 0, 1.0, total)


def route(logits, k, score="softmax", bias=None, groups=1, group_topk=None, group_score="max", renormalize=True,
          scale=1.0):
    """(ids [T, k], weights [T, k], margin [T]): margin is the smallest gap
    between unequal keys (or group scores) at a place that decides the choice
    or its order; a row without one is inf.  NaN logits are not covered."""
    T, E = logits.shape
    group_topk = groups if group_topk is None else group_topk
    s = scores(logits, score)
    ids = np.full((T, k), -1, np.int64)
    weights = np.zeros((T, k))
    margin = np.full(T, np.inf)
    for t in range(T):
        value = s[t] + (0.0 if bias is None else bias)
        value = np.where(np.isneginf(logits[t]), -np.inf, value)
        key = logits[t].copy() if bias is None else value.copy()
        if group_topk < groups:
            size = E // groups
            if group_score == "max":
                top = np.array([key[g * size:(g + 1) * size].max() for g in range(groups)])
            else:
                top = np.empty(groups)
                for g in range(groups):
                    best = np.sort(value[g * size:(g + 1) * size])[::-1][:2]
                    best = best[~np.isneginf(best)]
                    top[g] = best.sum() if best.size else -np.inf
            order = sorted(range(groups), key=lambda g: (-top[g], g))
            if not (group_score == "max" and bias is None):
                a, b = top[order[group_topk - 1]], top[order[group_topk]]
                if a != b and np.isfinite(b):
                    margin[t] = min(margin[t], a - b)
            for g in order[group_topk:]:
                key[g * size:(g + 1) * size] = -np.inf
        order = sorted(range(E), key=lambda e: (-key[e], e))
        if bias is not None:
            for a, b in zip(order[:k], order[1:k + 1]):
                if key[a] != key[b] and np.isfinite(key[b]):
                    margin[t] = min(margin[t], key[a] - key[b])
        for j, e in enumerate(order[:k]):
            if np.isneginf(key[e]):
                break
            ids[t, j] = e
            weights[t, j] = s[t, e]
    if renormalize:
        weights = weights / (weights.sum(1, keepdims=True) + RENORM_EPS)
    return ids, weights * scale, margin


def route_weights(logits, ids, score, renormalize, scale):
    """The weights of given ids (the function that the gradient is of)."""
    s = scores(logits, score)
    used = ids >= 0
    w = np.take_along_axis(s, np.where(used, ids, 0), 1) * used
    if renormalize:
        w = w / (w.sum(1, keepdims=True) + RENORM_EPS)
    return w * scale


def route_backward(grad, logits, ids, score, renormalize, scale):
    s = scores(logits, score)
    used = ids >= 0
    at = np.where(used, ids, 0)
    chosen = np.take_along_axis(s, at, 1) * used
    d = grad * used * scale
    if renormalize:
        total = chosen.sum(1, keepdims=True) + RENORM_EPS
        d = (d - (d * chosen).sum(1, keepdims=True) / total) / total * used
    de = np.zeros_like(s)
    np.add.at(de, (np.arange(len(s))[:, None], at), d)
    if score == "sigmoid":
        return s * scores(-logits, score) * de       # 1 - s, without its cancellation
    return s * (de - (s * de).sum(1, keepdims=True))


# ----------------------------------------------------------------- permutation

def plan(ids, experts):
    """(offsets [experts], row_of_slot [T, k]), ~row for slots without an expert."""
    flat = ids.reshape(-1)
    none = (flat < 0) | (flat >= experts)
    key = np.where(none, experts, flat)
    order = np.argsort(key, kind="stable")
    row = np.empty(flat.size, np.int64)
    row[order] = np.arange(flat.size)
    offsets = np.cumsum(np.bincount(key, minlength=experts + 1)[:experts])
    return offsets, np.where(none, ~row, row).reshape(ids.shape)


def dispatch(x, row_of_slot):
    T, k = row_of_slot.shape
    out = np.zeros((T * k, x.shape[1]), x.dtype)
    for t in range(T):
        for j in range(k):
            if row_of_slot[t, j] >= 0:
                out[row_of_slot[t, j]] = x[t]
    return out


def combine(rows, row_of_slot, weights=None):
    T, k = row_of_slot.shape
    out = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            r = row_of_slot[t, j]
            if r >= 0:
                out[t] += rows[r] * (1.0 if weights is None else weights[t, j])
    return out


def combine_backward(grad, rows, row_of_slot, weights=None):
    T, k = row_of_slot.shape
    gr = np.zeros((T * k, grad.shape[1]))
    gw = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = row_of_slot[t, j]
            if r >= 0:
                gr[r] = grad[t] * (1.0 if weights is None else weights[t, j])
                gw[t, j] = grad[t] @ rows[r]
    return gr, gw


# ------------------------------------------------------------ gated activation

def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def swiglu(x):
    gate, up = np.split(x, 2, axis=1)
    return gate * sigmoid(gate) * up


def swiglu_backward(grad_h, x):
    gate, up = np.split(x, 2, axis=1)
    sig = sigmoid(gate)
    return np.concatenate([grad_h * up * sig * (1.0 + gate * (1.0 - sig)), grad_h * gate * sig], 1)
