"""Float64 definitions of the operators around a block's dense products and its
router: RMS norm, balance loss, low-rank adapters.  Plain numpy, arrays of float64 in
and out; gradients from the formulas (the tests check them against differences)."""

import numpy as np

from . import moe


# -------------------------------------------------------------------- RMS norm

def rms_norm(h, weight=None, eps=1e-6):
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None]
    return (y if weight is None else y * weight), rstd


def rms_norm_backward(dy, h, weight, rstd, grad_h=None):
    hr = h * rstd[:, None]
    a = dy if weight is None else dy * weight
    dx = rstd[:, None] * (a - hr * (a * hr).mean(1, keepdims=True))
    return (dx if grad_h is None else dx + grad_h), (dy * hr).sum(0)


# ---------------------------------------------------------------- balance loss

def probabilities(logits, score):
    """(p, used): softmax, or sigmoids divided by their sum; zeros in rows of -inf."""
    used = ~np.isneginf(logits).all(1)
    if score == "softmax":
        return moe.scores(logits, score), used
    # sigmoid(x) exp(-min(max x, 0)), whose sum float64 holds for any row
    top = np.minimum(np.where(used, logits.max(1), 0.0), 0.0)[:, None]
    s = np.exp(np.minimum(logits, 0.0) - top) / (1.0 + np.exp(-np.abs(logits)))
    total = s.sum(1, keepdims=True)
    return s / np.where(total == 0, 1.0, total), used


def runs(ends, T):
    ends = [T] if ends is None else [int(e) for e in ends]
    return list(zip([0] + ends[:-1], ends))


def balance_loss(logits, ids, score="softmax", coeff=1.0, ends=None):
    """(loss, counts [S, E], tokens [S])."""
    T, E = logits.shape
    p, used = probabilities(logits, score)
    counts, tokens, losses = [], [], []
    for begin, end in runs(ends, T):
        at = np.arange(begin, end)[used[begin:end]]
        c = np.bincount(ids[at][(ids[at] >= 0) & (ids[at] < E)], minlength=E)
        counts.append(c)
        tokens.append(len(at))
        if len(at):
            losses.append((E * c / (ids.shape[1] * len(at)) * p[at].mean(0)).sum())
    return coeff * np.mean(losses) if losses else 0.0, np.array(counts), np.array(tokens)


def balance_loss_backward(grad_loss, logits, counts, tokens, k, score="softmax", coeff=1.0, ends=None):
    T, E = logits.shape
    p, used = probabilities(logits, score)
    grad = np.zeros_like(logits)
    alive = max(1, (tokens > 0).sum())
    for (begin, end), c, n in zip(runs(ends, T), counts, tokens):
        at = np.arange(begin, end)[used[begin:end]]
        if len(at):
            d = grad_loss * coeff * E * c / (alive * k * float(n) ** 2)
            # sum_j p_j (d_e - d_j): no small difference of large numbers
            q = p[at]
            g = np.zeros_like(q)
            for e in range(E):
                g[:, e] = q[:, e] * (q * (d[e] - d)).sum(1)
            if score == "sigmoid":
                x = logits[at]
                g *= np.exp(np.minimum(-x, 0.0)) / (1.0 + np.exp(-np.abs(x)))
            grad[at] = g
    return grad


# -------------------------------------------------------------------- adapters

def lora(x, down, up, ids, scales=None, base=None):
    """(out [T, N], v [T, r])."""
    n, r, _ = down.shape
    out = np.zeros((x.shape[0], up.shape[2])) if base is None else base.copy()
    v = np.zeros((x.shape[0], r))
    for a in range(n):
        at = np.flatnonzero(ids == a)
        v[at] = x[at] @ down[a].T
        out[at] += (1.0 if scales is None else scales[a]) * (v[at] @ up[a])
    return out, v


def lora_backward(dy, x, down, up, ids, scales=None):
    """(dx, ddown, dup)."""
    dx, ddown, dup = np.zeros_like(x), np.zeros_like(down), np.zeros_like(up)
    for a in range(down.shape[0]):
        at = np.flatnonzero(ids == a)
        s = 1.0 if scales is None else scales[a]
        dv = s * (dy[at] @ up[a].T)
        dx[at] = dv @ down[a]
        ddown[a] = dv.T @ x[at]
        dup[a] = s * (x[at] @ down[a].T).T @ dy[at]
    return dx, ddown, dup
