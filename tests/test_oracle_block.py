"""The float64 definitions of oracle/block.py: gradients against differences, and
hand-computed points."""

import numpy as np
import pytest

from oracle import block


def _difference(f, x, step=1e-6):
    """d f / d x by central differences (f gives one number)."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        g[i] = (f(a) - f(b)) / (2 * step)
    return g


def test_rms_norm_points():
    y, rstd = block.rms_norm(np.array([[3.0, -4.0], [0.0, 0.0]]), np.array([2.0, 1.0]), 0.0 + 1e-6)
    assert np.allclose(rstd, [1 / np.sqrt(12.5 + 1e-6), 1e3])
    assert np.allclose(y, [[6 * rstd[0], -4 * rstd[0]], [0, 0]])


@pytest.mark.parametrize("weighted", [True, False])
def test_rms_norm_gradients(weighted):
    r = np.random.default_rng(1)
    h, dy, gh = r.standard_normal((3, 5)), r.standard_normal((3, 5)), r.standard_normal((3, 5))
    w = 1 + 0.3 * r.standard_normal(5) if weighted else None
    rstd = block.rms_norm(h, w)[1]
    dx, dw = block.rms_norm_backward(dy, h, w, rstd, gh)
    assert np.allclose(dx, _difference(lambda t: (block.rms_norm(t, w)[0] * dy + t * gh).sum(), h), atol=1e-7)
    if weighted:
        assert np.allclose(dw, _difference(lambda t: (block.rms_norm(h, t)[0] * dy).sum(), w), atol=1e-7)


def test_balance_loss_of_even_load_is_the_coefficient():
    """Equal probabilities and equal counts: E sum_e (1 / E) (1 / E) = 1."""
    E, T, k = 4, 8, 2
    ids = np.arange(T * k).reshape(T, k) % E
    for score in ("softmax", "sigmoid"):
        loss, counts, tokens = block.balance_loss(np.zeros((T, E)), ids, score, 0.5)
        assert np.isclose(loss, 0.5) and (counts == T * k // E).all() and tokens == [T]


def test_balance_loss_leaves_out_padding_and_rows_behind():
    r = np.random.default_rng(2)
    x = r.standard_normal((9, 4))
    ids = np.argsort(-x, 1)[:, :2]
    x[3], ids[3] = -np.inf, -1
    loss, counts, tokens = block.balance_loss(x, ids, ends=[4, 4, 7])
    assert tokens.tolist() == [3, 0, 3] and counts.sum(1).tolist() == [6, 0, 6]
    a = block.balance_loss(x[:3], ids[:3])[0]
    b = block.balance_loss(x[4:7], ids[4:7])[0]
    assert np.isclose(loss, (a + b) / 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_loss_gradient(score):
    r = np.random.default_rng(3)
    x = r.standard_normal((7, 5)) * 2
    ids = np.argsort(-x, 1)[:, :2]
    x[2], ids[2] = -np.inf, -1
    ends = [3, 6]
    _, counts, tokens = block.balance_loss(x, ids, score, 0.3, ends)
    g = block.balance_loss_backward(1.7, x, counts, tokens, 2, score, 0.3, ends)
    keep = [0, 1, 3, 4, 5, 6]

    def loss(t):
        full = x.copy()
        full[keep] = t
        return 1.7 * block.balance_loss(full, ids, score, 0.3, ends)[0]

    assert np.allclose(g[keep], _difference(loss, x[keep]), atol=1e-8)
    assert (g[2] == 0).all() and (g[6] == 0).all()


def test_probabilities_below_the_smallest_number():
    for score in ("softmax", "sigmoid"):
        p, used = block.probabilities(np.array([[-800.0, -801.0], [-np.inf, -np.inf]]), score)
        assert np.allclose(p[0], np.array([1, np.exp(-1)]) / (1 + np.exp(-1))) and used.tolist() == [True, False]
        assert (p[1] == 0).all()


@pytest.mark.parametrize("scaled", [True, False])
def test_lora_gradients(scaled):
    r = np.random.default_rng(4)
    x, dy = r.standard_normal((6, 4)), r.standard_normal((6, 5))
    down, up = r.standard_normal((3, 2, 4)), r.standard_normal((3, 2, 5))
    scales = np.array([0.5, 2.0, 1.5]) if scaled else None
    ids = np.array([2, -1, 0, 0, 2, 7])
    out, v = block.lora(x, down, up, ids, scales, dy)
    assert (out[[1, 5]] == dy[[1, 5]]).all() and (v[[1, 5]] == 0).all()
    dx, ddown, dup = block.lora_backward(dy, x, down, up, ids, scales)
    assert np.allclose(dx, _difference(lambda t: (block.lora(t, down, up, ids, scales)[0] * dy).sum(), x), atol=1e-7)
    assert np.allclose(ddown, _difference(lambda t: (block.lora(x, t, up, ids, scales)[0] * dy).sum(), down), atol=1e-7)
    assert np.allclose(dup, _difference(lambda t: (block.lora(x, down, t, ids, scales)[0] * dy).sum(), up), atol=1e-7)
    assert (ddown[1] == 0).all() and (dup[1] == 0).all()
