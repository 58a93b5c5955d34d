"""The float64 definitions of the operators around the grouped GEMMs: hand-made
values, and every gradient formula against central differences (step 1e-6 in
float64: truncation and rounding both stay below 1e-7 of the gradient's scale)."""

import numpy as np
import pytest

from oracle import moe

TOL = 1e-7


def _differences(f, x, step=1e-6):
    """d f / d x for a scalar f, one element at a time."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += step
        down[i] -= step
        g[i] = (f(up) - f(down)) / (2 * step)
    return g


def _close(a, b):
    assert np.abs(a - b).max() <= TOL * max(1.0, np.abs(b).max()), np.abs(a - b).max()


def test_layer_norm_values():
    y, mean, rstd = moe.layer_norm(np.array([[1.0, 3.0]]), np.array([2.0, 2.0]), np.array([0.5, 0.5]), eps=3.0)
    assert mean.tolist() == [2.0] and rstd.tolist() == [0.5]
    assert y.tolist() == [[-0.5, 1.5]]


def test_layer_norm_gradient():
    r = np.random.default_rng(1)
    x, dy = r.standard_normal((3, 7)), r.standard_normal((3, 7))
    w, b = r.standard_normal(7), r.standard_normal(7)
    loss = lambda x, w, b: (moe.layer_norm(x, w, b)[0] * dy).sum()  # noqa: E731
    _, mean, rstd = moe.layer_norm(x, w, b)
    dx, dw, db = moe.layer_norm_backward(dy, x, w, mean, rstd)
    _close(dx, _differences(lambda v: loss(v, w, b), x))
    _close(dw, _differences(lambda v: loss(x, v, b), w))
    _close(db, _differences(lambda v: loss(x, w, v), b))


def test_route_ties_groups_and_empty_rows():
    inf = np.inf
    logits = np.array([[1.0, 1.0, 0.0, 1.0], [-inf] * 4, [-inf, 2.0, -inf, -inf]])
    ids, w, _ = moe.route(logits, 2)
    assert ids.tolist() == [[0, 1], [-1, -1], [1, -1]]
    assert np.allclose(w, [[0.5, 0.5], [0, 0], [1, 0]])
    # group 1 has the best expert, group 0 the best pair
    logits = np.array([[1.0, 1.0, 1.5, -9.0]])
    assert moe.route(logits, 1, groups=2, group_topk=1)[0].tolist() == [[2]]
    assert moe.route(logits, 1, score="sigmoid", groups=2, group_topk=1, group_score="top2")[0].tolist() == [[0]]
    # the bias chooses, the score weighs
    ids, w, _ = moe.route(np.array([[0.0, 0.0]]), 1, score="sigmoid", bias=np.array([0.0, 1.0]), renormalize=False)
    assert ids.tolist() == [[1]] and w.tolist() == [[0.5]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient(score, renormalize):
    r = np.random.default_rng(2)
    logits, grad = r.standard_normal((4, 6)), r.standard_normal((4, 3))
    ids, _, _ = moe.route(logits, 3, score=score)
    ids[1, 2] = -1
    ids[2] = -1
    f = lambda v: (moe.route_weights(v, ids, score, renormalize, 2.5) * grad).sum()  # noqa: E731
    _close(moe.route_backward(grad, logits, ids, score, renormalize, 2.5), _differences(f, logits))


def test_plan_and_permutation():
    ids = np.array([[2, 0], [-1, 2], [0, 5]])
    offsets, rows = moe.plan(ids, 4)
    assert offsets.tolist() == [2, 2, 4, 4]
    assert rows.tolist() == [[2, 0], [~4, 3], [1, ~5]]
    x = np.arange(6.0).reshape(3, 2) + 1
    d = moe.dispatch(x, rows)
    assert d[4:].tolist() == [[0, 0], [0, 0]] and d[0].tolist() == x[0].tolist() and d[3].tolist() == x[1].tolist()
    r = np.random.default_rng(3)
    v, g, w = r.standard_normal((6, 2)), r.standard_normal((3, 2)), r.standard_normal((3, 2))
    gr, gw = moe.combine_backward(g, v, rows, w)
    _close(gr, _differences(lambda a: (moe.combine(a, rows, w) * g).sum(), v))
    _close(gw, _differences(lambda a: (moe.combine(v, rows, a) * g).sum(), w))
    # dispatch's gradient is the unweighted combine
    gd = r.standard_normal((6, 2))
    _close(moe.combine(gd, rows), _differences(lambda a: (moe.dispatch(a, rows) * gd).sum(), x))


def test_swiglu_gradient():
    r = np.random.default_rng(4)
    x, g = r.standard_normal((2, 8)) * 3, r.standard_normal((2, 4))
    _close(moe.swiglu_backward(g, x), _differences(lambda v: (moe.swiglu(v) * g).sum(), x))
