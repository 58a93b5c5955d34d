"""The operators around the grouped GEMMs against their float64 definitions.

Tolerances are worst-case bounds of float32 evaluation, U = 2^-24: a sum of n
terms whose longest chain of additions is D is off by at most D U sum|terms|;
bf16 results add half a bf16 ulp, 2^-8 |y|.  Whole numbers, dispatched rows and
checkpoint codes are exact."""

import numpy as np
import pytest
import torch

import precision_matmul_amd as fp8mm
from oracle import e4m3, moe
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8         # 8 significant bits: half an ulp is at most 2^-8 of the value
TINY = 1e-37            # results that are subnormal in float32 may be flushed ...
FLUSH = 2.0 ** -126     # ... and so may a sigmoid below the smallest normal number
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _dev(a, dtype):
    """float64 numpy -> (device tensor of dtype, the float64 values it holds)."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)
    return t, t.double().cpu().numpy()


def _strided(t, left=3, right=5):
    """The same values as columns [left, left + C) of a wider matrix: rows
    start at any element and the row stride is not the width."""
    wide = torch.full((t.shape[0], t.shape[1] + left + right), float("nan"), dtype=t.dtype, device=t.device)
    view = wide[:, left:left + t.shape[1]]
    view.copy_(t)
    return view


def _f64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def _within(got, ref, tol, what):
    off = np.abs(got - ref)
    bad = ~(off <= tol)
    worst = np.nanmax(off / np.maximum(tol, 1e-300)) if off.size else 0.0
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {worst:.3g} x"


def _depth(C):
    """Longest chain of additions of a row sum: a lane's own elements (at most
    32 in registers, C / 256 in the long form), then the wave and the waves."""
    return max(32, C / 256) + 6 + 4


# ------------------------------------------------------------------ layer norm

NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (4, 513), (9, 1024), (2, 1413), (7, 2048), (6, 2049), (5, 4104), (3, 5120),
               (2, 6200), (3, 8192), (2, 8193), (2, 20001)]


def _check_norm_forward(x, xv, w, wv, b, bv, eps, dtype):
    R, C = xv.shape
    half, D = BF16 if dtype == "bf16" else U, _depth(C) + 4
    y, mean, rstd = fp8mm.layer_norm_forward(x, w, b, eps)
    ref, rmean, rrstd = moe.layer_norm(xv, wv, bv, eps)
    wa = np.ones(C) if wv is None else np.abs(wv)
    ba = np.zeros(C) if bv is None else np.abs(bv)
    e_mean = D * U * np.abs(xv).mean(1)
    std = 1 / rrstd
    e_rstd = rrstd * (2 * e_mean / std + D * U)
    _within(_f64(mean), rmean, e_mean, "mean")
    _within(_f64(rstd), rrstd, e_rstd, "rstd")
    xh = (xv - rmean[:, None]) * rrstd[:, None]
    tol = wa * (rrstd * e_mean)[:, None] + np.abs(xh) * wa * (e_rstd / rrstd + 6 * U)[:, None] + 4 * U * ba
    _within(_f64(y), ref, tol + half * np.abs(ref) * (1 + half) + half * tol + TINY, "y")
    return y, mean, rstd


def _check_norm_backward(x, xv, dy, dyv, w, wv, mean, rstd, dtype, params):
    """layer_norm_backward against the formula with the same mean and rstd."""
    R, C = xv.shape
    half, D = BF16 if dtype == "bf16" else U, _depth(C) + 4
    wa = np.ones(C) if wv is None else np.abs(wv)
    m32, r32 = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    dx, dw, db = fp8mm.layer_norm_backward(dy, x, w, mean, rstd)
    rdx, rdw, rdb = moe.layer_norm_backward(dyv, xv, wv, m32, r32)
    a = np.abs(dyv) * wa
    xh = np.abs((xv - m32[:, None]) * r32[:, None])
    mx = (a * xh).mean(1, keepdims=True)
    tol = r32[:, None] * (6 * U * a + D * U * a.mean(1, keepdims=True) + (D + 10) * U * xh * mx + 6 * U * xh * mx)
    _within(_f64(dx), rdx, tol + half * np.abs(rdx) * (1 + half) + half * tol + TINY, "dx")
    p_half = BF16 if params == "bf16" else U
    n = R + 24            # rows of one workgroup, its waves, the partial rows: at most R + 24 in a chain
    tol = (n + 4) * U * (np.abs(dyv) * xh).sum(0)
    _within(_f64(dw), rdw, tol + p_half * np.abs(rdw) + p_half * tol + TINY, "dweight")
    tol = n * U * np.abs(dyv).sum(0)
    _within(_f64(db), rdb, tol + p_half * np.abs(rdb) + p_half * tol + TINY, "dbias")
    return dx, dw, db


@pytest.mark.parametrize("params", ["bf16", "fp32"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,C", [(512, 100), (513, 100), (600, 513), (530, 1024), (521, 2047), (519, 2049), (520, 3560),
                                 (515, 4104), (514, 6200), (516, 8190)])
def test_layer_norm_backward_of_many_rows(R, C, dtype, params):
    """Both sides of the step from one launch to partial sums, in every width."""
    say(f"layer norm backward {R}x{C} {dtype} params {params}")
    r = np.random.default_rng(R + C)
    x, xv = _dev(r.standard_normal((R, C)) + r.standard_normal((R, 1)), DT[dtype])
    dy, dyv = _dev(r.standard_normal((R, C)), DT[dtype])
    w, wv = _dev(1 + 0.3 * r.standard_normal(C), DT[params])
    _, mean, rstd = fp8mm.layer_norm_forward(x, w)
    out = _check_norm_backward(x, xv, dy, dyv, w, wv, mean, rstd, dtype, params)
    for got, want in zip(fp8mm.layer_norm_backward(_strided(dy, 1, 2), _strided(x), w, mean, rstd), out):
        assert torch.equal(got, want)


@pytest.mark.parametrize("params", ["bf16", "fp32", None])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,C", NORM_SHAPES)
def test_layer_norm(R, C, dtype, params):
    say(f"layer norm {R}x{C} {dtype} params {params}")
    r = np.random.default_rng(R * 100003 + C)
    x, xv = _dev(r.standard_normal((R, C)) * 1.5 + r.standard_normal((R, 1)), DT[dtype])
    dy, dyv = _dev(r.standard_normal((R, C)), DT[dtype])
    w = b = wv = bv = None
    if params:
        w, wv = _dev(1 + 0.3 * r.standard_normal(C), DT[params])
        b, bv = _dev(r.standard_normal(C), DT[params])
    eps = 1e-5
    y, mean, rstd = _check_norm_forward(x, xv, w, wv, b, bv, eps, dtype)
    dx, dw, db = _check_norm_backward(x, xv, dy, dyv, w, wv, mean, rstd, dtype, params)
    # rows at any stride and start: the same bits
    ys, _, _ = fp8mm.layer_norm_forward(_strided(x), w, b, eps)
    assert torch.equal(ys, y)
    for got, want in zip(fp8mm.layer_norm_backward(_strided(dy, 1, 2), _strided(x), w, mean, rstd), (dx, dw, db)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("R,C,dtype", [(5000, 64, "fp32"), (4500, 1001, "bf16"), (2100, 3557, "bf16"),
                                       (1500, 5120, "bf16"), (1200, 8191, "fp32"), (17000, 2048, "bf16")])
def test_layer_norm_of_more_rows_than_workgroups(R, C, dtype):
    """Workgroups take further rows in turns; the last case is large enough for
    streaming accesses."""
    say(f"layer norm {R}x{C} {dtype}")
    r = np.random.default_rng(C)
    x, xv = _dev(r.standard_normal((R, C), dtype=np.float32) + r.standard_normal((R, 1), dtype=np.float32), DT[dtype])
    w, wv = _dev(1 + 0.3 * r.standard_normal(C), torch.float32)
    _, mean, rstd = _check_norm_forward(x, xv, w, wv, None, None, 1e-5, dtype)
    dy, dyv = _dev(r.standard_normal((R, C), dtype=np.float32), DT[dtype])
    _check_norm_backward(x, xv, dy, dyv, w, wv, mean, rstd, dtype, "fp32")


@pytest.mark.parametrize("R,C,dtype", [(600, 4097, "fp32"), (600, 6144, "fp32"), (1800, 4764, "fp32"),
                                       (1800, 4762, "fp32"), (1500, 6148, "fp32"), (1100, 8192, "fp32"),
                                       (1100, 7999, "fp32"), (2800, 3003, "fp32"), (700, 4096, "fp32"), (700, 6152, "bf16"),
                                       (8200, 2056, "bf16"), (4000, 4104, "bf16"),
                                       (2400, 7177, "bf16")])
def test_layer_norm_of_rows_shared_by_waves(R, C, dtype):
    """Rows of four and of eight waves, whole and ending within a chunk, with
    plain and (more than 32 MiB) with streaming accesses."""
    say(f"layer norm {R}x{C} {dtype}")
    r = np.random.default_rng(R + C)
    x, xv = _dev(r.standard_normal((R, C), dtype=np.float32) + r.standard_normal((R, 1), dtype=np.float32), DT[dtype])
    w, wv = _dev(1 + 0.3 * r.standard_normal(C), torch.float32)
    b, bv = _dev(r.standard_normal(C), torch.float32)
    y, mean, rstd = _check_norm_forward(x, xv, w, wv, b, bv, 1e-5, dtype)
    dy, dyv = _dev(r.standard_normal((R, C), dtype=np.float32), DT[dtype])
    grads = _check_norm_backward(x, xv, dy, dyv, w, wv, mean, rstd, dtype, "fp32")
    assert torch.equal(fp8mm.layer_norm_forward(_strided(x), w, b, 1e-5)[0], y)
    for got, want in zip(fp8mm.layer_norm_backward(_strided(dy, 1, 2), _strided(x), w, mean, rstd), grads):
        assert torch.equal(got, want)


def test_swiglu_code_scales_are_those_of_float32_values():
    """A block's scale is max|h| / 448 of h = gate / (1 + exp(-gate)) up: the
    hardware's exp2 is within 2 U, its correction, the sum, the product and the
    scale's division add 1 U each, the quotient less than 2 U: 8 U bounds it."""
    say("swiglu scales 64x1024")
    r = np.random.default_rng(12)
    gate = r.uniform(-60, 60, (64, 1024)) * r.random((64, 1))
    gate[0] = -np.abs(gate[0])
    x, xv = _dev(np.concatenate([gate, r.standard_normal((64, 1024))], 1), torch.bfloat16)
    (_, scale), _ = fp8mm.fp8_swiglu_forward(x, "fp8", checkpoint=False)
    g, u = xv[:, :1024], xv[:, 1024:]
    ref = np.abs(g / (1 + np.exp(-g)) * u).reshape(64, 8, 128).max(2) / 448
    _within(_f64(scale).T, ref, 8 * U * ref, "scale")


@pytest.mark.parametrize("C", [64, 2048, 5120, 9000])
def test_layer_norm_gradients_over_many_rows(C):
    """More rows than one turn of the workgroups; partial results in a fixed
    order, so that a second call gives the same bits."""
    R = 2500
    say(f"layer norm backward {R}x{C}")
    r = np.random.default_rng(C)
    x, xv = _dev(r.standard_normal((R, C)), torch.bfloat16)
    dy, dyv = _dev(r.standard_normal((R, C)), torch.bfloat16)
    _, mean, rstd = fp8mm.layer_norm_forward(x)
    out = fp8mm.layer_norm_backward(dy, x, None, mean, rstd)
    again = fp8mm.layer_norm_backward(dy, x, None, mean, rstd)
    m, s = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    rdx, rdw, rdb = moe.layer_norm_backward(dyv, xv, None, m, s)
    xh = np.abs((xv - m[:, None]) * s[:, None])
    _within(_f64(out[1]), rdw, (R + 28) * U * (np.abs(dyv) * xh).sum(0), "dweight")
    _within(_f64(out[2]), rdb, (R + 24) * U * np.abs(dyv).sum(0), "dbias")
    for a, b in zip(out, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,C", [(5, 1), (6, 100), (3, 1152), (4, 2056), (600, 3), (600, 513), (530, 1152), (520, 2056),
                                 (515, 4099), (2, 8200), (3, 8203)])
def test_layer_norm_backward_of_rows_of_one_large_value(R, C, dtype):
    """x - mean is 0 in the row, and mean rstd = 2^110 1e6 is past float32's range:
    dx = rstd (dy - mean dy), with the places past the row's end out of the sums."""
    say(f"layer norm backward of constant rows {R}x{C} {dtype}")
    x = torch.full((R, C), 2.0 ** 110, dtype=DT[dtype], device=DEV)
    dy, dyv = _dev(np.random.default_rng(C).standard_normal((R, C)), DT[dtype])
    _, mean, rstd = fp8mm.layer_norm_forward(x, eps=1e-12)
    assert bool((mean == 2.0 ** 110).all())                 # the sums of equal powers of two are exact here
    _check_norm_backward(x, np.full((R, C), 2.0 ** 110), dy, dyv, None, None, mean, rstd, dtype, "fp32")


def test_layer_norm_empty_and_partial_results():
    x = torch.empty((0, 130), dtype=torch.bfloat16, device=DEV)
    y, mean, rstd = fp8mm.layer_norm_forward(x)
    assert y.shape == (0, 130) and mean.shape == (0,)
    _, dw, db = fp8mm.layer_norm_backward(x, x, None, mean, rstd)
    assert not _f64(dw).any() and not _f64(db).any()
    x = torch.randn((4, 130), device=DEV)
    y, mean, rstd = fp8mm.layer_norm_forward(x)
    full = fp8mm.layer_norm_backward(y, x, None, mean, rstd)
    assert fp8mm.layer_norm_backward(y, x, None, mean, rstd, need_params=False)[1] is None
    assert torch.equal(fp8mm.layer_norm_backward(y, x, None, mean, rstd, need_params=False)[0], full[0])
    assert torch.equal(fp8mm.layer_norm_backward(y, x, None, mean, rstd, need_dx=False)[1], full[1])


def test_layer_norm_autograd_and_non_finite_rows():
    r = np.random.default_rng(5)
    x, xv = _dev(r.standard_normal((2, 3, 96)), torch.float32)
    w, wv = _dev(1 + 0.1 * r.standard_normal(96), torch.float32)
    b = torch.zeros(96, device=DEV)
    g, gv = _dev(r.standard_normal((2, 3, 96)), torch.float32)
    for t in (x, w, b):
        t.requires_grad_(True)
    fp8mm.layer_norm(x, w, b).backward(g)
    _, mean, rstd = moe.layer_norm(xv.reshape(6, 96), wv)
    dx, dw, db = moe.layer_norm_backward(gv.reshape(6, 96), xv.reshape(6, 96), wv, mean, rstd)
    for got, ref in ((x.grad.reshape(6, 96), dx), (w.grad, dw), (b.grad, db)):
        _within(_f64(got), ref, 200 * U * np.abs(ref).max(), "gradient")
    # a NaN or an infinity stays in its row
    x = torch.randn((4, 640), device=DEV)
    x[1, 5], x[2, 639] = float("nan"), float("inf")
    y, _, _ = fp8mm.layer_norm_forward(x)
    bad = torch.isnan(y).all(1)
    assert bad.tolist() == [False, True, True, False] and bool(torch.isfinite(y[[0, 3]]).all())


# --------------------------------------------------------------------- routing

ROUTE = [
    # T, E, k, score, bias, groups, group_topk, group_score
    (1, 1, 1, "softmax", False, 1, 1, "max"),
    (3, 8, 8, "softmax", False, 1, 1, "max"),
    (5, 60, 6, "sigmoid", False, 1, 1, "max"),
    (17, 64, 6, "softmax", True, 1, 1, "max"),
    (6, 65, 4, "softmax", False, 1, 1, "max"),
    (9, 128, 8, "sigmoid", True, 4, 2, "max"),
    (12, 182, 2, "sigmoid", True, 1, 1, "max"),
    (33, 256, 8, "sigmoid", True, 8, 4, "top2"),
    (7, 160, 6, "softmax", False, 8, 3, "max"),
    (7, 160, 6, "softmax", False, 8, 3, "top2"),
    (5, 66, 3, "sigmoid", False, 33, 5, "top2"),
    (4, 64, 4, "sigmoid", False, 64, 6, "max"),
    (5, 300, 12, "softmax", True, 3, 2, "top2"),
    (4, 1000, 64, "sigmoid", True, 1, 1, "max"),
    (3, 1024, 16, "softmax", False, 16, 2, "max"),
    (18, 64, 8, "sigmoid", True, 8, 2, "top2"),
    (19, 240, 8, "sigmoid", True, 15, 4, "top2"),
    (35, 256, 16, "softmax", False, 2, 1, "max"),
    (6, 200, 40, "sigmoid", True, 1, 1, "max"),
    (5, 128, 20, "softmax", False, 8, 4, "max"),
    (4, 60, 17, "softmax", True, 1, 1, "max"),
    (64, 9, 3, "sigmoid", False, 3, 2, "top2"),
]


def _route_data(T, E, bias, dtype, seed):
    r = np.random.default_rng(seed)
    grid = np.round(r.standard_normal((T, E)) * 16) / 16       # exact in bf16; equal logits are common
    logits, lv = _dev(grid, DT[dtype])
    b = bv = None
    if bias:
        b, bv = _dev(np.round(r.standard_normal(E) * 40) / 512, torch.float32)
    return logits, lv, b, bv


def _score_tol(lv):
    """Relative: the exponent's argument is off by U |x - max|, exp and the
    division by a few U, the softmax sum by its depth."""
    return (np.ptp(lv) + lv.shape[1] / 64 + 6 + 16) * 2 * U


@pytest.mark.parametrize("renormalize,scale", [(True, 1.0), (False, 2.5)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", ROUTE)
def test_route(case, dtype, renormalize, scale):
    T, E, k, score, bias, groups, group_topk, group_score = case
    say(f"route {case} {dtype} renormalize {renormalize}")
    logits, lv, b, bv = _route_data(T, E, bias, dtype, E * 1000 + k)
    ids, w = fp8mm.moe_route_forward(logits, k, score, b, groups, group_topk, group_score, renormalize, scale)
    rids, rw, margin = moe.route(lv, k, score, bv, groups, group_topk, group_score, renormalize, scale)
    clear = margin > 64 * U        # keys below 2 with errors of a few U each
    assert clear.mean() >= 0.6
    assert np.array_equal(ids.cpu().numpy()[clear], rids[clear])
    _within(_f64(w)[clear], rw[clear], 2 * _score_tol(lv) * np.abs(rw[clear]) + TINY, "weights")
    # rows at any stride
    ids2, w2 = fp8mm.moe_route_forward(_strided(logits, 1, 2), k, score, b, groups, group_topk, group_score,
                                       renormalize, scale)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)

    r = np.random.default_rng(7)
    g, gv = _dev(r.standard_normal((T, k)), torch.float32)
    back = ids.clone()
    if k > 1:
        back[0, -1] = -1           # an empty slot
    grad = fp8mm.moe_route_backward(g, logits, back, score, renormalize, scale)
    at = back.cpu().numpy().astype(np.int64)
    ref = moe.route_backward(gv, lv, at, score, renormalize, scale)
    # the terms that cancel: |d_e| s_e and s_e sum |s d|, d bounded by 2 scale |g| / S
    s = moe.scores(lv, score)
    chosen = np.take_along_axis(s, np.where(at >= 0, at, 0), 1) * (at >= 0)
    S = chosen.sum(1, keepdims=True) if renormalize else np.ones((T, 1))
    size = 2 * scale * np.abs(gv).max(1, keepdims=True) / np.maximum(S, 1e-20)
    tol = s * size * (1 + chosen.sum(1, keepdims=True)) * 4 * (_score_tol(lv) + 64 * U)
    half = BF16 if dtype == "bf16" else U
    _within(_f64(grad), ref, tol + half * np.abs(ref) + TINY, "grad_logits")
    assert torch.equal(fp8mm.moe_route_backward(g, _strided(logits, 1, 2), back, score, renormalize, scale), grad)


def test_route_rows_with_few_or_no_experts():
    inf = float("inf")
    logits = torch.full((5, 70), -inf, device=DEV)
    logits[1, 3] = 2.0
    logits[2, 69], logits[2, 0] = 1.0, 1.0
    logits[3] = torch.finfo(torch.float32).min
    logits[4, 10:] = 0.0
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(70, device=DEV)):
            ids, w = fp8mm.moe_route_forward(logits, 3, score, bias)
            assert ids.tolist()[:3] == [[-1, -1, -1], [3, -1, -1], [0, 69, -1]]
            assert ids.tolist()[3] == [0, 1, 2] and ids.tolist()[4] == [10, 11, 12]
            assert w[0].tolist() == [0, 0, 0] and w[1].tolist() == [1, 0, 0]
            assert torch.allclose(w[2], torch.tensor([0.5, 0.5, 0], device=DEV))
            assert torch.allclose(w[4], torch.full((3,), 1 / 3, device=DEV))
            grad = fp8mm.moe_route_backward(torch.ones((5, 3), device=DEV), logits, ids, score, renormalize=False)
            assert bool(torch.isfinite(grad).all()) and not bool(grad[0].any())
    # groups without an eligible expert come last, and give nothing
    logits = torch.full((1, 8), -inf, device=DEV)
    logits[0, 5] = -3.0
    ids, _ = fp8mm.moe_route_forward(logits, 2, groups=4, group_topk=2, group_score="top2")
    assert ids.tolist() == [[5, -1]]
    # a bias of -inf takes an expert out
    bias = torch.zeros(8, device=DEV)
    bias[2] = -inf
    ids, _ = fp8mm.moe_route_forward(torch.zeros((1, 8), device=DEV), 3, "sigmoid", bias)
    assert ids.tolist() == [[0, 1, 3]]


def test_route_undefined_rows_show():
    logits = torch.zeros((4, 100), device=DEV)
    logits[1, 70] = float("nan")
    logits[2, 99] = float("inf")
    ids, w = fp8mm.moe_route_forward(logits, 2)
    assert ids.tolist() == [[0, 1]] * 4
    assert torch.isnan(w).all(1).tolist() == [False, True, True, False]
    ids, w = fp8mm.moe_route_forward(logits, 2, "sigmoid")
    assert ids.tolist() == [[0, 1], [0, 1], [99, 0], [0, 1]]
    assert torch.isnan(w).any(1).tolist() == [False, True, False, False]


@pytest.mark.parametrize("E", [100, 300])
def test_route_gradients_of_undefined_rows_show(E):
    logits = torch.zeros((4, E), device=DEV)
    logits[1, 70], logits[2, E - 1] = float("nan"), float("inf")
    ids = torch.tensor([[0, 1]] * 4, dtype=torch.int32, device=DEV)
    g = torch.ones((4, 2), device=DEV)
    for score, bad in (("softmax", [False, True, True, False]), ("sigmoid", [False, True, False, False])):
        grad = fp8mm.moe_route_backward(g, logits, ids, score, renormalize=False)
        assert torch.isnan(grad).all(1).tolist() == bad and torch.isnan(grad).any(1).tolist() == bad


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E", [24, 256, 300])
def test_route_gradients_of_saturated_sigmoids(E, dtype):
    """Slopes where the sigmoid is near 0 or 1, relative to themselves.  e =
    exp(-|x|) is off by 4 U (the hardware's exp2 2 U, its correction and the
    rounding of the sum), 1 + e by 5 U, its reciprocal by 7 U, e r r by 4 + 14 + 2
    U, the products with scale and gradient by 2 U more: 24 U bounds it."""
    say(f"route gradients of saturated sigmoids E={E} {dtype}")
    r = np.random.default_rng(E)
    size = np.array([0.0, 1.0, 4.0, 8.0, 10.0, 12.0, 16.0, 17.0, 20.0, 30.0, 60.0, 80.0])
    logits, lv = _dev(r.choice(np.concatenate([size, -size]), (33, E)), DT[dtype])
    ids = np.argsort(r.random((33, E)), axis=1)[:, :8]
    ids[3, 5] = -1
    g, gv = _dev(r.standard_normal((33, 8)), torch.float32)
    grad = fp8mm.moe_route_backward(g, logits, torch.from_numpy(ids.astype(np.int32)).to(DEV), "sigmoid", False, 2.5)
    ref = moe.route_backward(gv, lv, ids, "sigmoid", False, 2.5)
    half = BF16 if dtype == "bf16" else 0.0
    _within(_f64(grad), ref, (24 * U + half + 24 * U * half) * np.abs(ref), "grad_logits")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E,k", [(24, 1), (24, 2), (60, 6), (256, 8), (256, 16), (300, 1), (300, 12), (60, 40)])
def test_route_renormalised_gradients_of_a_dominating_slot(E, k, dtype, score):
    """d_j = scale (sum_l s_l (g_j - g_l) + 1e-20 g_j) / S^2, relative to the sum of
    its terms' sizes (0 but for 1e-20 with k = 1), against the formula in long double.
    Scores are off by _score_tol or 8 U each and come in four times (s_l, S twice,
    s_j or the slope, at most 20 U); differences, products and k additions add 3 + k U,
    S's sum 2 k U, divisions and products with scale and slope 6 U."""
    say(f"renormalised route gradients E={E} k={k} {dtype} {score}")
    r = np.random.default_rng(E + k)
    T, scale = 21, 2.5
    grid = np.round(r.standard_normal((T, E)) * 16) / 16 - (6 if score == "sigmoid" else 0)
    ids = np.argsort(r.random((T, E)), axis=1)[:, :k]
    grid[np.arange(T), ids[:, 0]] += np.arange(T) * 0.5          # from level with the others to far above
    logits, lv = _dev(grid, DT[dtype])
    if k > 1:
        ids[4, -1] = -1
    g, gv = _dev(r.standard_normal((T, k)), torch.float32)
    grad = fp8mm.moe_route_backward(g, logits, torch.from_numpy(ids.astype(np.int32)).to(DEV), score, True, scale)
    lv, gv = lv.astype(np.longdouble), gv.astype(np.longdouble) * (ids >= 0)
    ref = moe.route_backward(gv, lv, ids, score, True, scale)
    s = moe.scores(lv, score)
    at = np.where(ids >= 0, ids, 0)
    chosen = np.take_along_axis(s, at, 1) * (ids >= 0)
    S = chosen.sum(1, keepdims=True) + 1e-20
    size = (np.abs(gv[:, :, None] - gv[:, None, :]) * chosen[:, None, :]).sum(2) + 1e-20 * np.abs(gv)
    noise = np.abs(gv).max(1, keepdims=True) * S * 2.0 ** -58    # of the formula's own cancellation in long double
    terms = np.zeros_like(lv)
    np.add.at(terms, (np.arange(T)[:, None], at), (size + noise) * (ids >= 0) * scale / S ** 2)
    if score == "softmax":
        terms += 1e-20 * (chosen * np.abs(gv)).sum(1, keepdims=True) * scale / S ** 2 + noise * scale / S ** 2
    factor = s if score == "softmax" else s * moe.scores(-lv, score)
    half = BF16 if dtype == "bf16" else U
    tol = factor * terms * (4 * _score_tol(lv) + (20 + 20 + 9 + 3 * k) * U) + factor * noise * scale / S ** 2
    _within(_f64(grad), ref.astype(np.float64), (tol + half * np.abs(ref) + half * tol).astype(np.float64),
            "grad_logits")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E,k", [(2, 1), (24, 1), (24, 2), (60, 6), (256, 8), (256, 16), (16, 16), (300, 1), (300, 12),
                                 (60, 40), (40, 40), (1000, 5)])
def test_route_softmax_gradients_of_a_dominating_expert(E, k, dtype):
    """s_j (d_j rest + sum_l s_l (d_j - d_l)) for the chosen, -s_e sum_l s_l d_l for the
    others, relative to the sum of their terms' sizes.  The scores come in twice and
    their sum of the rest once (_score_tol each), differences, products and k
    additions add k + 12 U."""
    say(f"softmax route gradients E={E} k={k} {dtype}")
    r = np.random.default_rng(E + k)
    T, scale = 27, 2.5
    grid = np.round(r.standard_normal((T, E)) * 16) / 16
    ids = np.argsort(r.random((T, E)), axis=1)[:, :k]
    grid[np.arange(T), ids[:, 0]] += np.arange(T)                # from level with the others to far above
    logits, lv = _dev(grid, DT[dtype])
    if k > 1:
        ids[4, -1] = -1
    g, gv = _dev(r.standard_normal((T, k)), torch.float32)
    grad = fp8mm.moe_route_backward(g, logits, torch.from_numpy(ids.astype(np.int32)).to(DEV), "softmax", False, scale)
    used = ids >= 0
    d = scale * gv * used
    s = moe.scores(lv, "softmax")
    chosen = np.take_along_axis(s, np.where(used, ids, 0), 1) * used
    others = s.copy()
    np.put_along_axis(others, np.where(used, ids, ids[:, :1]), 0.0, 1)      # an empty slot: the first's again
    rest = others.sum(1, keepdims=True)
    ref, size = (-s * (chosen * d).sum(1, keepdims=True), s * (chosen * np.abs(d)).sum(1, keepdims=True))
    diff = d[:, :, None] - d[:, None, :]
    for t in range(T):
        at = ids[t][used[t]]
        ref[t, at] = (s[t, at] * (d[t] * rest[t] + (chosen[t] * diff[t]).sum(1))[used[t]])
        size[t, at] = (s[t, at] * (np.abs(d[t]) * rest[t] + (chosen[t] * np.abs(diff[t])).sum(1))[used[t]])
    assert np.abs(ref - moe.route_backward(gv, lv, ids, "softmax", False, scale)).max() <= 1e-14 * scale * 4
    half = BF16 if dtype == "bf16" else U
    tol = size * (3 * _score_tol(lv) + (k + 12) * U)
    _within(_f64(grad), ref, tol + half * np.abs(ref) + half * tol + TINY, "grad_logits")


@pytest.mark.parametrize("T,E,k", [(70001, 8, 2), (70003, 100, 3), (17001, 300, 4)])
def test_route_more_tokens_than_workgroups(T, E, k):
    say(f"route {T}x{E}")
    logits, lv, _, _ = _route_data(T, E, False, "bf16", T)
    ids, w = fp8mm.moe_route_forward(logits, k)
    at = np.argsort(-lv, axis=1, kind="stable")[:, :k]
    assert np.array_equal(ids.cpu().numpy(), at)
    ref = moe.route_weights(lv, at, "softmax", True, 1.0)
    _within(_f64(w), ref, 2 * _score_tol(lv) * ref + TINY, "weights")
    g, gv = _dev(np.random.default_rng(1).standard_normal((T, k)), torch.float32)
    grad = fp8mm.moe_route_backward(g, logits, ids, renormalize=False)
    ref = moe.route_backward(gv, lv, at, "softmax", False, 1.0)
    s = moe.scores(lv, "softmax")
    tol = s * 2 * np.abs(gv).max(1, keepdims=True) * 2 * 4 * (_score_tol(lv) + 64 * U)
    _within(_f64(grad), ref, tol + BF16 * np.abs(ref) + TINY, "grad_logits")


def test_route_many_tokens_and_autograd():
    T, E, k = 9001, 64, 6
    logits, lv, _, _ = _route_data(T, E, False, "fp32", 3)
    ids, w = fp8mm.moe_route_forward(logits, k)
    order = np.argsort(-lv, axis=1, kind="stable")[:, :k]
    assert np.array_equal(ids.cpu().numpy(), order)
    leaf = logits.clone().requires_grad_(True)
    ids2, w2 = fp8mm.moe_route(leaf, k)
    g = torch.randn((T, k), device=DEV)
    w2.backward(g)
    assert torch.equal(ids, ids2) and torch.equal(w, w2.detach())
    assert torch.equal(leaf.grad, fp8mm.moe_route_backward(g, logits, ids))


# ----------------------------------------------------------------- permutation

def _ids(T, k, E, seed, empty=0.1):
    r = np.random.default_rng(seed)
    p = r.random(E) ** 3 + 1e-3
    ids = r.choice(E, size=(T, k), p=p / p.sum()).astype(np.int32)
    gone = r.random((T, k)) < empty
    ids[gone] = r.choice(np.array([-1, E, E + 7, -2 ** 31, 2 ** 31 - 1]), size=gone.sum()).astype(np.int32)
    return ids


@pytest.mark.parametrize("T,k,E", [(0, 2, 5), (1, 1, 1), (7, 3, 4), (16, 6, 64), (65, 2, 64), (511, 8, 8),
                                   (512, 8, 63), (100, 8, 1000), (1000, 4, 256), (2049, 2, 255), (3000, 8, 1024),
                                   (20011, 7, 64),
                                   (40000, 8, 257)])
def test_plan(T, k, E):
    say(f"plan {T}x{k} E={E}")
    ids = _ids(T, k, E, T + E)
    offsets, rows = fp8mm.moe_plan(torch.from_numpy(ids).to(DEV), E)
    roff, rrows = moe.plan(ids.astype(np.int64), E)
    assert np.array_equal(offsets.cpu().numpy(), roff)
    assert np.array_equal(rows.cpu().numpy(), rrows)


@pytest.mark.parametrize("one", [0, 3, -1])
def test_plan_one_expert_takes_all(one):
    ids = torch.full((3000, 3), one, dtype=torch.int32, device=DEV)
    offsets, rows = fp8mm.moe_plan(ids, 5)
    want = torch.arange(9000, dtype=torch.int32, device=DEV).view(3000, 3)
    assert torch.equal(rows, ~want if one < 0 else want)
    assert offsets.tolist() == [9000 if 0 <= one <= e else 0 for e in range(5)]


PERMUTE = [(1, 1, 1, 3), (5, 130, 2, 4), (3, 77, 6, 16), (33, 512, 8, 8), (130, 1030, 3, 64), (9, 5000, 4, 6),
           (700, 256, 1, 5)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,C,k,E", PERMUTE)
def test_dispatch_and_combine(T, C, k, E, dtype):
    say(f"dispatch/combine T={T} C={C} k={k} E={E} {dtype}")
    r = np.random.default_rng(T + C)
    ids = _ids(T, k, E, C)
    _, rv = moe.plan(ids.astype(np.int64), E)
    slots = torch.from_numpy(rv.astype(np.int32)).to(DEV)
    x, xv = _dev(r.standard_normal((T, C)), DT[dtype])
    d = fp8mm.moe_dispatch_forward(x, slots)
    assert np.array_equal(_f64(d), moe.dispatch(xv, rv))
    assert torch.equal(fp8mm.moe_dispatch_forward(_strided(x), slots), d)

    rows, rowsv = _dev(r.standard_normal((T * k, C)), DT[dtype])
    w, wv = _dev(r.random((T, k)) + 0.1, torch.float32)
    if (rv < 0).any():
        rows[torch.from_numpy(~rv[rv < 0]).to(DEV)] = float("nan")     # rows of empty slots are not read
        w[slots < 0] = float("nan")
        rowsv[~rv[rv < 0]] = 0.0
        wv[rv < 0] = 0.0
    half = BF16 if dtype == "bf16" else U
    g, gv = _dev(r.standard_normal((T, C)), DT[dtype])
    for weights, weightsv in ((w, wv), (None, None)):
        y = fp8mm.moe_combine_forward(rows, slots, weights)
        ref = moe.combine(rowsv, rv, weightsv)
        tol = (k + 1) * U * moe.combine(np.abs(rowsv), rv, weightsv)
        _within(_f64(y), ref, tol + half * np.abs(ref) + half * tol + TINY, "combine")
        assert torch.equal(fp8mm.moe_combine_forward(_strided(rows), slots, weights), y)
        gr, gw = fp8mm.moe_combine_backward(g, rows, slots, weights)
        rgr, rgw = moe.combine_backward(gv, rowsv, rv, weightsv)
        _within(_f64(gr), rgr, (half + 2 * U) * np.abs(rgr) + TINY, "grad_rows")
        depth = C / 64 + 6 + 10
        size = moe.combine_backward(np.abs(gv), np.abs(rowsv), rv)[1]
        _within(_f64(gw), rgw, depth * U * size + TINY, "grad_weights")
        grs, gws = fp8mm.moe_combine_backward(_strided(g), _strided(rows, 1, 1), slots, weights)
        assert torch.equal(grs, gr) and torch.equal(gws, gw)
        assert torch.equal(fp8mm.moe_combine_backward(g, None, slots, weights, need_weights=False)[0], gr)
        assert torch.equal(fp8mm.moe_combine_backward(g, rows, slots, weights, need_rows=False)[1], gw)


@pytest.mark.parametrize("T,C,k,E", [(1, 128, 1, 2), (7, 256, 6, 16), (50, 1152, 8, 12), (333, 2048, 2, 64),
                                     (20, 5120, 3, 4)])
def test_fp8_dispatch_is_the_quantization_of_the_rows(T, C, k, E):
    say(f"fp8 dispatch T={T} C={C} k={k} E={E}")
    r = np.random.default_rng(C)
    ids = torch.from_numpy(_ids(T, k, E, C)).to(DEV)
    offsets, slots = fp8mm.moe_plan(ids, E)
    x = torch.from_numpy(r.standard_normal((T, C)) * np.exp(r.standard_normal((T, 1)) * 4)).to(torch.bfloat16).to(DEV)
    x[0, :128] = 0
    q, s = fp8mm.fp8_moe_dispatch(x, slots)
    rq, rs = fp8mm.fp8_quantize_blockwise(fp8mm.moe_dispatch_forward(x, slots), (1, 128))
    assert torch.equal(q, rq) and torch.equal(s, rs)
    wide = torch.zeros((T, C + 16), dtype=torch.bfloat16, device=DEV)
    wide[:, 8:8 + C] = x
    q2, s2 = fp8mm.fp8_moe_dispatch(wide[:, 8:8 + C], slots)
    assert torch.equal(q2, q) and torch.equal(s2, s)


def test_permutation_autograd():
    T, C, k, E = 40, 96, 3, 5
    r = np.random.default_rng(11)
    slots = fp8mm.moe_plan(torch.from_numpy(_ids(T, k, E, 1)).to(DEV), E)[1]
    x = torch.randn((T, C), device=DEV, requires_grad=True)
    w = torch.rand((T, k), device=DEV, requires_grad=True)
    g = torch.from_numpy(r.standard_normal((T, C))).float().to(DEV)
    y = fp8mm.moe_combine(fp8mm.moe_dispatch(x, slots), slots, w)
    y.backward(g)
    used = (slots >= 0).double()
    wsum = (w.detach().double() * used).sum(1, keepdim=True)
    assert torch.allclose(y.detach().double(), wsum * x.detach().double(), rtol=1e-5, atol=1e-6)
    assert torch.allclose(x.grad.double(), wsum * g.double(), rtol=1e-5, atol=1e-6)
    dot = (x.detach().double() * g.double()).sum(1, keepdim=True)
    assert torch.allclose(w.grad.double(), dot * used, rtol=1e-4, atol=1e-4)


def test_differentiable_functions_take_any_strides():
    """Transposed, sliced and broadcast inputs give the bits and gradients of dense ones."""
    T, C, k, E = 33, 256, 4, 16
    torch.manual_seed(4)

    def strided(t):
        return t.t().contiguous().t() if t.dim() == 2 else torch.stack([t, t], 1)[:, 0]

    def check(f, *inputs):
        got = []
        for change in (strided, lambda t: t):
            leaves = [t.detach().clone().requires_grad_(t.is_floating_point()) for t in inputs]
            views = [change(t) for t in leaves]
            out = f(*views)
            out.backward(torch.ones_like(out))
            got.append([out.detach()] + [t.grad for t in leaves if t.is_floating_point()])
        for a, b in zip(*got):
            assert torch.equal(a, b)

    x, v = torch.randn((T, C), device=DEV), torch.randn((C,), device=DEV)
    check(fp8mm.layer_norm, x, v, v + 1)
    balance = strided(torch.randn((E,), device=DEV) * 0.1)
    assert not balance.is_contiguous()
    logits = torch.randn((T, E), device=DEV)
    check(lambda l: fp8mm.moe_route(l, k, "sigmoid", balance)[1], logits)
    slots = fp8mm.moe_plan(fp8mm.moe_route_forward(logits, k)[0], E)[1]
    check(lambda x, s: fp8mm.moe_dispatch(x, s), x, slots)
    check(lambda r, s, w: fp8mm.moe_combine(r, s, w), torch.randn((T * k, C), device=DEV), slots,
          torch.rand((T, k), device=DEV))
    check(fp8mm.fp8_swiglu, x.bfloat16())
    w_in, w_out = (torch.randn(s, device=DEV).bfloat16() for s in ((E, 2 * 128, C), (E, C, 128)))
    check(lambda x, i, w: fp8mm.fp8_moe(x, w_in, w_out, i, w), x.bfloat16(), torch.arange(
        T * k, device=DEV, dtype=torch.int32).view(T, k) % E, torch.rand((T, k), device=DEV))
    g = torch.randn((1, C), device=DEV).expand(T, C)                         # a broadcast gradient
    leaf = x.clone().requires_grad_(True)
    fp8mm.layer_norm(leaf).backward(g)
    again = x.clone().requires_grad_(True)
    fp8mm.layer_norm(again).backward(g.contiguous())
    assert torch.equal(leaf.grad, again.grad)


# ------------------------------------------------------------ gated activation

def _dequantize(q, s):
    """1x128 codes and scales [blocks, R] as float64 values."""
    return e4m3.decode(q.cpu().numpy()).astype(np.float64) * np.repeat(s.double().cpu().numpy().T, 128, axis=1)


def _h_tol(x):
    """|h| times: sigmoid's exponent is off by |g| 2 U, exp2, reciprocal and
    the products by a few U."""
    gate, up = np.split(x, 2, axis=1)
    return np.abs(moe.swiglu(x)) * (np.abs(gate) * 4 + 16) * U + np.abs(gate * up) * FLUSH + TINY


@pytest.mark.parametrize("R,F", [(1, 128), (31, 256), (33, 384), (70, 1408), (5, 5120), (257, 128)])
def test_swiglu(R, F):
    say(f"swiglu {R}x{F}")
    r = np.random.default_rng(R + F)
    x, xv = _dev(r.standard_normal((R, 2 * F)) * np.exp(r.standard_normal((R, 1)) * 1.5), torch.bfloat16)
    x[0, :128] = 0
    xv[0, :128] = 0
    ref, tol = moe.swiglu(xv), _h_tol(xv)
    h, (c, cs) = fp8mm.fp8_swiglu_forward(x)
    _within(_f64(h), ref, tol + BF16 * np.abs(ref) * (1 + BF16), "h")
    rc, rcs = fp8mm.fp8_quantize_blockwise(x, (1, 128))
    assert torch.equal(c, rc) and torch.equal(cs, rcs)
    # codes of the float32 values: scale from their amax, each within half a code step
    (q, s), none = fp8mm.fp8_swiglu_forward(x, "fp8", checkpoint=False)
    assert none is None
    amax = np.abs(ref).reshape(R, F // 128, 128).max(2).T
    want = np.where(amax < 448 * 1e-45, 1.0, amax / 448)
    rel = tol.max() / max(np.abs(ref).max(), 1e-30) + (np.abs(xv).max() * 4 + 24) * U
    _within(_f64(s), want, want * rel, "scale")
    step = np.maximum(np.abs(ref) * 2.0 ** -4, np.repeat(_f64(s).T, 128, axis=1) * 2.0 ** -10)
    _within(_dequantize(q, s), ref, step * (1 + 1e-4) + 2 * tol, "codes")
    for out in ("bf16", "fp8"):
        for ckpt in (False, True):
            a, b = fp8mm.fp8_swiglu_forward(x, out, ckpt)
            for got, keep in zip(a if out == "fp8" else (a,), (q, s) if out == "fp8" else (h,)):
                assert torch.equal(got, keep)
            assert (b is None) == (not ckpt) and (b is None or torch.equal(b[0], c) and torch.equal(b[1], cs))
    wide = torch.zeros((R, 2 * F + 16), dtype=torch.bfloat16, device=DEV)
    wide[:, 8:8 + 2 * F] = x
    assert torch.equal(fp8mm.fp8_swiglu_forward(wide[:, 8:8 + 2 * F])[0], h)

    g, gv = _dev(r.standard_normal((R, F)), torch.bfloat16)
    gx, again = fp8mm.fp8_swiglu_backward(g, c, cs, recompute=True)
    x8 = _dequantize(c, cs)
    ref = moe.swiglu_backward(gv, x8)
    gate, up = np.split(x8, 2, axis=1)
    sig = moe.sigmoid(gate)
    rel = (np.abs(gate) * 4 + 24) * U
    tol = np.concatenate([np.abs(gv * up) * (1 + np.abs(gate)) * (sig * rel + FLUSH),
                          np.abs(gv * gate) * (sig * rel + FLUSH)], 1) + TINY
    _within(_f64(gx), ref, tol + BF16 * np.abs(ref) * (1 + BF16), "grad_x")
    ref = moe.swiglu(x8)
    _within(_f64(again), ref, _h_tol(x8) * 2 + BF16 * np.abs(ref) * (1 + BF16), "h again")
    alone, none = fp8mm.fp8_swiglu_backward(g, c, cs)
    assert none is None and torch.equal(alone, gx)
    leaf = x.clone().requires_grad_(True)
    y = fp8mm.fp8_swiglu(leaf)
    y.backward(g)
    assert torch.equal(y.detach(), h) and torch.equal(leaf.grad, gx)


@pytest.mark.parametrize("R,F", [(10007, 1408), (20003, 1408), (65000, 128)])
def test_large_swiglu(R, F):
    """Streaming stores (above 32 MiB) and loads (64 MiB) against calls on a few rows
    each, which have neither: every output has the same bits."""
    say(f"swiglu {R}x{F}")
    torch.manual_seed(R)
    x = (torch.randn((R, 2 * F), device=DEV) * torch.exp(torch.randn((R, 1), device=DEV))).bfloat16()
    g = torch.randn((R, F), device=DEV).bfloat16()
    parts = 16

    def flat(out):
        return [t for t in (out if isinstance(out, (tuple, list)) else (out,)) for t in
                (flat(t) if isinstance(t, (tuple, list)) else [t]) if t is not None]

    def check(whole, pieces):
        whole, pieces = flat(whole), [flat(p) for p in pieces]
        for i, t in enumerate(whole):
            rows = 1 if t.dtype == torch.float32 else 0            # scales are [blocks, R]
            assert torch.equal(t, torch.cat([p[i] for p in pieces], rows))

    c, cs = fp8mm.fp8_quantize_blockwise(x, (1, 128))
    for out in ("bf16", "fp8"):
        for ckpt in (False, True):
            check(fp8mm.fp8_swiglu_forward(x, out, ckpt),
                  [fp8mm.fp8_swiglu_forward(p, out, ckpt) for p in x.chunk(parts)])
    lib, st = fp8mm._lib.load(), torch.cuda.current_stream().cuda_stream
    h, (q, s) = fp8mm.fp8_swiglu_forward(x)[0], fp8mm.fp8_swiglu_forward(x, "fp8")[0]
    for ckpt in (False, True):                                     # both forms of h, from the C call
        h2, q2, s2 = torch.empty_like(h), torch.empty_like(q), torch.empty_like(s)
        c2, cs2 = torch.empty_like(c), torch.empty_like(cs)
        assert lib.fp8_swiglu(x.data_ptr(), R, F, 2 * F, h2.data_ptr(), F, q2.data_ptr(), F, s2.data_ptr(),
                              c2.data_ptr() if ckpt else None, 2 * F, cs2.data_ptr(), st) == 0
        assert torch.equal(q2, q) and torch.equal(s2, s)
        # bf16 of the float32 values that the codes come from, of the fast sigmoid alone: an ulp apart
        assert bool(((h2.float() - h.float()).abs() <= 2 ** -7 * h.float().abs()).all())
        assert not ckpt or torch.equal(c2, c) and torch.equal(cs2, cs)
    for again in (False, True):
        check(fp8mm.fp8_swiglu_backward(g, c, cs, recompute=again),
              [fp8mm.fp8_swiglu_backward(a, b, d.contiguous(), recompute=again)
               for a, b, d in zip(g.chunk(parts), c.chunk(parts), cs.chunk(parts, 1))])


def test_swiglu_empty_and_extreme_values():
    x = torch.empty((0, 512), dtype=torch.bfloat16, device=DEV)
    h, (c, s) = fp8mm.fp8_swiglu_forward(x)
    assert h.shape == (0, 256) and c.shape == (0, 512)
    assert fp8mm.fp8_swiglu_backward(h, c, s)[0].shape == (0, 512)
    # gates far out on both sides saturate without NaN; a NaN stays in its group
    x = torch.ones((2, 512), dtype=torch.bfloat16, device=DEV)
    x[0, 0], x[0, 1], x[0, 130] = 3e4, -3e4, float("nan")
    h, _ = fp8mm.fp8_swiglu_forward(x)
    assert float(h[0, 0]) == float(x[0, 0]) and float(h[0, 1]) == 0.0
    assert torch.isnan(h).sum() == 1
    (q, s), (c, cs) = fp8mm.fp8_swiglu_forward(x, "fp8")
    assert torch.isnan(s).sum() == 1 and bool(torch.isnan(s[1, 0]))
    assert torch.isnan(cs).sum() == 1 and bool(torch.isnan(cs[1, 0]))


# ---------------------------------------------------------------- expert layer

def _sqnr(got, ref):
    return 10 * np.log10((ref ** 2).sum() / ((got - ref) ** 2).sum())


@pytest.mark.parametrize("T,C,F,E,k", [(96, 256, 128, 4, 2), (257, 384, 256, 8, 3)])
def test_expert_layer(T, C, F, E, k):
    """Forward and gradients against the float64 layer.  Each E4M3 operand adds
    an error of at most 2^-4 relative and about 2^-5.3 (-32 dB) in the mean;
    the output sees five of them (two products, the activation's slope), the
    gradients up to eight: 20 and 17 dB leave a factor of two."""
    say(f"expert layer T={T} C={C} F={F} E={E} k={k}")
    r = np.random.default_rng(T)
    x, xv = _dev(r.standard_normal((T, C)), torch.bfloat16)
    w_in, iv = _dev(r.standard_normal((E, 2 * F, C)) / np.sqrt(C), torch.bfloat16)
    w_out, ov = _dev(r.standard_normal((E, C, F)) / np.sqrt(F), torch.bfloat16)
    logits, _ = _dev(r.standard_normal((T, E)), torch.float32)
    logits[5] = float("-inf")                  # a padding token
    ids, w = fp8mm.moe_route_forward(logits, k)
    g, gv = _dev(r.standard_normal((T, C)), torch.bfloat16)
    leaves = [t.requires_grad_(True) for t in (x, w_in, w_out, w)]
    y = fp8mm.fp8_moe(x, w_in, w_out, ids, w)
    y.backward(g)
    wv, at = w.detach().double().cpu().numpy(), ids.cpu().numpy()
    ry, gx, gi, go, gw = (np.zeros(v) for v in ((T, C), (T, C), iv.shape, ov.shape, (T, k)))
    for t in range(T):
        for j in range(k):
            e = at[t, j]
            if e < 0:
                continue
            u = (iv[e] @ xv[t])[None]
            h = moe.swiglu(u)[0]
            out = ov[e] @ h
            ry[t] += wv[t, j] * out
            gw[t, j] = gv[t] @ out
            gout = wv[t, j] * gv[t]
            go[e] += np.outer(gout, h)
            gu = moe.swiglu_backward((gout @ ov[e])[None], u)[0]
            gi[e] += np.outer(gu, xv[t])
            gx[t] += gu @ iv[e]
    assert not _f64(y.detach())[5].any() and not _f64(x.grad)[5].any()
    for got, ref, bar, what in ((y.detach(), ry, 20, "y"), (x.grad, gx, 17, "grad_x"), (w_in.grad, gi, 17, "grad_w_in"),
                                (w_out.grad, go, 17, "grad_w_out"), (w.grad, gw, 17, "grad_weights")):
        db = _sqnr(_f64(got), ref)
        say(f"  {what}: {db:.1f} dB")
        assert db >= bar, (what, db)
    # without gradients, the public calls in order: the same bits
    with torch.no_grad():
        offsets, slots = fp8mm.moe_plan(ids, E)
        q, s = fp8mm.fp8_moe_dispatch(x, slots)
        qi, si = fp8mm.fp8_quantize_blockwise(w_in.view(E * 2 * F, C), (128, 128))
        qo, so = fp8mm.fp8_quantize_blockwise(w_out.view(E * C, F), (128, 128))
        u = fp8mm.fp8_scaled_grouped_mm_v2(q, qi.view(E, 2 * F, C), offsets, s, "1x128", si, "128x128")
        (hq, hs), _ = fp8mm.fp8_swiglu_forward(u, "fp8", checkpoint=False)
        rows = fp8mm.fp8_scaled_grouped_mm_v2(hq, qo.view(E, C, F), offsets, hs, "1x128", so, "128x128")
        assert torch.equal(fp8mm.moe_combine_forward(rows, slots, w), y)
        assert torch.equal(fp8mm.fp8_moe(x, w_in, w_out, ids, w), y)
    assert len(leaves) == 4


def test_expert_layer_graph_follows_new_routing():
    """One captured block (norm, routing, plan, dispatch, experts, combine)
    replayed on new tokens; each replay against the eager calls."""
    T, C, F, E, k = 600, 256, 128, 16, 4
    torch.manual_seed(3)
    w_in = (torch.randn((E, 2 * F, C), device=DEV) / 16).bfloat16()
    w_out = (torch.randn((E, C, F), device=DEV) / 11).bfloat16()
    router = (torch.randn((C, E), device=DEV) / 16).bfloat16()
    gamma = torch.ones(C, dtype=torch.bfloat16, device=DEV)

    def block(x):
        n = fp8mm.layer_norm_forward(x, gamma)[0]
        ids, w = fp8mm.moe_route_forward(n @ router, k, "sigmoid", groups=4, group_topk=2, group_score="top2")
        return ids, w, fp8mm.fp8_moe(n, w_in, w_out, ids, w)

    with torch.no_grad():
        static = torch.randn((T, C), device=DEV).bfloat16()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            on_side = block(static)
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(on_side, block(static)):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
        say("capturing the block")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = block(static)
        for rep in range(3):
            x = torch.randn((T, C), device=DEV).bfloat16()
            static.copy_(x)
            graph.replay()
            torch.cuda.synchronize()
            eager = block(x)
            torch.cuda.synchronize()
            for a, b in zip(captured, eager):
                assert torch.equal(a, b)
            assert float(eager[2].float().abs().max()) > 0


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_no_checkpoint_where_no_gradient_can_follow(mode, monkeypatch):
    """Parameters need gradients under no_grad too; the activation's codes are not
    made there, and the results have the same bits."""
    asked = []
    forward = fp8mm.moe.fp8_swiglu_forward

    def spy(x, out="bf16", checkpoint=True):
        asked.append(bool(checkpoint))
        return forward(x, out, checkpoint)

    monkeypatch.setattr(fp8mm.moe, "fp8_swiglu_forward", spy)
    E, C, F, k, T = 4, 256, 128, 2, 40
    torch.manual_seed(2)
    w_in = torch.nn.Parameter(torch.randn((E, 2 * F, C), device=DEV).bfloat16() / 16)
    w_out = torch.nn.Parameter(torch.randn((E, C, F), device=DEV).bfloat16() / 11)
    x = torch.randn((T, C), device=DEV).bfloat16()
    u = torch.nn.Parameter(torch.randn((T, C), device=DEV).bfloat16())
    ids, w = fp8mm.moe_route_forward(torch.randn((T, E), device=DEV), k)
    y, h = fp8mm.fp8_moe(x, w_in, w_out, ids, w), fp8mm.fp8_swiglu(u)
    assert asked == [True, True] and y.requires_grad and h.requires_grad
    with mode():
        assert torch.equal(fp8mm.fp8_moe(x, w_in, w_out, ids, w), y)
        assert torch.equal(fp8mm.fp8_swiglu(u), h)
    assert torch.equal(fp8mm.fp8_moe(x, w_in.detach(), w_out.detach(), ids, w), y)
    assert asked[2:] == [False] * 3
    y.float().sum().backward()
    assert bool(w_in.grad.any()) and bool(w_out.grad.any())


def test_expert_layer_reads_no_row_without_an_expert(monkeypatch):
    """The grouped products leave the rows of empty slots as they find them; whatever
    is there, the layer's results and gradients have the same bits."""
    E, C, F, k, T = 6, 256, 128, 3, 70
    product = fp8mm.moe.fp8_scaled_grouped_mm_v2
    r = np.random.default_rng(8)
    ids = torch.from_numpy(_ids(T, k, E, 5, empty=0.4)).to(DEV)
    assert int(((ids < 0) | (ids >= E)).sum()) > 40
    torch.manual_seed(8)
    inputs = (torch.randn((T, C), device=DEV).bfloat16(), torch.randn((E, 2 * F, C), device=DEV).bfloat16() / 16,
              torch.randn((E, C, F), device=DEV).bfloat16() / 11, torch.rand((T, k), device=DEV))
    g = torch.from_numpy(r.standard_normal((T, C))).to(torch.bfloat16).to(DEV)
    results = []
    for left in (0.0, float("nan"), float("inf"), -3e38):
        def filled(*args, out, **kw):
            return product(*args, out=out.fill_(left), **kw)

        monkeypatch.setattr(fp8mm.moe, "fp8_scaled_grouped_mm_v2", filled)
        for needs in ((True,) * 4, (True, False, False, False), (False, True, False, True), (False, False, True, False)):
            leaves = [t.clone().requires_grad_(n) for t, n in zip(inputs, needs)]
            y = fp8mm.fp8_moe(leaves[0], leaves[1], leaves[2], ids, leaves[3])
            y.backward(g)
            results.append([y.detach()] + [t.grad for t in leaves])
    n = len(results) // 4
    for i, got in enumerate(results):
        for a, b in zip(got, results[i % n]):
            assert (a is None) == (b is None) and (a is None or torch.equal(a, b) and bool(torch.isfinite(a).all()))


def test_rows_are_kept_for_the_gradient_of_the_weights_alone():
    E, C, F, k, T = 4, 256, 128, 2, 40
    torch.manual_seed(6)
    w_in = torch.randn((E, 2 * F, C), device=DEV).bfloat16() / 16
    w_out = torch.randn((E, C, F), device=DEV).bfloat16() / 11
    ids, w = fp8mm.moe_route_forward(torch.randn((T, E), device=DEV), k)
    slots = fp8mm.moe_plan(ids, E)[1]
    x, rows = torch.randn((T, C), device=DEV).bfloat16(), torch.randn((T * k, C), device=DEV).bfloat16()
    grads = []
    for needs in (True, False):
        weights = w.clone().requires_grad_(needs)
        a, b = (t.clone().requires_grad_(True) for t in (x, rows))
        y, z = fp8mm.fp8_moe(a, w_in, w_out, ids, weights), fp8mm.moe_combine(b, slots, weights)
        for out in (y, z):
            kept = [t for t in out.grad_fn.saved_tensors if t is not None and t.shape == rows.shape
                    and t.dtype == rows.dtype]
            assert len(kept) == needs
            out.backward(torch.ones_like(out))
        grads.append((a.grad, b.grad))
        assert (weights.grad is not None) == needs
    for with_weights, without in zip(*grads):
        assert torch.equal(with_weights, without)


def test_no_tokens_and_tokens_without_experts():
    E, C, F, k = 4, 256, 128, 2
    w_in = torch.randn((E, 2 * F, C), device=DEV).bfloat16().requires_grad_(True)
    w_out = torch.randn((E, C, F), device=DEV).bfloat16().requires_grad_(True)
    for T in (0, 1, 5):
        logits = torch.full((T, E), float("-inf"), device=DEV)
        ids, w = fp8mm.moe_route_forward(logits, k)
        assert ids.shape == (T, k) and bool((ids == -1).all()) and not bool(w.any())
        assert fp8mm.moe_route_backward(w, logits, ids).shape == (T, E)
        offsets, slots = fp8mm.moe_plan(ids, E)
        assert offsets.tolist() == [0] * E and bool((slots < 0).all())
        x = torch.randn((T, C), device=DEV).bfloat16().requires_grad_(True)
        rows = fp8mm.moe_dispatch_forward(x.detach(), slots)
        q, s = fp8mm.fp8_moe_dispatch(x.detach(), slots)
        assert rows.shape == (T * k, C) and not bool(rows.any()) and not bool(q.any()) and bool((s == 1).all())
        gr, gw = fp8mm.moe_combine_backward(x.detach(), rows, slots, w)
        assert not bool(gr.any()) and not bool(gw.any())
        w_in.grad = w_out.grad = None
        y = fp8mm.fp8_moe(x, w_in, w_out, ids, w)
        y.backward(torch.ones_like(y))
        assert y.shape == (T, C) and not bool(y.any())
        for g in (x.grad, w_in.grad, w_out.grad):
            assert not bool(g.any())


def test_offsets_past_32_bits():
    """More than 2^31 elements (4 GiB of bf16) in every large operand."""
    T, k, C, E = 280000, 4, 2048, 16
    assert T * k * C > 2 ** 31
    say("dispatch and combine of 1.1 million rows")
    ids = (torch.arange(T * k, device=DEV, dtype=torch.int64) * 7919 % E).to(torch.int32).view(T, k)
    slots = fp8mm.moe_plan(ids, E)[1]
    x = torch.randn((T, C), device=DEV, dtype=torch.bfloat16)
    rows = fp8mm.moe_dispatch_forward(x, slots)
    assert torch.equal(fp8mm.moe_combine_forward(rows, slots), x * 4)       # four equal bf16 values: exact
    last = slots[-1].tolist()
    gr, gw = fp8mm.moe_combine_backward(x, rows, slots)
    assert torch.equal(gr[last], x[-1:].expand(k, C))
    assert torch.equal(gw[:, :1].expand(T, k), gw)
    del gr, rows
    q, s = fp8mm.fp8_moe_dispatch(x, slots)
    q1, s1 = fp8mm.fp8_quantize_blockwise(x[-3:].contiguous(), (1, 128))
    assert torch.equal(q[slots[-3:].flatten().long()], q1.repeat_interleave(k, 0))
    assert torch.equal(s[:, slots[-3:].flatten().long()], s1.repeat_interleave(k, 1))
    del q, s
    say("layer norm and gated activation of 2.2e9 elements")
    big = x.repeat(4, 1)
    y, mean, rstd = fp8mm.layer_norm_forward(big)
    y1, m1, r1 = fp8mm.layer_norm_forward(x[-5:].contiguous())
    assert torch.equal(y[-5:], y1) and torch.equal(mean[-5:], m1) and torch.equal(rstd[-5:], r1)
    dx = fp8mm.layer_norm_backward(y, big, None, mean, rstd, need_params=False)[0]
    assert torch.equal(dx[-5:], fp8mm.layer_norm_backward(y1, x[-5:].contiguous(), None, m1, r1, need_params=False)[0])
    del y, dx
    (hq, hs), (c, cs) = fp8mm.fp8_swiglu_forward(big, "fp8")
    (hq1, hs1), (c1, cs1) = fp8mm.fp8_swiglu_forward(x[-5:].contiguous(), "fp8")
    assert torch.equal(hq[-5:], hq1) and torch.equal(hs[:, -5:], hs1)
    assert torch.equal(c[-5:], c1) and torch.equal(cs[:, -5:], cs1)
    grad = torch.ones((T * 4, C // 2), device=DEV, dtype=torch.bfloat16)
    gx, h = fp8mm.fp8_swiglu_backward(grad, c, cs, recompute=True)
    gx1, h1 = fp8mm.fp8_swiglu_backward(grad[:5].contiguous(), c1, cs1.contiguous(), recompute=True)
    assert torch.equal(gx[-5:], gx1) and torch.equal(h[-5:], h1)


# Expert-order rows on both sides of 32 MiB (streaming stores) and 64 MiB (streaming
# loads): rows of 16 lanes a slot and of a wave, whole and ending within a chunk.
LARGE = [(C, k, mib) for C, k in ((339, 4), (220, 4), (256, 8), (2375, 4), (2048, 6), (1030, 3)) for mib in (30, 34, 62, 70)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("C,k,mib", LARGE)
def test_large_dispatch_and_combine(C, k, mib, dtype):
    T = mib * 2 ** 20 // (C * k * (2 if dtype == "bf16" else 4)) + 1
    E = 64
    say(f"dispatch/combine T={T} C={C} k={k} {dtype}: {mib} MiB")
    torch.manual_seed(C + mib)
    slots = fp8mm.moe_plan(torch.from_numpy(_ids(T, k, E, C)).to(DEV), E)[1]
    used = slots >= 0
    at = torch.where(used, slots, ~slots).long()
    x = torch.randn((T, C), device=DEV).to(DT[dtype])
    d = fp8mm.moe_dispatch_forward(x, slots)
    want = torch.empty_like(d)
    want[at.flatten()] = torch.where(used[..., None], x[:, None, :], torch.zeros_like(x[:, None, :])).flatten(0, 1)
    assert torch.equal(d, want)
    assert torch.equal(fp8mm.moe_dispatch_forward(_strided(x), slots), d)
    del d, want
    rows = torch.randn((T * k, C), device=DEV).to(DT[dtype])
    w = torch.rand((T, k), device=DEV) + 0.1
    rows[at[~used]] = float("nan")                    # rows and weights of empty slots are not read
    w[~used] = float("nan")
    wv = torch.where(used, w, torch.zeros_like(w)).double()
    rv = torch.where(used[..., None], rows[at], torch.zeros_like(rows[at])).double()        # [T, k, C]
    half = BF16 if dtype == "bf16" else U

    def within(got, ref, tol, what):
        off = (got.double() - ref).abs()
        assert bool((off <= tol).all()), f"{what}: {int((~(off <= tol)).sum())} of {off.numel()} outside"

    y = fp8mm.moe_combine_forward(rows, slots, w)
    ref, tol = (wv[..., None] * rv).sum(1), (k + 1) * U * (wv[..., None] * rv.abs()).sum(1)
    within(y, ref, tol + half * ref.abs() + half * tol + TINY, "combine")
    assert torch.equal(fp8mm.moe_combine_forward(_strided(rows), slots, w), y)
    g = torch.randn((T, C), device=DEV).to(DT[dtype])
    gr, gw = fp8mm.moe_combine_backward(g, rows, slots, w)
    gv = g.double()[:, None, :]
    ref = wv[..., None] * gv
    within(gr[at], ref, (half + 2 * U) * ref.abs() + TINY, "grad_rows")
    depth = C / 16 + 6 + 14                           # of a slot's 16 or 64 lanes
    within(gw, (gv * rv).sum(2), depth * U * (gv * rv).abs().sum(2) + TINY, "grad_weights")
    grs, gws = fp8mm.moe_combine_backward(_strided(g), _strided(rows, 1, 1), slots, w)
    assert torch.equal(grs, gr) and torch.equal(gws, gw)
    assert torch.equal(fp8mm.moe_combine_backward(g, None, slots, w, need_weights=False)[0], gr)
    assert torch.equal(fp8mm.moe_combine_backward(g, rows, slots, w, need_rows=False)[1], gw)


@pytest.mark.parametrize("T,C,k", [(6000, 1152, 6), (35000, 128, 8), (5000, 2048, 3)])
def test_large_fp8_dispatch(T, C, k):
    say(f"fp8 dispatch T={T} C={C} k={k}")
    slots = fp8mm.moe_plan(torch.from_numpy(_ids(T, k, 64, C)).to(DEV), 64)[1]
    x = (torch.randn((T, C), device=DEV) * torch.exp(torch.randn((T, 1), device=DEV) * 4)).bfloat16()
    q, s = fp8mm.fp8_moe_dispatch(x, slots)
    rq, rs = fp8mm.fp8_quantize_blockwise(fp8mm.moe_dispatch_forward(x, slots), (1, 128))
    assert torch.equal(q, rq) and torch.equal(s, rs)


def test_gradients_of_weights_past_32_bits():
    T, k, C, E = 270001, 4, 2048, 16
    assert T * k * C > 2 ** 31
    say("gradient of the weights of 1.1 million rows")
    ids = (torch.arange(T * k, device=DEV, dtype=torch.int64) * 7919 % E).to(torch.int32).view(T, k)
    slots = fp8mm.moe_plan(ids, E)[1]
    x = torch.randn((T, C), device=DEV, dtype=torch.bfloat16)
    gw = fp8mm.moe_combine_backward(x, fp8mm.moe_dispatch_forward(x, slots), slots, need_rows=False)[1]
    dot = torch.cat([(part.double() ** 2).sum(1, keepdim=True) for part in x.split(30000)])
    assert bool(((gw - dot).abs() <= (C / 64 + 6 + 10) * U * dot).all())


def test_permutation_of_more_slots_than_waves():
    """More than 2^25 slots: dispatch and combine take a wave a token, combine's
    backward of short rows a quarter of one a slot."""
    T, k, C, E = 600011, 64, 128, 16
    assert T * k > 2 ** 25
    say("permutation of 38 million slots")
    ids = (torch.arange(T * k, device=DEV, dtype=torch.int64) * 7919 % E).to(torch.int32).view(T, k)
    slots = fp8mm.moe_plan(ids, E)[1]
    x = torch.randn((T, C), device=DEV, dtype=torch.bfloat16)
    rows = fp8mm.moe_dispatch_forward(x, slots)
    some = torch.arange(0, T, 9973, device=DEV)
    at = slots[some].flatten().long()
    assert torch.equal(rows[at], x[some].repeat_interleave(k, 0))
    assert torch.equal(fp8mm.moe_combine_forward(rows, slots), x * k)       # 64 equal bf16 values: exact
    gr, gw = fp8mm.moe_combine_backward(x, rows, slots)
    assert torch.equal(gr, rows)
    dot = (x.double() ** 2).sum(1, keepdim=True)
    assert bool(((gw - dot).abs() <= (128 / 16 + 4 + 10) * U * dot).all())
    del gr, rows
    q, s = fp8mm.fp8_moe_dispatch(x, slots)
    q1, s1 = fp8mm.fp8_quantize_blockwise(x[some].contiguous(), (1, 128))
    assert torch.equal(q[at], q1.repeat_interleave(k, 0)) and torch.equal(s[:, at], s1.repeat_interleave(k, 1))


def test_strided_outputs_leave_the_padding_alone():
    """The C calls take a row stride for each output: columns past the row stay."""
    lib = fp8mm._lib.load()
    st = torch.cuda.current_stream().cuda_stream
    T, k, C = 9, 2, 200
    x = torch.randn((T, C), device=DEV).bfloat16()
    slots = fp8mm.moe_plan((torch.arange(T * k, device=DEV, dtype=torch.int32) % 4).view(T, k), 4)[1]

    def padded(rows, cols, pad=24, dtype=torch.bfloat16):
        return torch.full((rows, cols + pad), 7, device=DEV, dtype=dtype)

    def untouched(t, cols, ref):
        torch.cuda.synchronize()
        assert bool((t[:, cols:] == 7).all()) and torch.equal(t[:, :cols], ref)

    y = padded(T, C)
    assert lib.fp8mm_layer_norm(x.data_ptr(), 0, T, C, C, None, None, 0, 1e-5, y.data_ptr(), C + 24, None, None,
                                st) == 0
    yr, mean, rstd = fp8mm.layer_norm_forward(x)
    untouched(y, C, yr)
    dx = padded(T, C)
    assert lib.fp8mm_layer_norm_backward(yr.data_ptr(), C, x.data_ptr(), C, 0, T, C, None, 0, mean.data_ptr(),
                                         rstd.data_ptr(), dx.data_ptr(), C + 24, None, None, None, 0, st) == 0
    untouched(dx, C, fp8mm.layer_norm_backward(yr, x, None, mean, rstd)[0])
    rows = padded(T * k, C)
    assert lib.fp8mm_moe_dispatch(x.data_ptr(), 0, T, C, C, slots.data_ptr(), k, rows.data_ptr(), C + 24, st) == 0
    r = fp8mm.moe_dispatch_forward(x, slots)
    untouched(rows, C, r)
    out = padded(T, C)
    assert lib.fp8mm_moe_combine(r.data_ptr(), 0, T, C, C, slots.data_ptr(), None, k, out.data_ptr(), C + 24, st) == 0
    untouched(out, C, fp8mm.moe_combine_forward(r, slots))
    gr = padded(T * k, C)
    assert lib.fp8mm_moe_combine_backward(x.data_ptr(), C, None, 0, 0, T, C, slots.data_ptr(), None, k, gr.data_ptr(),
                                          C + 24, None, st) == 0
    untouched(gr, C, r)
    logits = torch.randn((T, 50), device=DEV)
    ids, w = fp8mm.moe_route_forward(logits, k)
    gl = padded(T, 50, dtype=torch.float32)
    assert lib.fp8mm_moe_route_backward(w.data_ptr(), logits.data_ptr(), 1, T, 50, 50, ids.data_ptr(), k, 0, 1, 1.0,
                                        gl.data_ptr(), 74, st) == 0
    untouched(gl, 50, fp8mm.moe_route_backward(w, logits, ids))
    u = torch.randn((T, 512), device=DEV).bfloat16()
    h, q, c = padded(T, 256), padded(T, 256, 32, torch.uint8), padded(T, 512, 32, torch.uint8)
    s, cs = torch.empty((2, T), device=DEV), torch.empty((4, T), device=DEV)
    assert lib.fp8_swiglu(u.data_ptr(), T, 256, 512, h.data_ptr(), 280, q.data_ptr(), 288, s.data_ptr(), c.data_ptr(),
                          544, cs.data_ptr(), st) == 0
    (qr, sr), (cr, csr) = fp8mm.fp8_swiglu_forward(u, "fp8")
    untouched(h, 256, fp8mm.fp8_swiglu_forward(u)[0])
    untouched(q, 256, qr)
    untouched(c, 512, cr)
    assert torch.equal(s, sr) and torch.equal(cs, csr)
    gx, h2 = padded(T, 512), padded(T, 256)
    g = torch.randn((T, 256), device=DEV).bfloat16()
    assert lib.fp8_swiglu_backward(g.data_ptr(), 256, c.data_ptr(), 544, cs.data_ptr(), T, 256, gx.data_ptr(), 536,
                                   h2.data_ptr(), 280, st) == 0
    gxr, hr = fp8mm.fp8_swiglu_backward(g, cr, csr, recompute=True)
    untouched(gx, 512, gxr)
    untouched(h2, 256, hr)
    xd = torch.randn((T, 256), device=DEV).bfloat16()
    qd, sd = padded(T * k, 256, 32, torch.uint8), torch.empty((2, T * k), device=DEV)
    assert lib.fp8_moe_dispatch(xd.data_ptr(), T, 256, 256, slots.data_ptr(), k, qd.data_ptr(), 288, sd.data_ptr(),
                                st) == 0
    qdr, sdr = fp8mm.fp8_moe_dispatch(xd, slots)
    untouched(qd, 256, qdr)
    assert torch.equal(sd, sdr)


# -------------------------------------------------------------------- refusals

def test_refusals():
    bf = dict(dtype=torch.bfloat16, device=DEV)
    x = torch.zeros((4, 256), **bf)
    slots = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    wide = torch.zeros((4, 512), **bf)
    for call in (
        lambda: fp8mm.layer_norm_forward(x.half()),
        lambda: fp8mm.layer_norm_forward(x.cpu()),
        lambda: fp8mm.layer_norm_forward(x.t()),
        lambda: fp8mm.layer_norm_forward(x, torch.zeros(255, **bf)),
        lambda: fp8mm.layer_norm_forward(x, torch.zeros(256, **bf), torch.zeros(256, device=DEV)),
        lambda: fp8mm.layer_norm_forward(x, eps=-1.0),
        lambda: fp8mm.layer_norm_forward(torch.zeros((4, 0), **bf)),
        lambda: fp8mm.layer_norm_backward(x, wide, None, torch.zeros(4, device=DEV), torch.zeros(4, device=DEV)),
        lambda: fp8mm.layer_norm_backward(x, x, None, torch.zeros(3, device=DEV), torch.zeros(4, device=DEV)),
        lambda: fp8mm.moe_route_forward(x, 0),
        lambda: fp8mm.moe_route_forward(x, 257),
        lambda: fp8mm.moe_route_forward(x, 2, groups=3),
        lambda: fp8mm.moe_route_forward(x, 2, groups=4, group_topk=5),
        lambda: fp8mm.moe_route_forward(x, 2, score="tanh"),
        lambda: fp8mm.moe_route_forward(x, 2, bias=torch.zeros(256, **bf)),
        lambda: fp8mm.moe_route_forward(x, 2, scale=float("inf")),
        lambda: fp8mm.moe_route_backward(torch.zeros((4, 3), device=DEV), x, slots),
        lambda: fp8mm.moe_plan(slots.long(), 4),
        lambda: fp8mm.moe_plan(slots, 0),
        lambda: fp8mm.moe_plan(slots.t(), 4),
        lambda: fp8mm.moe_dispatch_forward(x, slots[:3]),
        lambda: fp8mm.moe_dispatch_forward(x, slots.float()),
        lambda: fp8mm.fp8_moe_dispatch(torch.zeros((4, 130), **bf), slots),
        lambda: fp8mm.fp8_moe_dispatch(x.float(), slots),
        lambda: fp8mm.moe_combine_forward(x, slots),
        lambda: fp8mm.moe_combine_forward(torch.zeros((8, 256), **bf), slots, torch.zeros((2, 4), device=DEV)),
        lambda: fp8mm.moe_combine_backward(x, None, slots),
        lambda: fp8mm.fp8_swiglu_forward(torch.zeros((4, 384), **bf)),
        lambda: fp8mm.fp8_swiglu_forward(x, "fp16"),
        lambda: fp8mm.fp8_swiglu_forward(x.float()),
        lambda: fp8mm.fp8_swiglu_backward(x, torch.zeros((4, 256), dtype=torch.uint8, device=DEV),
                                          torch.zeros((4, 4), device=DEV)),
        lambda: fp8mm.fp8_moe(x, torch.zeros((2, 256, 256), **bf), torch.zeros((3, 256, 128), **bf), slots,
                              torch.zeros((4, 2), device=DEV)),
    ):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(NotImplementedError):
        fp8mm.moe_route_forward(torch.zeros((1, 1025), device=DEV), 2)
    with pytest.raises(NotImplementedError):
        fp8mm.moe_route_forward(torch.zeros((1, 128), device=DEV), 65)
    with pytest.raises(NotImplementedError):
        fp8mm.moe_plan(slots, 1025)
