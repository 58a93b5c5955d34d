"""The operators around a block's dense products and its router against their
float64 definitions.

Tolerances are worst-case bounds of float32 evaluation, U = 2^-24: a sum of n terms
whose longest chain of additions is D is off by at most D U sum|terms|; bf16 results
add half a bf16 step, 2^-8 |y|, E4M3 codes half a step of theirs, 2^-4 of the value
or 2^-10 of the scale, whichever is more.  Whole numbers are exact."""

import numpy as np
import pytest
import torch

import precision_matmul_amd as fp8mm
from oracle import block, e4m3
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8         # half a step of bf16, relative
TINY = 1e-37             # results that are subnormal in float32 may be flushed
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
NAN, INF = float("nan"), float("inf")


def _dev(a, dtype):
    """float64 numpy -> (device tensor of dtype, the float64 values it holds)."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)
    return t, t.double().cpu().numpy()


def _strided(t, left=3, right=5):
    """The same values as columns [left, left + C) of a wider matrix: rows start at
    any element and the row stride is not the width."""
    wide = torch.full((t.shape[0], t.shape[1] + left + right), NAN, dtype=t.dtype, device=t.device)
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


def _rounded(ref, tol, half):
    """Tolerance after one rounding of a value that was off by tol."""
    return tol + half * np.abs(ref) + half * tol + TINY


# -------------------------------------------------------------------- RMS norm

def _depth(C):
    """Longest chain of additions of a row sum: a lane's own elements (at most 32 in
    registers, C / 256 in the long form), then the wave and the waves."""
    return max(32, C / 256) + 6 + 8


def _add(x, res, dtype):
    """h as the kernel rounds it: one float32 addition, one rounding to the type."""
    if res is None:
        return x, _f64(x)
    h = (x.cpu().float() + res.cpu().float()).to(DT[dtype])
    return h, h.double().numpy()


def _norm_inputs(R, C, dtype, params, residual, seed):
    r = np.random.default_rng(seed)
    x, _ = _dev(r.standard_normal((R, C), dtype=np.float32) * 1.5, DT[dtype])
    res = _dev(r.standard_normal((R, C), dtype=np.float32) * 2, DT[dtype])[0] if residual else None
    w, wv = _dev(1 + 0.3 * r.standard_normal(C), DT[params]) if params else (None, None)
    return r, x, res, w, wv


def _check_forward(x, res, w, wv, dtype, eps=1e-6):
    y, h, rstd = fp8mm.rms_norm_forward(x, w, res, eps)
    want, hv = _add(x, res, dtype)
    assert torch.equal(h.cpu(), want.cpu())
    ref, rref = block.rms_norm(hv, wv, eps)
    e = (_depth(hv.shape[1]) / 2 + 8) * U          # half of the sum's, division, root, reciprocal
    _within(_f64(rstd), rref, e * rref, "rstd")
    tol = (e + 4 * U) * np.abs(ref)
    _within(_f64(y), ref, _rounded(ref, tol, BF16 if dtype == "bf16" else U), "y")
    return y, h, rstd, hv, ref, e


def _check_codes(x, res, w, wv, recipe, ref, e, want_y, eps=1e-6):
    q, s, y, h, rstd = fp8mm.fp8_rms_norm_forward(x, w, res, eps, recipe=recipe, y=want_y)
    R, C = ref.shape
    groups = np.abs(ref).reshape(R, -1, 128 if recipe == "1x128" else C).max(2)
    sref = groups / 448 + (1e-12 if recipe == "rowwise" else 0)
    sref[sref == 0] = 1.0
    got = _f64(s).T if recipe == "1x128" else _f64(s)
    rel = e + 8 * U                                 # of y, its amax and the quotient by 448
    _within(got, sref, rel * sref, "scale")
    per = np.repeat(got, C // got.shape[1], 1)
    value = e4m3.decode(q.cpu().numpy()).astype(np.float64) * per
    _within(value, ref, np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * per) + 4 * rel * np.abs(ref), "codes")
    return q, s, y, h, rstd


def _check_backward(dy, dyv, h, hv, w, wv, rstd, gh, ghv, dtype, params):
    R, C = hv.shape
    half, D = BF16 if dtype == "bf16" else U, _depth(C)
    r64 = _f64(rstd)
    dx, dw = fp8mm.rms_norm_backward(dy, h, w, rstd, gh)
    rdx, rdw = block.rms_norm_backward(dyv, hv, wv, r64, ghv)
    a = np.abs(dyv) * (1 if wv is None else np.abs(wv))
    hr = np.abs(hv) * r64[:, None]
    tol = r64[:, None] * (6 * U * a + (D + 12) * U * hr * (a * hr).mean(1, keepdims=True))
    tol = tol + 2 * U * (np.abs(rdx) + (0 if ghv is None else np.abs(ghv)))
    _within(_f64(dx), rdx, _rounded(rdx, tol, half), "dx")
    tol = (R + 28) * U * (np.abs(dyv) * hr).sum(0)  # rows of one workgroup, its waves, the partial rows
    _within(_f64(dw), rdw, _rounded(rdw, tol, BF16 if params == "bf16" else U), "dweight")
    return dx, dw


NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (4, 513), (9, 1024), (2, 1413), (7, 2048), (6, 2049), (5, 4104), (3, 5120),
               (2, 6200), (3, 8192), (2, 8193), (2, 20001)]


@pytest.mark.parametrize("params", ["bf16", "fp32", None])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,C", NORM_SHAPES)
def test_rms_norm(R, C, dtype, params):
    say(f"rms norm {R}x{C} {dtype} params {params}")
    for residual in (False, True):
        r, x, res, w, wv = _norm_inputs(R, C, dtype, params, residual, R * 100003 + C)
        y, h, rstd, hv, _, _ = _check_forward(x, res, w, wv, dtype)
        dy, dyv = _dev(r.standard_normal((R, C)), DT[dtype])
        gh, ghv = _dev(r.standard_normal((R, C)), DT[dtype]) if residual else (None, None)
        dx, dw = _check_backward(dy, dyv, h, hv, w, wv, rstd, gh, ghv, dtype, params or "fp32")
        # rows at any stride and start: the same bits
        sres, sgh = (None, None) if res is None else (_strided(res, 1, 4), _strided(gh, 2, 1))
        ys, hs, _ = fp8mm.rms_norm_forward(_strided(x), w, sres)
        assert torch.equal(ys, y) and torch.equal(hs, h)
        for got, want in zip(fp8mm.rms_norm_backward(_strided(dy, 1, 2), _strided(h), w, rstd, sgh), (dx, dw)):
            assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,C", [(512, 100), (513, 100), (600, 513), (530, 1024), (521, 2047), (519, 2049), (520, 3560),
                                 (515, 4104), (514, 6200), (516, 8190), (2100, 1001), (4500, 3557), (700, 8200),
                                 (520, 16384), (300, 12289), (260, 16385)])
def test_rms_norm_of_many_rows(R, C, dtype):
    """Both sides of the step from one launch of the backward to partial sums, more
    rows than workgroups, every width."""
    say(f"rms norm {R}x{C} {dtype}")
    r, x, res, w, wv = _norm_inputs(R, C, dtype, "fp32", True, R + C)
    y, h, rstd, hv, _, _ = _check_forward(x, res, w, wv, dtype)
    dy, dyv = _dev(r.standard_normal((R, C), dtype=np.float32), DT[dtype])
    gh, ghv = _dev(r.standard_normal((R, C), dtype=np.float32), DT[dtype])
    dx, dw = _check_backward(dy, dyv, h, hv, w, wv, rstd, gh, ghv, dtype, "fp32")
    for got, want in zip(fp8mm.rms_norm_backward(_strided(dy, 1, 2), _strided(h), w, rstd, _strided(gh)), (dx, dw)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("R,C,dtype", [(9000, 2048, "bf16"), (8200, 2056, "bf16"), (4000, 5120, "bf16"),
                                       (2400, 7177, "bf16"), (3000, 4097, "fp32"), (1500, 6148, "fp32"),
                                       (1100, 8192, "fp32"), (2100, 8201, "bf16")])
def test_rms_norm_past_the_caches(R, C, dtype):
    """More than 32 MiB of rows: streaming accesses."""
    test_rms_norm_of_many_rows(R, C, dtype)


# Rows of more than 32 MiB, of each number of waves and chunks a lane.
STREAMED = [(33000, 512, "bf16"), (16400, 1024, "bf16"), (15300, 1100, "bf16"), (11000, 1536, "bf16"), (4200, 4096, "bf16"),
            (2100, 8192, "bf16"), (1100, 16384, "bf16"), (33000, 256, "fp32"), (16500, 511, "fp32"), (11100, 768, "fp32"),
            (8300, 1024, "fp32")]


@pytest.mark.parametrize("R,C,dtype", STREAMED)
def test_rms_norm_past_the_caches_is_that_of_fewer_rows(R, C, dtype):
    """Rows are independent: streaming accesses give the bits that parts of the rows, which
    stay below 32 MiB, give by themselves."""
    say(f"rms norm streamed {R}x{C} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(R)
    x, res, dy, gh = (torch.randn((R, C), generator=g, device=DEV).to(DT[dtype]) for _ in range(4))
    w = torch.randn(C, generator=g, device=DEV)
    parts = [slice(0, R // 2), slice(R // 2, R)]
    y, h, rstd = fp8mm.rms_norm_forward(x, w, res)
    dx, dw = fp8mm.rms_norm_backward(dy, h, w, rstd, gh)
    plain = fp8mm.rms_norm_forward(x, w)[0]
    for p in parts:
        for got, want in zip((y, h, rstd), fp8mm.rms_norm_forward(x[p], w, res[p])):
            assert torch.equal(got[p], want)
        assert torch.equal(fp8mm.rms_norm_forward(x[p], w)[0], plain[p])
        assert torch.equal(fp8mm.rms_norm_backward(dy[p], h[p], w, rstd[p], gh[p], need_weight=False)[0], dx[p])
    hr = h.double() * rstd.double()[:, None]
    ref, size = (dy.double() * hr).sum(0).cpu().numpy(), (dy.double() * hr).abs().sum(0).cpu().numpy()
    _within(_f64(dw), ref, _rounded(ref, (R + 28) * U * size, U), "dweight")
    for recipe, group in (("1x128", 128), ("rowwise", 16)) if dtype == "bf16" else ():
        if C % group == 0:
            q, s, y2, h2, _ = fp8mm.fp8_rms_norm_forward(x, w, res, recipe=recipe, y=True)
            assert torch.equal(y2, y) and torch.equal(h2, h)
            for p in parts:
                want = fp8mm.fp8_rms_norm_forward(x[p], w, res[p], recipe=recipe)
                assert torch.equal(q[p], want[0])
                assert torch.equal(s[:, p] if recipe == "1x128" else s[p], want[1])


@pytest.mark.parametrize("recipe", ["1x128", "rowwise"])
@pytest.mark.parametrize("R,C", [(1, 128), (3, 256), (130, 512), (5, 640), (33, 1024), (9, 1152), (40, 2048), (7, 2176),
                                 (11, 5120), (6, 6272), (5, 8192), (4, 8320), (3, 16384), (9000, 2048), (3400, 5120)])
def test_rms_norm_codes(R, C, recipe):
    say(f"rms norm codes {R}x{C} {recipe}")
    for residual, params, want_y in ((True, "bf16", False), (False, "fp32", True)):
        _, x, res, w, wv = _norm_inputs(R, C, "bf16", params, residual, R + C)
        x[R // 2] *= 100
        y, h, rstd, _, ref, e = _check_forward(x, res, w, wv, "bf16")
        q, s, y2, h2, rstd2 = _check_codes(x, res, w, wv, recipe, ref, e, want_y)
        assert torch.equal(h2, h) and torch.equal(rstd2, rstd) and (torch.equal(y2, y) if want_y else y2 is None)
        sres = None if res is None else _strided(res, 1, 4)
        again = fp8mm.fp8_rms_norm_forward(_strided(x), w, sres, recipe=recipe)
        assert torch.equal(again[0], q) and torch.equal(again[1], s)


def test_rms_norm_codes_of_any_sixteen_columns():
    for C in (16, 48, 1040, 2064, 5136, 8208):
        _, x, res, w, wv = _norm_inputs(5, C, "bf16", "bf16", True, C)
        ref, e = _check_forward(x, res, w, wv, "bf16")[4:]
        _check_codes(x, res, w, wv, "rowwise", ref, e, False)


def test_rms_norm_codes_feed_the_product():
    """Codes straight into the scaled product, against the product of the float64 rows:
    each factor is off by half an E4M3 step at most, 2^-4 of its size."""
    _, x, res, w, wv = _norm_inputs(256, 512, "bf16", "bf16", True, 5)
    ref = _check_forward(x, res, w, wv, "bf16")[4]
    weight, weight_v = _dev(np.random.default_rng(6).standard_normal((128, 512)) * 0.05, torch.bfloat16)
    exact = ref @ weight_v.T
    bound = (2 * 2.0 ** -4 + 2.0 ** -8) * (np.abs(ref) @ np.abs(weight_v).T) + 2.0 ** -8 * np.abs(exact)
    q, s = fp8mm.fp8_rms_norm_forward(x, w, res)[:2]
    qw, sw = fp8mm.fp8_quantize_blockwise(weight, (128, 128))
    # small values of a group keep 2^-10 of its scale at least: amax / 448 / 1024 a value
    tail = np.abs(ref).reshape(256, 4, 128).max(2).sum(1)[:, None] * 128 / 448 / 1024 * np.abs(weight_v).max()
    tail_w = np.abs(weight_v).max() / 448 / 1024 * np.abs(ref).sum(1)[:, None]
    _within(_f64(fp8mm.fp8_scaled_mm(q, qw, s, "1x128", sw, "128x128")), exact, bound + tail + tail_w, "1x128 product")
    q, s = fp8mm.fp8_rms_norm_forward(x, w, res, recipe="rowwise")[:2]
    qw, sw = fp8mm.fp8_quantize_rowwise(weight)
    tail = np.abs(ref).max(1)[:, None] * 512 / 448 / 1024 * np.abs(weight_v).max()
    _within(_f64(fp8mm.fp8_scaled_mm(q, qw, s, "rowwise", sw, "rowwise")), exact, bound + tail + tail_w, "rowwise product")


def test_rms_norm_special_rows():
    """Zeros, one large value, NaN and infinity: each stays in its row."""
    for dtype in ("bf16", "fp32"):
        for C in (256, 3200, 9088):
            x = torch.randn((6, C), device=DEV).to(DT[dtype])
            x[1] = 0
            x[2] = 0
            x[2, C // 2] = 1e15
            x[3, 5] = NAN
            x[4, C - 1] = INF
            y, _, rstd = fp8mm.rms_norm_forward(x, None, None, 1e-30)
            assert torch.equal(y[[0, 5]], fp8mm.rms_norm_forward(x[[0, 5]].contiguous(), None, None, 1e-30)[0])
            assert (y[1] == 0).all() and abs(float(y[2, C // 2]) / C ** 0.5 - 1) < 0.01 and int((y[2] != 0).sum()) == 1
            assert y[3].isnan().all() and y[4, C - 1].isnan() and (y[4, :C - 1] == 0).all()
            dx, dw = fp8mm.rms_norm_backward(torch.ones_like(x[:3]), x[:3].contiguous(), None, rstd[:3].contiguous())
            assert not dw.isnan().any() and not dx[[0, 2]].isnan().any()
    x = torch.zeros((2, 256), device=DEV).bfloat16()
    q, s = fp8mm.fp8_rms_norm_forward(x)[:2]
    assert (q == 0).all() and (s == 1).all()
    q, s = fp8mm.fp8_rms_norm_forward(x, recipe="rowwise")[:2]
    assert (q == 0).all() and (s == np.float32(1e-12)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norms_under_a_large_eps(dtype):
    """Beside it the row's own size hardly counts."""
    _, x, _, w, wv = _norm_inputs(5, 384, dtype, "fp32", False, 3)
    for eps in (2e30, 3e38):
        _check_forward(x, None, w, wv, dtype, eps)
        y, mean, rstd = fp8mm.layer_norm_forward(x, w, None, eps)
        xv = _f64(x)
        centred = xv - xv.mean(1, keepdims=True)
        ref = centred / np.sqrt((centred ** 2).mean(1, keepdims=True) + eps) * wv
        # the mean's sum, up to 64 values a lane and 6 steps of the wave; difference, root, reciprocal, products
        tol = (80 * U * np.abs(xv).mean(1, keepdims=True) + 8 * U * np.abs(centred)) / np.sqrt(eps) * np.abs(wv)
        _within(_f64(y), ref, _rounded(ref, tol, BF16 if dtype == "bf16" else U), "layer norm")


def test_rms_norm_without_rows():
    x = torch.empty((0, 256), device=DEV, dtype=torch.bfloat16)
    w = torch.ones(256, device=DEV)
    y, h, rstd = fp8mm.rms_norm_forward(x, w, x)
    assert y.shape == h.shape == (0, 256) and rstd.shape == (0,)
    q, s = fp8mm.fp8_rms_norm_forward(x, w)[:2]
    assert q.shape == (0, 256) and s.shape == (2, 0)
    dx, dw = fp8mm.rms_norm_backward(x, x, w, rstd)
    assert dx.shape == (0, 256) and (dw == 0).all()
    dx, dw = fp8mm.rms_norm_backward(x, x, w, rstd, need_dx=False)
    assert dx is None and (dw == 0).all()


def test_rms_norm_writes_nothing_else():
    """Strided outputs through the C ABI: the columns around them stay, and so does h
    where there is no residual; dx may be the gradient that it adds."""
    lib, st = fp8mm._lib.load(), torch.cuda.current_stream().cuda_stream
    R, C = 37, 384
    x, res = (torch.randn((R, C), device=DEV).bfloat16() for _ in range(2))
    want = fp8mm.fp8_rms_norm_forward(x, None, res, y=True)
    wide = [torch.full((R + 2, C + 32), 7.0, device=DEV).bfloat16() for _ in range(2)]
    q = torch.full((R + 2, C + 32), 9, device=DEV, dtype=torch.uint8)
    s, rstd = torch.empty((C // 128, R), device=DEV), torch.empty(R, device=DEV)
    inner = [t[1:R + 1, 16:16 + C] for t in (*wide, q)]
    args = (x.data_ptr(), C, res.data_ptr(), C, 0, R, C, None, 1, 1e-6, inner[0].data_ptr(), C + 32, inner[1].data_ptr(),
            C + 32, inner[2].data_ptr(), C + 32, s.data_ptr(), 2, rstd.data_ptr(), st)
    assert lib.fp8mm_rms_norm(*args) == 0
    for got, ref in zip((*inner, s, rstd), (want[3], want[2], want[0], want[1], want[4])):
        assert torch.equal(got, ref)
    for t, v in zip((*wide, q), (7, 7, 9)):
        mask = torch.ones_like(t, dtype=torch.bool)
        mask[1:R + 1, 16:16 + C] = False
        assert (t[mask] == v).all()
    gh = torch.randn((R, C), device=DEV).bfloat16()
    dx = fp8mm.rms_norm_backward(x, want[3], None, rstd, gh, need_weight=False)[0]
    assert lib.fp8mm_rms_norm_backward(x.data_ptr(), C, want[3].data_ptr(), C, gh.data_ptr(), C, 0, R, C, None, 1,
                                       rstd.data_ptr(), gh.data_ptr(), C, None, None, 0, st) == 0
    assert torch.equal(gh, dx)


@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_autograd(residual):
    r = np.random.default_rng(7)
    leaves = [torch.randn((2, 5, 320), device=DEV, requires_grad=True) for _ in range(1 + residual)]
    w = torch.randn(320, device=DEV, requires_grad=True)
    dy, gh = (torch.randn((2, 5, 320), device=DEV) for _ in range(2))
    out = fp8mm.rms_norm(leaves[0], w, leaves[1] if residual else None)
    y, h = out if residual else (out, None)
    loss = (y * dy).sum() + ((h * gh).sum() if residual else 0)
    loss.backward()
    hv = sum(_f64(t.detach()) for t in leaves).reshape(10, 320)
    hv = hv.astype(np.float32).astype(np.float64)
    rstd = block.rms_norm(hv, None)[1]
    dx, dw = block.rms_norm_backward(_f64(dy).reshape(10, 320), hv, _f64(w.detach()), rstd,
                                     _f64(gh).reshape(10, 320) if residual else None)
    for t in leaves:        # 100 U: the depth of a row sum and the rounding of rstd, times terms of size 1 to 20
        _within(_f64(t.grad).reshape(10, 320), dx, 100 * U * 20, "dx")
    _within(_f64(w.grad), dw, 100 * U * 20, "dweight")
    if residual:            # h alone used, y alone used
        for part in range(2):
            a, b = (t.detach().clone().requires_grad_() for t in leaves)
            out = fp8mm.rms_norm(a, w.detach().requires_grad_(), b)
            (out[part] * dy).sum().backward()
            assert torch.equal(a.grad, b.grad)
            if part == 1:
                assert torch.equal(a.grad, dy)
    with pytest.raises(RuntimeError):       # second derivatives are refused
        x = leaves[0].detach().requires_grad_()
        g, = torch.autograd.grad(fp8mm.rms_norm(x, w).sum(), x, create_graph=True)
        g.sum().backward()


# ---------------------------------------------------------------- balance loss

def _router(T, E, k, dtype, seed, spread=1.5, masked=0.1, empty=0.1):
    """Logits and chosen ids, some rows padding, some slots empty."""
    r = np.random.default_rng(seed)
    a = r.standard_normal((T, E)) * spread + r.standard_normal(E)
    pad = r.random(T) < masked
    a[pad] = -np.inf
    x, xv = _dev(a, DT[dtype])
    ids = np.argsort(-xv + r.random((T, E)) * 1e-9, 1)[:, :k].astype(np.int32)
    ids[r.random((T, k)) < empty] = -1
    ids[r.random((T, k)) < empty / 2] = E + 5
    return r, x, xv, torch.from_numpy(ids).to(DEV), ids


def _p_error(xv, p, used, score, E):
    """Relative error of each probability: the argument's rounding |x - m| U, the
    exponential, quotient and sum (a lane's 16 values, then the lanes)."""
    top = np.where(used, np.max(np.where(np.isneginf(xv), -1e9, xv), 1), 0.0)[:, None]
    m = np.minimum(top, 0) if score == "sigmoid" else top
    away = np.where(p > 0, np.abs(np.where(np.isneginf(xv), 0.0, xv) - m), 0.0)
    return (away + (p * away).sum(1, keepdims=True) + 16 + 6 + 16) * U


def _check_balance(x, xv, ids, idv, score, coeff, ends, endv, g=1.7, strided=True):
    T, E = xv.shape
    loss, counts, tokens = fp8mm.moe_balance_loss_forward(x, ids, score, coeff, ends)
    rloss, rcounts, rtokens = block.balance_loss(xv, idv, score, coeff, endv)
    assert np.array_equal(counts.cpu().numpy(), rcounts) and np.array_equal(tokens.cpu().numpy(), rtokens)
    p, used = block.probabilities(xv, score)
    e = _p_error(xv, p, used, score, E)
    tol, alive = 0.0, max(1, (rtokens > 0).sum())
    for (begin, end), c, n in zip(block.runs(endv, T), rcounts, rtokens):
        if n:
            # a token a turn of 4 to 16 slots, the slots, the runs of 256 chunks, the experts
            chain = 16 + T / 1024 + 16 + 260 + 64 + 16
            tol += (E * c / (idv.shape[1] * n) * ((p * (e + chain * U))[begin:end].sum(0) / n)).sum() + 8 * U * abs(rloss)
    tol = abs(coeff) * tol / alive + 8 * U * abs(rloss)
    _within(_f64(loss), np.array(rloss), tol + TINY, "loss")
    grad_loss = torch.tensor(g, device=DEV)
    gv = float(grad_loss)
    k = idv.shape[1]
    grad = fp8mm.moe_balance_loss_backward(grad_loss, x, counts, tokens, k, score, coeff, ends)
    ref = block.balance_loss_backward(gv, xv, rcounts, rtokens, k, score, coeff, endv)
    tol = np.zeros_like(ref)
    for (begin, end), c, n in zip(block.runs(endv, T), rcounts, rtokens):
        if n:
            q, eq = p[begin:end], e[begin:end]
            D = np.abs(c[None, :] - c[q.argmax(1)][:, None]).astype(float)
            mean = (q * D).sum(1, keepdims=True)
            scale = abs(gv * coeff) * E / (alive * k * float(n) ** 2)
            tol[begin:end] = scale * q * (eq * (D + mean) + (q * D * eq).sum(1, keepdims=True) + 40 * U * (D + mean))
    if score == "sigmoid":
        x0 = np.where(np.isneginf(xv), 0.0, xv)
        slope = np.exp(np.minimum(-x0, 0.0)) / (1.0 + np.exp(-np.abs(x0)))
        tol = tol * slope + (np.abs(x0) + 12) * U * np.abs(ref)
    _within(_f64(grad), ref, _rounded(ref, tol, BF16 if x.dtype == torch.bfloat16 else U), "grad")
    if strided:
        again = fp8mm.moe_balance_loss_forward(_strided(x), ids, score, coeff, ends)
        assert all(torch.equal(a, b) for a, b in zip(again, (loss, counts, tokens)))
        assert torch.equal(fp8mm.moe_balance_loss_backward(grad_loss, _strided(x), counts, tokens, k, score, coeff, ends),
                           grad)
    return loss, counts, tokens, grad


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 3), (5, 63, 6), (64, 64, 6), (65, 65, 1), (300, 128, 8),
                                   (129, 129, 2), (1000, 256, 8), (77, 257, 40), (140, 512, 17), (90, 1023, 64),
                                   (33, 1024, 5), (20000, 24, 2), (256, 1022, 3), (257, 1021, 9), (700, 600, 3),
                                   (16500, 260, 4)])
def test_balance_loss(T, E, k, score, dtype):
    say(f"balance loss {T}x{E} k {k} {score} {dtype}")
    _, x, xv, ids, idv = _router(T, E, min(k, E), dtype, T + E)
    _check_balance(x, xv, ids, idv, score, 0.25, None, None)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,endv", [(10, 16, [3, 3, 7]), (200, 64, [0, 0, 63, 64, 65, 128, 200]), (130, 70, [130]),
                                      (130, 70, [1]), (64, 300, [64, 64]), (9, 16, [0]), (500, 33, list(range(0, 500))),
                                      (3000, 128, [64, 700, 701, 2111, 2990]), (40, 600, [5, 39]),
                                      (1024, 40, [1024, 1024]), (1025, 40, [1, 1025]),
                                      (800, 40, list(range(0, 800, 10))), (900, 300, sorted(i * 613 % 901 for i in range(70))),
                                      (2100, 301, list(range(0, 2080, 32))), (1500, 1023, [700, 702, 1400]),
                                      (1200, 18, sorted(i * 7919 % 1201 for i in range(200)))])
def test_balance_loss_of_sequences(T, E, endv, score):
    """Ends inside, on and around chunks; empty sequences; rows behind the last."""
    say(f"balance loss {T}x{E} ends {endv[:8]} {score}")
    _, x, xv, ids, idv = _router(T, E, 4, "fp32", T + E)
    ends = torch.tensor(endv, dtype=torch.int32, device=DEV)
    _, counts, tokens, grad = _check_balance(x, xv, ids, idv, score, 1.0, ends, endv)
    assert (grad[endv[-1]:] == 0).all()
    # more than one sequence gives what each by itself gives
    if len(endv) < 10:
        for s, (a, b) in enumerate(block.runs(endv, T)):
            if b > a:
                one = fp8mm.moe_balance_loss_forward(x[a:b].contiguous(), ids[a:b].contiguous(), score)
                assert torch.equal(one[1][0], counts[s]) and torch.equal(one[2][0], tokens[s])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,E,endv", [(20000, 24, [79, 80, 5000, 5040, 12345, 19999]),
                                      (17000, 100, [1, 66, 67, 9000, 16990]),
                                      (17000, 200, sorted(i * 4241 % 17001 for i in range(40))),
                                      (16600, 300, [64, 65, 8111, 16600]), (16500, 601, [16499]),
                                      (18000, 40, sorted(i * 7919 % 18001 for i in range(300)))])
def test_balance_loss_of_sequences_in_long_batches(T, E, endv, dtype):
    """More than 64 tokens a chunk: ends inside its turns, several in one of them."""
    say(f"balance loss {T}x{E} ends {endv[:8]} {dtype}")
    _, x, xv, ids, idv = _router(T, E, 3, dtype, T + E)
    ends = torch.tensor(endv, dtype=torch.int32, device=DEV)
    grad = _check_balance(x, xv, ids, idv, "sigmoid" if E % 8 else "softmax", 1.0, ends, endv, strided=E < 200)[3]
    assert (grad[endv[-1]:] == 0).all()


def test_balance_loss_with_nothing_in_it():
    for T, endv in ((0, None), (0, [0]), (5, [0, 0]), (3, None)):
        x = torch.full((T, 16), -INF, device=DEV)
        ids = torch.zeros((T, 2), dtype=torch.int32, device=DEV)
        ends = None if endv is None else torch.tensor(endv, dtype=torch.int32, device=DEV)
        loss, counts, tokens = fp8mm.moe_balance_loss_forward(x, ids, ends=ends)
        assert float(loss) == 0 and (counts == 0).all() and (tokens == 0).all()
        grad = fp8mm.moe_balance_loss_backward(torch.ones((), device=DEV), x, counts, tokens, 2, ends=ends)
        assert (grad == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_of_saturated_tokens(score):
    """One expert has nearly all of a token's probability: its gradient is built from
    differences, not from the rounding of two equal numbers.  And logits whose sigmoids
    float32 does not hold."""
    a = np.full((40, 8), -9.0)
    a[np.arange(40), np.arange(40) % 5] = 9.0
    a[20:30] -= 300.0
    a[30:] = np.arange(8) * 0.25 - 200.0
    x, xv = _dev(a, torch.float32)
    idv = np.argsort(-a, 1, kind="stable")[:, :2].astype(np.int32)
    ids = torch.from_numpy(idv).to(DEV)
    _, counts, tokens, grad = _check_balance(x, xv, ids, idv, score, 1.0, None, None)
    ref = block.balance_loss_backward(float(torch.tensor(1.7)), xv, counts.cpu().numpy(), tokens.cpu().numpy(), 2, score)
    big = np.abs(ref) > 1e-30
    # the exponentials' arguments, up to 18, and about 60 roundings
    assert (np.abs(_f64(grad) / np.where(big, ref, 1) - 1)[big] < (2 * 18 + 60) * U).all()


def test_balance_loss_shows_nan():
    for score in ("softmax", "sigmoid"):
        x = torch.randn((70, 32), device=DEV)
        x[66, 3] = NAN
        ids = torch.zeros((70, 2), dtype=torch.int32, device=DEV)
        loss, counts, tokens = fp8mm.moe_balance_loss_forward(x, ids, score)
        assert loss.isnan() and int(tokens) == 70 and int(counts[0, 0]) == 140
        grad = fp8mm.moe_balance_loss_backward(torch.ones((), device=DEV), x, counts, tokens, 2, score)
        assert grad[66].isnan().all() and not grad[:66].isnan().any() and not grad[67:].isnan().any()
        x[66] = NAN                       # a row of NaN alone is no padding
        assert fp8mm.moe_balance_loss_forward(x, ids, score)[0].isnan()
        # rows behind the last sequence do not count
        loss, _, tokens = fp8mm.moe_balance_loss_forward(x, ids, score, ends=torch.tensor([50], dtype=torch.int32,
                                                                                           device=DEV))
        assert not loss.isnan() and int(tokens) == 50


def test_balance_ends_out_of_range_stay_in_range():
    """Ends that are not ascending or past the rows give wrong sums, and nothing else."""
    x, ids = torch.randn((100, 40), device=DEV), torch.zeros((100, 3), dtype=torch.int32, device=DEV)
    for endv in ([-5, 20], [90, 10, 300], [2 ** 31 - 1, -2 ** 31], [300, 300]):
        ends = torch.tensor(endv, dtype=torch.int32, device=DEV)
        loss, counts, tokens = fp8mm.moe_balance_loss_forward(x, ids, ends=ends)
        fp8mm.moe_balance_loss_backward(torch.ones((), device=DEV), x, counts, tokens, 3, ends=ends)
    torch.cuda.synchronize()


def test_balance_loss_autograd():
    _, x, xv, ids, idv = _router(90, 48, 4, "fp32", 11)
    logits = x.clone().requires_grad_()
    ends = torch.tensor([30, 80], dtype=torch.int32, device=DEV)
    loss, counts = fp8mm.moe_balance_loss(logits, ids, "sigmoid", 0.5, ends)
    (3 * loss).backward()
    _, rc, rt = block.balance_loss(xv, idv, "sigmoid", 0.5, [30, 80])
    want = fp8mm.moe_balance_loss_backward(torch.tensor(3.0, device=DEV), x, counts, torch.from_numpy(rt.astype(np.int32)).to(DEV),
                                           4, "sigmoid", 0.5, ends)
    assert torch.equal(logits.grad, want) and np.array_equal(counts.cpu().numpy(), rc) and not counts.requires_grad


# -------------------------------------------------------------------- adapters

def _adapters(T, K, N, n, r, seed, segments=None, without=0.15):
    rng = np.random.default_rng(seed)
    x, xv = _dev(rng.standard_normal((T, K)), torch.bfloat16)
    base, basev = _dev(rng.standard_normal((T, N)), torch.bfloat16)
    down, downv = _dev(rng.standard_normal((n, r, K)) * K ** -0.5, torch.bfloat16)
    up, upv = _dev(rng.standard_normal((n, r, N)) * 0.5, torch.bfloat16)
    scales, sv = _dev(rng.random(n) + 0.5, torch.float32)
    if segments is None:
        idv = rng.integers(0, n, T)
    else:
        cuts = np.sort(rng.integers(0, T + 1, segments - 1)) if segments > 1 else np.array([], int)
        idv = rng.integers(0, n, segments)[np.searchsorted(cuts, np.arange(T), side="right")]
    idv = np.where(rng.random(T) < without, rng.choice([-1, n, n + 7, -2 ** 31], T), idv).astype(np.int32)
    return rng, (x, down, up, torch.from_numpy(idv).to(DEV), scales, base), (xv, downv, upv, idv, sv, basev)


def _gather(idv, panels, s):
    """Per token: |scale| and the adapter's panel by token chunks would be large, so
    bounds are taken adapter by adapter."""
    for a in range(panels.shape[0]):
        at = np.flatnonzero(idv == a)
        if len(at):
            yield a, at, (1.0 if s is None else s[a])


# of v kept as two bf16 numbers: half a step of half a step
V_SPLIT = 2.0 ** -16


def _check_lora(dev, val, scaled=True, based=True):
    x, down, up, ids, scales, base = dev
    xv, downv, upv, idv, sv, basev = val
    scales, sv = (scales, sv) if scaled else (None, None)
    base, basev = (base, basev) if based else (None, None)
    K, N, r = downv.shape[2], upv.shape[2], downv.shape[1]
    out, v = fp8mm.lora_forward(x, down, up, ids, scales, base)
    ref, vref = block.lora(xv, downv, upv, idv, sv, basev)
    tol = np.zeros_like(ref)
    got_v = _f64(v).sum(0)[:, :r]
    for a, at, s in _gather(idv, downv, sv):
        ev = (K + 24) * U * (np.abs(xv[at]) @ np.abs(downv[a]).T)
        _within(got_v[at], vref[at], ev, "v")
        both = ev + (V_SPLIT + (2 * r + 24) * U) * np.abs(vref[at])
        tol[at] = abs(s) * both @ np.abs(upv[a]) + 2 * U * np.abs(ref[at])
    _within(_f64(out), ref, _rounded(ref, tol, BF16), "out")
    none = (idv < 0) | (idv >= downv.shape[0])
    assert torch.equal(out.cpu()[none], torch.zeros_like(out.cpu()[none]) if base is None else base.cpu()[none])
    return out, v


def _check_lora_backward(dev, val, v, dy, dyv, scaled=True, grad="bf16"):
    x, down, up, ids, scales, _ = dev
    xv, downv, upv, idv, sv, _ = val
    scales, sv = (scales, sv) if scaled else (None, None)
    K, N, r, T = downv.shape[2], upv.shape[2], downv.shape[1], xv.shape[0]
    got = fp8mm.lora_backward(dy, x, v, down, up, ids, scales, out_dtype=DT[grad])
    ref = block.lora_backward(dyv, xv, downv, upv, idv, sv)
    tdx, tdd, tdu = (np.zeros_like(t) for t in ref)
    for a, at, s in _gather(idv, downv, sv):
        dv, vv = dyv[at] @ upv[a].T, xv[at] @ downv[a].T
        edv = abs(s) * ((N + 24) * U * (np.abs(dyv[at]) @ np.abs(upv[a]).T) + (V_SPLIT + 24 * U) * np.abs(dv))
        ev = abs(s) * ((K + 24) * U * (np.abs(xv[at]) @ np.abs(downv[a]).T) + (V_SPLIT + 24 * U) * np.abs(vv))
        adv, av = abs(s) * np.abs(dv), abs(s) * np.abs(vv)
        tdx[at] = (edv + 2 * r * U * adv) @ np.abs(downv[a])
        chain = (2 * len(at) + 40) * U
        tdd[a] = (edv + chain * adv).T @ np.abs(xv[at])
        tdu[a] = (ev + chain * av).T @ np.abs(dyv[at])
    half = BF16 if grad == "bf16" else U
    for g, q, t, h, name in zip(got, ref, (tdx, tdd, tdu), (BF16, half, half), ("dx", "ddown", "dup")):
        _within(_f64(g), q, _rounded(q, t, h), name)
    return got


LORA_SHAPES = [(1, 1, 1, 1, 1), (1, 64, 128, 3, 8), (3, 7, 130, 2, 5), (16, 513, 64, 70, 16), (63, 128, 1000, 3, 17),
               (64, 640, 513, 1, 32), (65, 130, 520, 4, 33), (200, 1000, 129, 70, 40), (256, 512, 512, 9, 64),
               (257, 260, 1030, 3, 65), (300, 2048, 1408, 5, 16), (130, 384, 640, 2, 130), (70, 256, 300, 2, 256),
               (1000, 333, 257, 6, 16), (5, 5120, 1024, 2, 24), (70, 3, 7, 2, 20), (90, 7, 64, 9, 64), (600, 8, 5, 3, 8),
               (500, 264, 136, 40, 16), (300, 130, 70, 400, 9), (513, 72, 1090, 2, 128)]


@pytest.mark.parametrize("T,K,N,n,r", LORA_SHAPES)
def test_lora(T, K, N, n, r):
    """Any order of adapters: decoding batches, and the worst order for longer ones."""
    say(f"lora {T}x{K}x{N} adapters {n} rank {r}")
    rng, dev, val = _adapters(T, K, N, n, r, T + K + r)
    out, v = _check_lora(dev, val)
    x, down, up, ids, scales, base = dev
    # strides and starts of any kind, and in place: the same bits
    wide = _strided(base)
    again, _ = fp8mm.lora_forward(_strided(x), down, up, ids, scales, base=wide, out=wide)
    assert torch.equal(again, out)
    _check_lora(dev, val, scaled=False, based=False)
    dy, dyv = _dev(rng.standard_normal((T, N)), torch.bfloat16)
    got = _check_lora_backward(dev, val, v, dy, dyv)
    for a, b in zip(fp8mm.lora_backward(_strided(dy, 1, 2), _strided(x), v, down, up, ids, scales), got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,K,N,n,r,segments", [(300, 512, 640, 4, 16, 1), (1025, 520, 777, 3, 64, 5),
                                                (2000, 1024, 384, 40, 8, 30), (4099, 256, 512, 2, 32, 3),
                                                (700, 2048, 5120, 2, 100, 4), (2100, 64, 2100, 2, 64, 3),
                                                (8300, 64, 2048, 2, 16, 3)])
def test_lora_of_packed_prompts(T, K, N, n, r, segments):
    say(f"lora {T}x{K}x{N} adapters {n} rank {r} segments {segments}")
    rng, dev, val = _adapters(T, K, N, n, r, T + r, segments, without=0.0 if T % 2 else 0.02)
    _, v = _check_lora(dev, val)
    dy, dyv = _dev(rng.standard_normal((T, N)), torch.bfloat16)
    _check_lora_backward(dev, val, v, dy, dyv)
    _check_lora_backward(dev, val, v, dy, dyv, grad="fp32")


@pytest.mark.parametrize("T,K,N,n,r", [(4200, 64, 4096, 3, 64), (4200, 64, 4096, 3, 100), (2100, 130, 8256, 2, 40),
                                       (100, 128, 200, 12, 100), (300, 64, 130, 40, 256), (300, 65, 131, 40, 70)])
def test_lora_in_place_of_large_ranks(T, K, N, n, r):
    """Results past the caches (streaming loads of base, in place too) and batches taken
    adapter by adapter, at ranks above 32 and above 64."""
    test_lora(T, K, N, n, r)
    _, (x, down, up, ids, scales, base), _ = _adapters(T, K, N, n, r, T + r)
    want, _ = fp8mm.lora_forward(x, down, up, ids, scales, base)
    assert fp8mm.lora_forward(x, down, up, ids, scales, base, out=base)[0] is base and torch.equal(base, want)


def test_lora_gradients_by_differences():
    """The kernels' own outputs, moved: the loss changes as the gradients say.  bf16
    outputs limit this to a few per cent of a direction's change."""
    rng, (x, down, up, ids, scales, base), _ = _adapters(96, 256, 384, 3, 16, 3)
    dy = torch.randn((96, 384), device=DEV).bfloat16()

    def loss(x, down, up):
        return float((fp8mm.lora_forward(x, down, up, ids, scales, None)[0].double() * dy.double()).sum())

    v = fp8mm.lora_forward(x, down, up, ids, scales, None)[1]
    for i, g in enumerate(fp8mm.lora_backward(dy, x, v, down, up, ids, scales, out_dtype=torch.float32)):
        at = [x, down, up]
        step = (torch.sign(g) * at[i].abs().mean()).bfloat16() * 0.25
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + step, at[i] - step
        moved = ((hi[i].double() - lo[i].double()) * g.double()).sum()
        change = loss(*hi) - loss(*lo)      # the loss is linear in each argument by itself
        # half a bf16 step of 2 x 96 x 384 outputs, each times dy, adds up as a random sum
        noise = 6 * BF16 * float((fp8mm.lora_forward(*hi, ids, scales, None)[0].double() * dy.double()).norm()) * 2
        assert abs(change - float(moved)) <= noise + BF16 * abs(float(moved)), (i, change, float(moved), noise)


def test_lora_rows_do_not_mix():
    """NaN and infinities of tokens with another adapter, or none, stay with them."""
    for T, segments in ((48, None), (300, 6)):
        rng, (x, down, up, ids, scales, base), val = _adapters(T, 200, 300, 3, 20, 9, segments, without=0.2)
        want, v = fp8mm.lora_forward(x, down, up, ids, scales, base)
        dy = torch.randn((T, 300), device=DEV).bfloat16()
        want_g = fp8mm.lora_backward(dy, x, v, down, up, ids, scales)
        bad = torch.from_numpy((val[3] < 0) | (val[3] >= 3) | (val[3] == 1)).to(DEV)
        x2, dy2, down2, up2 = x.clone(), dy.clone(), down.clone(), up.clone()
        x2[bad], dy2[bad] = NAN, INF
        down2[1], up2[1] = INF, NAN
        out, v2 = fp8mm.lora_forward(x2, down2, up2, ids, scales, base)
        assert torch.equal(out[~bad], want[~bad])
        none = torch.from_numpy((val[3] < 0) | (val[3] >= 3)).to(DEV)
        assert torch.equal(out[none], base[none])
        dx, ddown, dup = fp8mm.lora_backward(dy2, x2, v2, down2, up2, ids, scales)
        assert torch.equal(dx[~bad], want_g[0][~bad]) and (dx[none] == 0).all()
        for g, w in ((ddown, want_g[1]), (dup, want_g[2])):
            assert torch.equal(g[0], w[0]) and torch.equal(g[2], w[2])


def test_lora_infinite_products_stay_infinite():
    x = torch.full((4, 64), 1e30, device=DEV).bfloat16()
    down, up = torch.full((1, 8, 64), 1e30, device=DEV).bfloat16(), torch.ones((1, 8, 32), device=DEV).bfloat16()
    out, _ = fp8mm.lora_forward(x, down, up, torch.zeros(4, dtype=torch.int32, device=DEV))
    assert (out == INF).all()


def _with_infinities(t, rng, share=0.004):
    """t with some infinities of both signs, and its float64 values."""
    at = torch.from_numpy(rng.random(t.shape) < share).to(DEV)
    sign = torch.from_numpy(rng.choice([-INF, INF], t.shape)).to(t.dtype).to(DEV)
    t = torch.where(at, sign, t)
    return t, _f64(t)


def _same_infinities(got, ref, clean, what):
    """Infinite and NaN where the definition is, of its sign; what no infinity reaches has
    the bits that it has without any."""
    value = _f64(got)
    assert np.array_equal(np.isnan(value), np.isnan(ref)), what
    infinite = np.isinf(ref)
    assert np.array_equal(np.isinf(value), infinite) and np.array_equal(value[infinite], ref[infinite]), what
    finite = torch.from_numpy(np.isfinite(ref)).to(DEV)
    assert torch.equal(got[finite], clean[finite]), what


INFINITE_SHAPES = [(16, 64, 300, 3, 8), (300, 72, 130, 40, 16), (200, 130, 513, 3, 64), (130, 64, 264, 2, 100),
                   (70, 64, 96, 2, 256), (90, 100, 5, 3, 24), (90, 5, 100, 3, 24), (700, 40, 1100, 3, 32),
                   (4200, 24, 4096, 2, 20)]


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("T,K,N,n,r", INFINITE_SHAPES)
def test_lora_of_infinite_panels_and_rows(T, K, N, n, r, whole):
    """Times a finite number an infinity stays one, of the product's sign: the two halves of
    that number, the second of which may be 0 or of the other sign, must not show.  whole:
    inner products that are odd whole numbers, with no second half."""
    say(f"lora with infinities {T}x{K}x{N} adapters {n} rank {r}")
    if whole:
        K, N = K // 2 * 2 + 1, N // 2 * 2 + 1        # sums of that many ones of either sign
    rng, (x, down, up, ids, scales, base), (_, _, _, idv, sv, basev) = _adapters(T, K, N, n, r, T + r)
    dy = _dev(rng.standard_normal((T, N)), torch.bfloat16)[0]
    if whole:
        x, dy, down, up = (torch.where(t < 0, -1.0, 1.0).bfloat16() for t in (x, dy, down, up))
    xv, dyv, downv, upv = (_f64(t) for t in (x, dy, down, up))
    out, v = fp8mm.lora_forward(x, down, up, ids, scales, base)
    with np.errstate(all="ignore"):
        bad, badv = _with_infinities(up, rng)
        ref = block.lora(xv, downv, badv, idv, sv, basev)[0]
        _same_infinities(fp8mm.lora_forward(x, down, bad, ids, scales, base)[0], ref, out, "out")
        inplace = base.clone()
        fp8mm.lora_forward(x, down, bad, ids, scales, inplace, out=inplace)
        _same_infinities(inplace, ref, out, "out on base")
        for grad in (torch.bfloat16, torch.float32):
            clean = fp8mm.lora_backward(dy, x, v, down, up, ids, scales, out_dtype=grad)
            bad, badv = _with_infinities(down, rng)
            got = fp8mm.lora_backward(dy, x, v, bad, up, ids, scales, out_dtype=grad)
            _same_infinities(got[0], block.lora_backward(dyv, xv, badv, upv, idv, sv)[0], clean[0], "dx")
            bad, badv = _with_infinities(x, rng, 0.001)
            got = fp8mm.lora_backward(dy, bad, None, down, up, ids, scales, False, True, False, grad)
            _same_infinities(got[1], block.lora_backward(dyv, badv, downv, upv, idv, sv)[1], clean[1], "ddown")
            bad, badv = _with_infinities(dy, rng, 0.001)
            got = fp8mm.lora_backward(bad, x, v, down, up, ids, scales, False, False, True, grad)
            _same_infinities(got[2], block.lora_backward(badv, xv, downv, upv, idv, sv)[2], clean[2], "dup")


def test_lora_of_infinities_on_both_sides():
    """An infinite inner product with an infinite panel."""
    for r in (8, 40, 80):
        x = torch.full((20, 64), 1e30, device=DEV).bfloat16()
        down = torch.full((2, r, 64), 1e30, device=DEV).bfloat16()
        up = torch.ones((2, r, 32), device=DEV).bfloat16()
        up[1, :, 3], up[1, :, 4], up[1, 0, 5] = INF, -INF, -INF
        ids = torch.arange(20, device=DEV, dtype=torch.int32) % 2
        out, _ = fp8mm.lora_forward(x, down, up, ids)
        want = torch.full((20, 32), INF, device=DEV)
        want[1::2, 4], want[1::2, 5] = -INF, NAN
        assert torch.equal(out.float().nan_to_num(7.0, 1.0, -1.0), want.nan_to_num(7.0, 1.0, -1.0))


def test_lora_of_inner_products_past_the_range_of_bf16():
    """v is float32: between bf16's largest number and its own it is not an infinity."""
    # bf16's largest, 2^128 - 2^120, and 0.75 of a step of it: below 2^128, where float32 ends
    top, rest = 2.0 ** 128 - 2.0 ** 120, 1.5 * 2.0 ** 119
    for T, r in ((20, 4), (300, 40), (70, 100)):
        x = torch.ones((T, 2), device=DEV).bfloat16()
        x[::2] *= -1
        down = torch.tensor([top, rest], device=DEV).bfloat16().expand(40, r, 2).contiguous()
        up = torch.full((40, r, 16), 2.0 ** -60, device=DEV).bfloat16()
        ids = torch.arange(T, device=DEV, dtype=torch.int32) % 40
        out, v = fp8mm.lora_forward(x, down, up, ids)
        val = _f64(x), _f64(down), _f64(up), ids.cpu().numpy()
        ref, vref = block.lora(*val)
        assert np.array_equal(_f64(v).sum(0)[:, :r], vref) and np.isfinite(vref).all()
        tol = (V_SPLIT + (2 * r + 24) * U) * np.abs(ref)
        _within(_f64(out), ref, _rounded(ref, tol, BF16), "out")
        dy = torch.full((T, 16), 2.0 ** -60, device=DEV).bfloat16()
        for dtype, half in (("bf16", BF16), ("fp32", U)):
            dup = fp8mm.lora_backward(dy, None, v, down, up, ids, None, False, False, True, DT[dtype])[2]
            ref = np.zeros(dup.shape)
            for a in range(40):
                ref[a] = vref[val[3] == a].T @ _f64(dy)[val[3] == a]
            size = np.array([np.abs(vref[val[3] == a]).sum() for a in range(40)])[:, None, None] * 2.0 ** -60
            _within(_f64(dup), ref, _rounded(ref, (V_SPLIT + (2 * T + 40) * U) * size, half), "dup")


@pytest.mark.parametrize("T,K,N,n,r", [(40, 64, 40, 40, 8), (200, 100, 130, 100, 20), (90, 64, 72, 60, 33),
                                       (70, 40, 200, 70, 100), (30, 5, 40, 30, 16)])
def test_lora_gradients_in_float32_keep_all_bits_of_v(T, K, N, n, r):
    """A few tokens an adapter.  v and dv enter as three bf16 numbers each, whose products
    with bf16 are exact: what is lost are additions, three a token, at up to a step each,
    and those of the partial sums and the scale.  (As two numbers v is off by up to 128 U.)"""
    rng, (x, down, up, ids, scales, base), (xv, _, upv, _, sv, _) = _adapters(T, K, N, n, r, T + r)
    idv = (np.arange(T) * 7 % n).astype(np.int32)
    ids = torch.from_numpy(idv).to(DEV)
    shape = fp8mm.lora_forward(x, down, up, ids, scales)[1].shape
    v = torch.zeros(shape, device=DEV)
    v[0, :, :r] = torch.from_numpy(rng.standard_normal((T, r)).astype(np.float32)).to(DEV)
    dy, dyv = _dev(rng.standard_normal((T, N)), torch.bfloat16)
    dup = fp8mm.lora_backward(dy, None, v, down, up, ids, scales, False, False, True, torch.float32)[2]
    vv, ref, size = _f64(v)[0, :, :r], np.zeros(dup.shape), np.zeros(dup.shape)
    most = np.bincount(idv).max()
    for a in range(n):
        at = idv == a
        ref[a], size[a] = sv[a] * vv[at].T @ dyv[at], sv[a] * np.abs(vv[at]).T @ np.abs(dyv[at])
    _within(_f64(dup), ref, (6 * most + 4) * U * size + TINY, "dup")
    # dv = s up dy of three columns, all positive: three products and their additions
    dy, up = dy.abs(), up.abs()
    dy[:, 3:] = 0
    dyv, upv = _f64(dy), _f64(up)
    ddown = fp8mm.lora_backward(dy, x, None, down, up, ids, scales, False, True, False, torch.float32)[1]
    ref, size = np.zeros(ddown.shape), np.zeros(ddown.shape)
    for a in range(n):
        at = idv == a
        dv = sv[a] * dyv[at] @ upv[a].T
        ref[a], size[a] = dv.T @ xv[at], dv.T @ np.abs(xv[at])
    _within(_f64(ddown), ref, (6 * most + 4 + 6 + 4) * U * size + TINY, "ddown")


def test_lora_without_tokens_and_without_adapters():
    rng, (x, down, up, ids, scales, base), _ = _adapters(70, 64, 96, 3, 8, 1)
    out, v = fp8mm.lora_forward(x[:0], down, up, ids[:0], scales, base[:0])
    assert out.shape == (0, 96)
    dx, ddown, dup = fp8mm.lora_backward(base[:0], x[:0], v, down, up, ids[:0], scales)
    assert dx.shape == (0, 64) and (ddown == 0).all() and (dup == 0).all()
    none = torch.full_like(ids, -1)
    out, v = fp8mm.lora_forward(x, down, up, none, scales, base)
    assert torch.equal(out, base)
    assert (fp8mm.lora_forward(x, down, up, none)[0] == 0).all()
    dx, ddown, dup = fp8mm.lora_backward(base, x, v, down, up, none, scales)
    assert (dx == 0).all() and (ddown == 0).all() and (dup == 0).all()


def test_lora_gradients_of_adapters_without_tokens():
    """Zeros, whatever their panels and scales hold."""
    rng, (x, down, up, ids, scales, base), _ = _adapters(90, 64, 96, 4, 20, 1)
    ids[ids == 1], ids[ids == 2] = 0, 3
    v = fp8mm.lora_forward(x, down, up, ids, scales)[1]
    for dtype in (torch.bfloat16, torch.float32):
        want = fp8mm.lora_backward(base, x, v, down, up, ids, scales, out_dtype=dtype)
        for value in (NAN, INF):
            scales2, down2, up2 = scales.clone(), down.clone(), up.clone()
            scales2[1:3], down2[1:3], up2[1:3] = value, value, value
            dx, ddown, dup = fp8mm.lora_backward(base, x, v, down2, up2, ids, scales2, out_dtype=dtype)
            assert torch.equal(dx, want[0])
            for g, w in ((ddown, want[1]), (dup, want[2])):
                assert (g[1:3] == 0).all() and torch.equal(g[[0, 3]], w[[0, 3]])


def test_lora_parts_of_the_backward():
    rng, (x, down, up, ids, scales, base), _ = _adapters(150, 130, 200, 3, 12, 2)
    v = fp8mm.lora_forward(x, down, up, ids, scales)[1]
    dy = torch.randn((150, 200), device=DEV).bfloat16()
    whole = fp8mm.lora_backward(dy, x, v, down, up, ids, scales)
    for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)):
        part = fp8mm.lora_backward(dy, x if need[1] else None, v if need[2] else None, down, up, ids, scales, *need)
        for g, w, n in zip(part, whole, need):
            assert torch.equal(g, w) if n else g is None


def test_lora_autograd_and_refusals():
    rng, (x, down, up, ids, scales, base), _ = _adapters(80, 128, 192, 3, 16, 4)
    leaves = [t.clone().requires_grad_() for t in (x, down, up, base)]
    dy = torch.randn((80, 192), device=DEV).bfloat16()
    out = fp8mm.lora(leaves[0], leaves[1], leaves[2], ids, scales, leaves[3])
    want, v = fp8mm.lora_forward(x, down, up, ids, scales, base)
    assert torch.equal(out, want)
    out.backward(dy)
    grads = (*fp8mm.lora_backward(dy, x, v, down, up, ids, scales), dy)
    assert all(torch.equal(t.grad, g) for t, g in zip(leaves, grads))
    with torch.no_grad():
        assert torch.equal(fp8mm.lora(*leaves[:3], ids, scales, leaves[3]), want)
    for bad in (lambda: fp8mm.lora_forward(x.float(), down, up, ids), lambda: fp8mm.lora_forward(x, down, up, ids.long()),
                lambda: fp8mm.lora_forward(x, down[:, :8].contiguous(), up, ids),
                lambda: fp8mm.lora_forward(x, down, up, ids[:4]), lambda: fp8mm.lora_forward(x[:, :64], down, up, ids),
                lambda: fp8mm.lora_forward(x, down, up, ids, scales[:2]),
                lambda: fp8mm.lora_forward(x, down, up, ids, scales, base[:, :64]),
                lambda: fp8mm.lora_backward(dy, None, v, down, up, ids), lambda: fp8mm.lora_backward(dy, x, None, down, up, ids),
                lambda: fp8mm.lora_backward(dy, x, v, down, up, ids, out_dtype=torch.float16),
                lambda: fp8mm.rms_norm_forward(x.half()), lambda: fp8mm.rms_norm_forward(x, scales),
                lambda: fp8mm.rms_norm_forward(x, None, x.float()), lambda: fp8mm.fp8_rms_norm_forward(x.float()),
                lambda: fp8mm.fp8_rms_norm_forward(x, recipe="none"), lambda: fp8mm.rms_norm_forward(x.t()),
                lambda: fp8mm.fp8_rms_norm_forward(x[:, :120].contiguous()),
                lambda: fp8mm.moe_balance_loss_forward(x, ids), lambda: fp8mm.moe_balance_loss_forward(x, ids[:, None], "none"),
                lambda: fp8mm.moe_balance_loss_forward(x, ids[:, None].contiguous(), ends=ids[:0])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fp8mm.fp8_rms_norm_forward(x, recipe="tensorwise"),
                lambda: fp8mm.lora_forward(x, torch.zeros((1, 300, 128), device=DEV).bfloat16(),
                                           torch.zeros((1, 300, 8), device=DEV).bfloat16(), ids)):
        with pytest.raises(NotImplementedError):
            bad()


# -------------------------------------------------------------------- together

def _block_step(x, res, w, qw, sw, down, up, ids, scales, router, k=2):
    """Norm with residual and codes, FP8 product with adapters, norm, router with its
    balance loss."""
    q, s, y, h, _ = fp8mm.fp8_rms_norm_forward(x, w, res, y=True)
    out = fp8mm.fp8_scaled_mm(q, qw, s, "1x128", sw, "128x128")
    fp8mm.lora_forward(y, down, up, ids, scales, base=out, out=out)
    n, h2, _ = fp8mm.rms_norm_forward(out, w, h)
    experts, weights = fp8mm.moe_route_forward(n @ router, k)
    loss, counts, _ = fp8mm.moe_balance_loss_forward(n @ router, experts)
    return out, h2, n, weights, loss, counts


def _block_inputs(T, C=256, n=3, r=16, E=16):
    g = torch.Generator(device=DEV).manual_seed(T)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale).bfloat16()

    qw, sw = fp8mm.fp8_quantize_blockwise(normal(C, C, scale=C ** -0.5), (128, 128))
    ids = torch.randint(-1, n, (T,), generator=g, device=DEV).to(torch.int32)
    return (normal(T, C), normal(T, C), normal(C), qw, sw, normal(n, r, C, scale=C ** -0.5), normal(n, r, C, scale=0.5),
            ids, torch.rand(n, generator=g, device=DEV), normal(C, E, scale=C ** -0.5))


@pytest.mark.parametrize("T", [1, 5, 384])
def test_operators_run_together(T):
    inputs = _block_inputs(T)
    x, res, w, qw, sw, down, up, ids, scales, router = inputs
    out, h2, n, weights, loss, counts = _block_step(*inputs)
    y, h, _ = fp8mm.rms_norm_forward(x, w, res)
    plain = fp8mm.fp8_scaled_mm(*fp8mm.fp8_rms_norm_forward(x, w, res)[:1], qw,
                                fp8mm.fp8_rms_norm_forward(x, w, res)[1], "1x128", sw, "128x128")
    ref, _ = block.lora(_f64(y), _f64(down), _f64(up), ids.cpu().numpy(), _f64(scales), _f64(plain))
    size = np.abs(_f64(plain)) + block.lora(np.abs(_f64(y)), np.abs(_f64(down)), np.abs(_f64(up)), ids.cpu().numpy(),
                                            _f64(scales))[0]
    _within(_f64(out), ref, BF16 * np.abs(ref) + (2 * V_SPLIT + 600 * U) * size, "product with adapters")
    assert torch.equal(h2.cpu(), (out.cpu().float() + h.cpu().float()).bfloat16())
    assert int(counts.sum()) == 2 * T and float(loss) > 0


def test_captured_run_follows_its_inputs():
    """The run in a graph, replayed on new inputs between eager runs of the same calls on
    another stream: each replay gives the eager result."""
    inputs = _block_inputs(96)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            _block_step(*inputs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _block_step(*inputs)
    for seed in range(4):
        fresh = _block_inputs(96)
        for a, b in zip(inputs, fresh):
            if a.is_floating_point() and a.dtype == torch.bfloat16:
                a.copy_(b * (1 + 0.125 * seed))
        inputs[7].copy_((fresh[7] + seed) % 3)
        graph.replay()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            want = _block_step(*inputs)
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            assert torch.equal(got, ref), seed


def test_captured_training_step():
    """Forward and backward of the three differentiable operators in a graph, replayed,
    against the same step run eagerly."""
    x, res, w, _, _, down, up, ids, scales, router = _block_inputs(130)
    leaves = [t.clone().requires_grad_() for t in (x, res, w, down, up, router)]
    one, gw, gout = torch.ones((), device=DEV), torch.randn((130, 2), device=DEV), torch.randn_like(x)

    def step():
        for t in leaves:
            t.grad = None
        x, res, w, down, up, router = leaves
        y, h = fp8mm.rms_norm(x, w, res)
        out = fp8mm.lora(y, down, up, ids, scales, h)
        logits = fp8mm.rms_norm(out, w) @ router
        experts, weights = fp8mm.moe_route(logits, 2)
        loss, _ = fp8mm.moe_balance_loss(logits, experts, coeff=10.0)
        torch.autograd.backward([loss, weights, out], [one, gw, gout])
        return [t.grad for t in leaves]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            want = [g.clone() for g in step()]
        for t in leaves:
            t.grad = None
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step()
    for _ in range(3):
        for g in grads:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(grads, want):
            assert not ref.isnan().any() and torch.equal(got, ref)


def test_rows_far_apart():
    """Row strides that put the last rows past 2^31 and 2^32 elements: the bits of dense rows."""
    store = torch.empty(5 << 30, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)

    def far(t, start=1):
        flat = store.view(t.dtype)[start:]
        view = flat.as_strided(t.shape, ((flat.numel() - t.shape[1]) // (t.shape[0] - 1), 1))
        return view.copy_(t)

    for dtype in (torch.bfloat16, torch.float32):
        for R, C in ((5, 256), (600, 1040), (40, 20000)):
            x, dy = (torch.randn((R, C), generator=g, device=DEV).to(dtype) for _ in range(2))
            y, _, rstd = fp8mm.rms_norm_forward(x)
            assert torch.equal(fp8mm.rms_norm_forward(far(x))[0], y)
            want = fp8mm.rms_norm_backward(dy, x, None, rstd)
            for at in range(2):
                rows = (far(dy), x) if at == 0 else (dy, far(x))
                assert all(torch.equal(a, b) for a, b in zip(fp8mm.rms_norm_backward(*rows, None, rstd), want))
        for T, E in ((60, 64), (3000, 300)):
            x = torch.randn((T, E), generator=g, device=DEV).to(dtype)
            ids = torch.randint(0, E, (T, 3), generator=g, device=DEV, dtype=torch.int32)
            want = fp8mm.moe_balance_loss_forward(x, ids)
            assert all(torch.equal(a, b) for a, b in zip(fp8mm.moe_balance_loss_forward(far(x), ids), want))
            one = torch.ones((), device=DEV)
            assert torch.equal(fp8mm.moe_balance_loss_backward(one, far(x), *want[1:], 3),
                               fp8mm.moe_balance_loss_backward(one, x, *want[1:], 3))
    for T, n in ((40, 3), (300, 40), (1000, 5)):
        _, (x, down, up, ids, scales, base), _ = _adapters(T, 200, 264, n, 16, T)
        want, v = fp8mm.lora_forward(x, down, up, ids, scales, base)
        assert torch.equal(fp8mm.lora_forward(far(x), down, up, ids, scales, base)[0], want)
        inplace = far(base)
        assert torch.equal(fp8mm.lora_forward(x, down, up, ids, scales, inplace, out=inplace)[0], want)
        grads = fp8mm.lora_backward(want, x, v, down, up, ids, scales)
        for at in range(2):              # one at a time: they share the memory
            rows = (far(want), x) if at == 0 else (want, far(x))
            assert all(torch.equal(a, b) for a, b in zip(fp8mm.lora_backward(*rows, v, down, up, ids, scales), grads))


def test_two_streams_at_once():
    """Independent calls on two streams do not disturb each other (each has its own
    workspace)."""
    a, b = _block_inputs(300), _block_inputs(301)
    want = [_block_step(*t) for t in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, (s, t) in enumerate(zip(streams, (a, b))):
            with torch.cuda.stream(s):
                got[i] = _block_step(*t)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(g, w))


def test_results_repeat_bit_for_bit():
    rng, (x, down, up, ids, scales, base), _ = _adapters(600, 512, 512, 4, 16, 8, 5)
    logits = torch.randn((600, 64), device=DEV)
    e, _ = fp8mm.moe_route_forward(logits, 4)

    def once():
        out, v = fp8mm.lora_forward(x, down, up, ids, scales, base)
        y, h, rstd = fp8mm.rms_norm_forward(x, None, base)
        return (out, *fp8mm.lora_backward(base, x, v, down, up, ids, scales), y, h,
                *fp8mm.rms_norm_backward(x, h, None, rstd, base), *fp8mm.moe_balance_loss_forward(logits, e))

    first = once()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(once(), first))
