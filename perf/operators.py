"""Measured cases of the operators around the grouped FP8 GEMMs.

Five operations of a mixture-of-experts block: layer norm in front of it, the
routing of tokens to experts, the permutation of token rows into expert order
(dispatch) and back (combine), and the gated activation between the experts'
two products, which keeps its input in 8 bits for the backward pass.

``run`` computes each one in plain float32 torch operations, or through
``precision_matmul_amd`` where ``own`` is true.  ``exact`` gives the same
outputs from the definitions in float64.  A case is a dict of plain values:

  layer_norm   rows, cols, dtype, params (their dtype), backward
  route        tokens, experts, k, score, bias, groups, group_topk,
               group_score, renormalize, scale, dtype, masked (share of rows
               that are padding: every logit -inf), backward
  dispatch     tokens, cols, experts, k, form ("fp8": 1x128 codes and scales,
               else the rows themselves in "bf16" or "fp32"), empty (share of
               slots without an expert)
  combine      tokens, cols, experts, k, dtype, weighted, empty, backward
  swiglu       rows, half, out ("fp8" codes or "bf16"), checkpoint, backward
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5           # layer norm
RENORM_EPS = 1e-20   # renormalised weights: w / (sum + RENORM_EPS)


# --------------------------------------------------------------------- cases

def listed():
    return [
        # the norm of one decoding step: a handful of sequences, latency only
        dict(name="norm_tokens_5x2048", op="layer_norm", rows=5, cols=2048, dtype="bf16", params="bf16", backward=False),
        # the norm in front of the dense layers, training batch
        dict(name="norm_16640x5120", op="layer_norm", rows=16640, cols=5120, dtype="bf16", params="bf16", backward=False),
        # its backward pass at the expert layer's width, float32 parameters
        dict(name="norm_grad_16384x2048", op="layer_norm", rows=16384, cols=2048, dtype="bf16", params="fp32",
             backward=True),
        # routing of one decoding step
        dict(name="route_tokens_7x64", op="route", tokens=7, experts=64, k=6, score="softmax", bias=False, groups=1,
             group_topk=1, group_score="max", renormalize=True, scale=1.0, dtype="bf16", masked=0.0, backward=False),
        # routing of a training batch: sigmoid scores, balance bias, groups
        dict(name="route_groups_16384x256", op="route", tokens=16384, experts=256, k=8, score="sigmoid", bias=True,
             groups=8, group_topk=4, group_score="top2", renormalize=True, scale=2.5, dtype="fp32", masked=0.02,
             backward=False),
        # gradient of the logits, plain softmax weights
        dict(name="route_grad_16384x64", op="route", tokens=16384, experts=64, k=6, score="softmax", bias=False,
             groups=1, group_topk=1, group_score="max", renormalize=False, scale=1.0, dtype="fp32", masked=0.0,
             backward=True),
        # decoding step: plan, gather and quantization of a few tokens
        dict(name="dispatch_tokens_16x2048", op="dispatch", tokens=16, cols=2048, experts=64, k=6, form="fp8", empty=0.0),
        # training batch into the expert layer of 64 x 1408 x 2048
        dict(name="dispatch_16384x2048", op="dispatch", tokens=16384, cols=2048, experts=64, k=6, form="fp8", empty=0.0),
        # a prompt of ragged length with padding tokens
        dict(name="combine_4099x2048", op="combine", tokens=4099, cols=2048, experts=64, k=6, dtype="bf16",
             weighted=True, empty=0.05, backward=False),
        # backward of the training batch: gradients of the rows and of the weights
        dict(name="combine_grad_16384x2048", op="combine", tokens=16384, cols=2048, experts=64, k=6, dtype="bf16",
             weighted=True, empty=0.0, backward=True),
        # forward of a ragged prompt: codes for the second product, codes kept for the backward
        dict(name="swiglu_10007x1408", op="swiglu", rows=10007, half=1408, out="fp8", checkpoint=True, backward=False),
        # backward of the training batch from the kept codes, the activation again for the weight gradient
        dict(name="swiglu_grad_98304x1408", op="swiglu", rows=98304, half=1408, out="bf16", checkpoint=True,
             backward=True),
    ]


MOST_ELEMENTS = 16384 * 6 * 2048      # expert-order rows x columns of the largest listed cases
UNUSED = 3072                         # not a size of any configuration here


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(hi, max(lo, n))
    return n + 1 if n == UNUSED else n


def draw(rng):
    op = rng.choice(["layer_norm", "route", "dispatch", "combine", "swiglu"])
    if op == "layer_norm":
        cols = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024), 128 * _log(rng, 1, 64)])
        cols += 8 if cols == UNUSED else 0
        rows = _log(rng, 1, min(16640, 16640 * 5120 // cols))
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        if dtype == "fp32":
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows + (rows == UNUSED), cols=cols, dtype=dtype, params=rng.choice(["bf16", "fp32"]),
                    backward=rng.random() < 0.5)
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * _log(rng, max(2, 8 // groups), 256 // groups)
        group_topk = 1 if groups == 1 else rng.randint(1, groups // 2)
        k = rng.randint(1, min(8, experts // groups * group_topk))
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, k=k, score=score, bias=rng.random() < 0.5,
                    groups=groups, group_topk=group_topk, group_score=rng.choice(["max", "top2"]),
                    renormalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["bf16", "fp32"]),
                    masked=rng.choice([0.0, 0.1]), backward=rng.random() < 0.4)
    k = rng.randint(1, 8)
    experts = _log(rng, max(8, k), 256)
    empty = rng.choice([0.0, 0.0, 0.1])
    if op == "dispatch":
        form = rng.choice(["fp8", "fp8", "bf16", "fp32"])
        cols = 128 * _log(rng, 1, 40)
        cols += 128 if cols == UNUSED else 0
        most = MOST_ELEMENTS // (cols * k) // {"fp8": 1, "bf16": 2, "fp32": 4}[form]
        return dict(op=op, tokens=_log(rng, 1, max(1, min(16384, most))), cols=cols, experts=experts, k=k, form=form,
                    empty=empty)
    if op == "combine":
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        cols = rng.choice([128 * _log(rng, 1, 40), _log(rng, 64, 5120)])
        cols += 128 if cols == UNUSED else 0
        most = MOST_ELEMENTS // (cols * k) // (2 if dtype == "fp32" else 1)
        backward = rng.random() < 0.5
        return dict(op=op, tokens=_log(rng, 1, max(1, min(16384, most))), cols=cols, experts=experts, k=k, dtype=dtype,
                    weighted=backward or rng.random() < 0.6, empty=empty, backward=backward)
    half = 128 * _log(rng, 1, 40)
    half += 128 if 2 * half == UNUSED or half == UNUSED else 0
    rows = _log(rng, 1, min(98304, 98304 * 1408 // half))
    backward = rng.random() < 0.5
    return dict(op=op, rows=rows, half=half, out="bf16" if backward else rng.choice(["fp8", "fp8", "bf16"]),
                checkpoint=backward or rng.random() < 0.7, backward=backward)


# -------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, sigma, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _draw_ids(g, case):
    """Distinct experts for each token, popular ones more often; empty slots
    (padding tokens, dropped slots) are -1."""
    T, E, k = case["tokens"], case["experts"], case["k"]
    popular = torch.randn((E,), generator=g, device="cuda") * 0.7
    noise = torch.rand((T, E), generator=g, device="cuda").clamp_min(1e-9)
    ids = (popular - torch.log(-torch.log(noise))).argsort(-1, descending=True)[:, :k].to(torch.int32)
    if case["empty"]:
        gone = torch.rand((T, k), generator=g, device="cuda") < case["empty"] / 2
        gone |= torch.rand((T, 1), generator=g, device="cuda") < case["empty"] / 2
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.contiguous()


def _logits(g, case):
    """Router logits whose choice does not hang on the last bit of a score:
    rows with two keys (or group scores) of unequal experts nearer than 4e-6
    at a place that decides are drawn again, so that the chosen ids are whole
    numbers with one right answer."""
    T, E = case["tokens"], case["experts"]
    dtype = DTYPES[case["dtype"]]
    popular = torch.randn((E,), generator=g, device="cuda") * 0.5
    bias = torch.round(torch.randn((E,), generator=g, device="cuda") * 30) * 1e-3 if case["bias"] else None
    out = torch.empty((T, E), dtype=dtype, device="cuda")
    todo = torch.arange(T, device="cuda")
    for _ in range(12):
        fresh = (torch.randn((todo.numel(), E), generator=g, device="cuda") * 1.3 + popular).to(dtype)
        out[todo] = fresh
        todo = todo[~_clear(fresh, bias, case)]
        if todo.numel() == 0:
            break
    else:
        out[todo] = (torch.arange(E, device="cuda") * -0.0625).to(dtype)   # far apart in every key
    if case["masked"]:
        out[torch.rand((T,), generator=g, device="cuda") < case["masked"]] = -math.inf
    return out, bias


def _clear(logits, bias, case):
    T, E = logits.shape
    x = logits.double()
    s = torch.softmax(x, -1) if case["score"] == "softmax" else torch.sigmoid(x)
    value = s if bias is None else s + bias.double()
    fine = torch.ones((T,), dtype=torch.bool, device=x.device)

    def apart(sorted_keys, at):
        gap = sorted_keys[:, :-1] - sorted_keys[:, 1:]
        gap = gap[:, at] if at is not None else gap
        return ((gap == 0) | (gap > 4e-6)).reshape(T, -1).all(-1)

    keys = x if bias is None else value
    G = case["groups"]
    if G > 1 and case["group_topk"] < G:
        by_max = case["group_score"] == "max"
        grouped = (keys if by_max else value).reshape(T, G, E // G)
        top = grouped.amax(-1) if by_max else grouped.sort(dim=-1, descending=True)[0][..., :2].sum(-1)
        ranked, order = top.sort(dim=-1, descending=True, stable=True)
        if not (by_max and bias is None):
            fine &= apart(ranked, case["group_topk"] - 1)
        kept = torch.zeros((T, G), dtype=torch.bool, device=x.device)
        kept.scatter_(1, order[:, :case["group_topk"]], True)
        keys = keys.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
    if bias is not None:
        best = keys.sort(dim=-1, descending=True)[0][:, :case["k"] + 1]
        best = torch.nan_to_num(best, neginf=-100.0)
        fine &= apart(best, None)
    return fine


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "layer_norm":
        dtype, params = DTYPES[case["dtype"]], DTYPES[case["params"]]
        R, C = case["rows"], case["cols"]
        offset = torch.randn((R, 1), generator=g, device="cuda") * 0.5
        st["x"] = (torch.randn((R, C), generator=g, device="cuda") * 1.5 + offset).to(dtype)
        st["weight"] = (1 + 0.1 * torch.randn((C,), generator=g, device="cuda")).to(params)
        st["bias"] = _normal(g, (C,), 0.1, params)
        if case["backward"]:
            st["dy"] = _normal(g, (R, C), 1e-2, dtype)
            x = st["x"].float()
            st["mean"] = x.mean(-1)
            st["rstd"] = 1 / torch.sqrt((x - st["mean"][:, None]).square().mean(-1) + EPS)
    elif op == "route":
        st["logits"], st["bias"] = _logits(g, case)
        if case["backward"]:
            st["ids"], st["weights"] = _route_plain(st["logits"], st["bias"], case)
            st["grad"] = _normal(g, (case["tokens"], case["k"]), 1.0, torch.float32)
    elif op == "dispatch":
        dtype = torch.bfloat16 if case["form"] == "fp8" else DTYPES[case["form"]]
        st["ids"] = _draw_ids(g, case)
        st["x"] = _normal(g, (case["tokens"], case["cols"]), 1.0, dtype)
    elif op == "combine":
        dtype = DTYPES[case["dtype"]]
        T, C, k = case["tokens"], case["cols"], case["k"]
        ids = _draw_ids(g, case)
        st["offsets"], st["row_of_slot"] = _plan_plain(ids, case["experts"])
        st["rows"] = _normal(g, (T * k, C), 1.0, dtype)
        st["weights"] = None
        if case["weighted"]:
            w = torch.rand((T, k), generator=g, device="cuda") + 0.05
            st["weights"] = (w / w.sum(-1, keepdim=True)).contiguous()
        if case["backward"]:
            st["grad"] = _normal(g, (T, C), 1e-2, dtype)
    else:
        R, F = case["rows"], case["half"]
        x = _normal(g, (R, 2 * F), 1.2, torch.bfloat16)
        if case["backward"]:
            st["codes"], st["scale"] = _quantize_plain(x.float())
            st["grad"] = _normal(g, (R, F), 1e-2, torch.bfloat16)
        else:
            st["x"] = x
    return st


# --------------------------------------------------------------- plain forms

def _norm_plain(x, weight, bias):
    v = x.float()
    mean = v.sum(-1) / v.shape[1]
    d = v - mean[:, None]
    rstd = 1 / torch.sqrt(d.square().sum(-1) / v.shape[1] + EPS)
    return (d * rstd[:, None] * weight.float() + bias.float()).to(x.dtype), mean, rstd


def _norm_grad_plain(dy, x, weight, mean, rstd):
    g, C = dy.float(), x.shape[1]
    xh = (x.float() - mean[:, None]) * rstd[:, None]
    a = g * weight.float()
    dx = rstd[:, None] * (a - a.sum(-1, keepdim=True) / C - xh * ((a * xh).sum(-1, keepdim=True) / C))
    return dx.to(x.dtype), (g * xh).sum(0).to(weight.dtype), g.sum(0).to(weight.dtype)


def _scores_plain(logits, score):
    x = logits.float()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _route_plain(logits, bias, case):
    T, E = logits.shape
    G, k = case["groups"], case["k"]
    x = logits.float()
    s = _scores_plain(logits, case["score"])
    off = x == -math.inf
    value = (s if bias is None else s + bias).masked_fill(off, -math.inf)
    keys = x if bias is None else value
    if G > 1 and case["group_topk"] < G:
        if case["group_score"] == "max":
            top = keys.reshape(T, G, E // G).amax(-1)
        else:
            two = value.reshape(T, G, E // G).sort(dim=-1, descending=True)[0][..., :2]
            top = torch.where(two[..., 1] == -math.inf, two[..., 0], two[..., 0] + two[..., 1])
        order = top.sort(dim=-1, descending=True, stable=True)[1]
        kept = torch.zeros((T, G), dtype=torch.bool, device=x.device)
        kept.scatter_(1, order[:, :case["group_topk"]], True)
        keys = torch.where(kept.repeat_interleave(E // G, 1), keys, torch.full_like(keys, -math.inf))
    best, ids = keys.sort(dim=-1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    none = best == -math.inf
    w = torch.where(none, torch.zeros_like(best), s.gather(1, ids))
    if case["renormalize"]:
        w = w / (w.sum(-1, keepdim=True) + RENORM_EPS)
    return torch.where(none, torch.full_like(ids, -1), ids).to(torch.int32), w * case["scale"]


def _route_grad_plain(logits, ids, grad, case):
    s = _scores_plain(logits, case["score"])
    none = ids < 0
    at = torch.where(none, torch.zeros_like(ids), ids).long()
    chosen = torch.where(none, torch.zeros_like(grad), s.gather(1, at))
    gw = torch.where(none, torch.zeros_like(grad), grad) * case["scale"]
    if case["renormalize"]:
        total = chosen.sum(-1, keepdim=True) + RENORM_EPS
        gw = (gw - (gw * chosen).sum(-1, keepdim=True) / total) / total
        gw = torch.where(none, torch.zeros_like(gw), gw)
    ds = torch.zeros_like(s).scatter_add_(1, at, gw)
    if case["score"] == "sigmoid":
        return (s * (1 - s) * ds).to(logits.dtype)
    return (s * (ds - (s * ds).sum(-1, keepdim=True))).to(logits.dtype)


def _plan_plain(ids, E):
    """offsets [E] (cumulative ends) and each slot's row in expert order; slots
    without an expert take the trailing rows, written as ~row."""
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    ranked, order = key.sort(stable=True)
    row = torch.empty_like(flat)
    row[order] = torch.arange(flat.numel(), device=flat.device, dtype=torch.int32)
    offsets = torch.searchsorted(ranked, torch.arange(E, device=flat.device, dtype=torch.int32), right=True)
    return offsets.to(torch.int32), torch.where(flat < 0, ~row, row).reshape(ids.shape)


def _quantize_plain(x):
    """1x128 E4M3 codes [R, C] and scales [C/128, R] of float32 x."""
    R, C = x.shape
    v = x.reshape(R, C // 128, 128)
    amax = v.abs().amax(-1)
    s = amax / torch.full_like(amax, 448.0)
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = (v / s[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.reshape(R, C).view(torch.uint8), s.t().contiguous()


def _dispatch_plain(x, ids, case):
    T, C = x.shape
    k = case["k"]
    offsets, row_of_slot = _plan_plain(ids, case["experts"])
    flat = row_of_slot.reshape(-1)
    none = flat < 0
    row = torch.where(none, ~flat, flat).long()
    token = torch.arange(T, device=x.device).repeat_interleave(k)
    out = {"offsets": offsets, "row_of_slot": row_of_slot}
    if case["form"] == "fp8":
        q, s = _quantize_plain(x.float())
        rows = torch.empty((T * k, C), dtype=torch.uint8, device=x.device)
        rows[row] = q[token].masked_fill(none[:, None], 0)
        scale = torch.empty((C // 128, T * k), dtype=torch.float32, device=x.device)
        scale[:, row] = s[:, token].masked_fill(none, 1.0)
        out["codes"], out["scale"] = rows.view(torch.float8_e4m3fn), scale
    else:
        rows = torch.empty((T * k, C), dtype=x.dtype, device=x.device)
        rows[row] = x[token].masked_fill(none[:, None], 0)
        out["rows"] = rows
    return out


def _combine_plain(rows, row_of_slot, weights):
    T, k = row_of_slot.shape
    none = row_of_slot < 0
    v = rows[torch.where(none, torch.zeros_like(row_of_slot), row_of_slot).long().reshape(-1)].float()
    v = v.reshape(T, k, -1)
    if weights is not None:
        v = v * weights[..., None]
    return v.masked_fill(none[..., None], 0).sum(1).to(rows.dtype)


def _combine_grad_plain(grad, rows, row_of_slot, weights):
    T, k = row_of_slot.shape
    none = row_of_slot < 0
    row = torch.where(none, ~row_of_slot, row_of_slot).long().reshape(-1)
    g = grad.float()[:, None, :]
    gw = (g * rows[row].reshape(T, k, -1).float()).sum(-1).masked_fill(none, 0)
    gr = torch.empty_like(rows)
    gr[row] = (g * weights[..., None]).masked_fill(none[..., None], 0).to(rows.dtype).reshape(T * k, -1)
    return gr, gw


def _swiglu_plain(x, case):
    F = case["half"]
    v = x.float()
    gate, up = v[:, :F], v[:, F:]
    h = gate / (1 + torch.exp(-gate)) * up
    out = {}
    if case["out"] == "fp8":
        q, out["scale"] = _quantize_plain(h)
        out["codes"] = q.view(torch.float8_e4m3fn)
    else:
        out["h"] = h.to(x.dtype)
    if case["checkpoint"]:
        q, out["checkpoint_scale"] = _quantize_plain(v)
        out["checkpoint"] = q.view(torch.float8_e4m3fn)
    return out


def _swiglu_grad_plain(grad, codes, scale, F):
    R = codes.shape[0]
    v = codes.view(torch.float8_e4m3fn).float().reshape(R, -1, 128) * scale.t()[..., None]
    v = v.reshape(R, 2 * F)
    gate, up, g = v[:, :F], v[:, F:], grad.float()
    sig = 1 / (1 + torch.exp(-gate))
    grad_x = torch.cat([g * up * sig * (1 + gate * (1 - sig)), g * gate * sig], 1)
    return {"grad_x": grad_x.to(grad.dtype), "h": (gate * sig * up).to(grad.dtype)}


def _plain(st, case):
    op = case["op"]
    if op == "layer_norm":
        if case["backward"]:
            return _norm_grad_plain(st["dy"], st["x"], st["weight"], st["mean"], st["rstd"])
        return _norm_plain(st["x"], st["weight"], st["bias"])
    if op == "route":
        if case["backward"]:
            return _route_grad_plain(st["logits"], st["ids"], st["grad"], case)
        return _route_plain(st["logits"], st["bias"], case)
    if op == "dispatch":
        return _dispatch_plain(st["x"], st["ids"], case)
    if op == "combine":
        if case["backward"]:
            return _combine_grad_plain(st["grad"], st["rows"], st["row_of_slot"], st["weights"])
        return _combine_plain(st["rows"], st["row_of_slot"], st["weights"])
    if case["backward"]:
        return _swiglu_grad_plain(st["grad"], st["codes"], st["scale"], case["half"])
    return _swiglu_plain(st["x"], case)


# ------------------------------------------------------ the framework's calls

def _kernels(st, case):
    import precision_matmul_amd as fp8mm

    op = case["op"]
    if op == "layer_norm":
        if case["backward"]:
            return fp8mm.layer_norm_backward(st["dy"], st["x"], st["weight"], st["mean"], st["rstd"])
        return fp8mm.layer_norm_forward(st["x"], st["weight"], st["bias"], EPS)
    if op == "route":
        if case["backward"]:
            return fp8mm.moe_route_backward(st["grad"], st["logits"], st["ids"], score=case["score"],
                                            renormalize=case["renormalize"], scale=case["scale"])
        return fp8mm.moe_route_forward(st["logits"], case["k"], score=case["score"], bias=st["bias"],
                                       groups=case["groups"], group_topk=case["group_topk"],
                                       group_score=case["group_score"], renormalize=case["renormalize"],
                                       scale=case["scale"])
    if op == "dispatch":
        offsets, row_of_slot = fp8mm.moe_plan(st["ids"], case["experts"])
        out = {"offsets": offsets, "row_of_slot": row_of_slot}
        if case["form"] == "fp8":
            q, out["scale"] = fp8mm.fp8_moe_dispatch(st["x"], row_of_slot)
            out["codes"] = q.view(torch.float8_e4m3fn)
        else:
            out["rows"] = fp8mm.moe_dispatch_forward(st["x"], row_of_slot)
        return out
    if op == "combine":
        if case["backward"]:
            return fp8mm.moe_combine_backward(st["grad"], st["rows"], st["row_of_slot"], st["weights"])
        return fp8mm.moe_combine_forward(st["rows"], st["row_of_slot"], st["weights"])
    if case["backward"]:
        grad_x, h = fp8mm.fp8_swiglu_backward(st["grad"], st["codes"], st["scale"], recompute=True)
        return {"grad_x": grad_x, "h": h}
    h, checkpoint = fp8mm.fp8_swiglu_forward(st["x"], out=case["out"], checkpoint=case["checkpoint"])
    out = {}
    if case["out"] == "fp8":
        out["codes"], out["scale"] = h[0].view(torch.float8_e4m3fn), h[1]
    else:
        out["h"] = h
    if checkpoint is not None:
        out["checkpoint"], out["checkpoint_scale"] = checkpoint[0].view(torch.float8_e4m3fn), checkpoint[1]
    return out


def run(state):
    return _kernels(state, state["case"]) if own else _plain(state, state["case"])


# ----------------------------------------------------------- what a pass needs

def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op == "layer_norm":
        R, C, s, p = case["rows"], case["cols"], size[case["dtype"]], size[case["params"]]
        if case["backward"]:
            return {"bytes": 3 * R * C * s + 8 * R + 3 * C * p, "flops": 14 * R * C}
        return {"bytes": 2 * R * C * s + 8 * R + 2 * C * p, "flops": 8 * R * C}
    if op == "route":
        T, E, k, s = case["tokens"], case["experts"], case["k"], size[case["dtype"]]
        if case["backward"]:
            return {"bytes": 2 * T * E * s + 8 * T * k, "flops": 8 * T * E}
        return {"bytes": T * E * s + 8 * T * k + (4 * E if case["bias"] else 0), "flops": (4 + k) * T * E}
    if op == "swiglu":
        R, F = case["rows"], case["half"]
        if case["backward"]:
            return {"bytes": R * F * (2 + 2 + 4 + 2) + 8 * R * F // 128, "flops": 20 * R * F}
        moved = 4 * R * F + (R * F + 4 * R * F // 128 if case["out"] == "fp8" else 2 * R * F)
        return {"bytes": moved + (2 * R * F + 8 * R * F // 128 if case["checkpoint"] else 0), "flops": 12 * R * F}
    T, C, k, E = case["tokens"], case["cols"], case["k"], case["experts"]
    full = T * k * (1 - case["empty"])
    if op == "dispatch":
        if case["form"] == "fp8":
            return {"bytes": 2 * T * C + T * k * (C + C // 32) + 8 * T * k + 4 * E, "flops": 4 * T * C}
        return {"bytes": (T + T * k) * C * size[case["form"]] + 8 * T * k + 4 * E, "flops": T * k}
    s = size[case["dtype"]]
    if case["backward"]:
        return {"bytes": int((T + full + T * k) * C * s) + 12 * T * k, "flops": 3 * T * k * C}
    return {"bytes": int((T + full) * C * s) + (8 if case["weighted"] else 4) * T * k, "flops": 2 * T * k * C}


# ------------------------------------------------------- definitions, 64 bits

def _e4m3_64(v):
    """v rounded to the nearest E4M3 value, ties to even, kept within +-448."""
    mag = v.abs().clamp(max=448.0)
    exponent = torch.floor(torch.log2(mag.clamp_min(2.0 ** -6))).clamp(-6, 8)
    step = torch.pow(torch.full_like(mag, 2.0), exponent - 3)
    return torch.copysign(torch.round(mag / step) * step, v)


def _quantize_64(v):
    blocks = v.unflatten(1, (-1, 128))
    s = blocks.abs().max(-1)[0] / 448
    s[s == 0] = 1
    return _e4m3_64(blocks / s.unsqueeze(-1)).flatten(1), s.T


def _first_largest(v):
    """Each row's largest value's index, the lowest of equal ones."""
    index = torch.arange(v.shape[1], device=v.device)
    return torch.where(v == v.max(1, keepdim=True)[0], index, v.shape[1]).min(1)[0]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "layer_norm":
        x, w, C = st["x"].double(), st["weight"].double(), case["cols"]
        if not case["backward"]:
            mean, var = x.mean(1), x.var(1, correction=0)
            rstd = (var + EPS).rsqrt()
            return torch.addcmul(st["bias"].double(), (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), w), mean, rstd
        dy = st["dy"].double()
        centred, r = x - st["mean"].double().unsqueeze(1), st["rstd"].double().unsqueeze(1)
        dw = dy * w
        proj = (dw * centred).mean(1, keepdim=True) * r ** 2
        return r * (dw - dw.mean(1, keepdim=True) - centred * proj), (dy * centred * r).sum(0), dy.sum(0)
    if op == "route":
        x = st["logits"].double()
        if case["score"] == "softmax":
            s = torch.nan_to_num(torch.softmax(x, 1), nan=0.0)       # a row of -inf alone: no scores
        else:
            s = torch.sigmoid(x)
        if case["backward"]:
            # dw/dl of the chosen scores, through autograd in 64 bits
            x = torch.nan_to_num(x, neginf=-1e4).requires_grad_(True)
            s = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
            used = st["ids"] >= 0
            w = s.gather(1, st["ids"].clamp_min(0).long()) * used
            if case["renormalize"]:
                w = w / (w.sum(1, keepdim=True) + RENORM_EPS)
            (w * case["scale"]).backward(st["grad"].double())
            return x.grad
        value = s if st["bias"] is None else s + st["bias"].double()
        value[torch.isneginf(x)] = -math.inf
        keys = x.clone() if st["bias"] is None else value.clone()
        G, rows = case["groups"], torch.arange(case["tokens"], device=x.device)
        if case["group_topk"] < G:
            per = [v.unflatten(1, (G, -1)) for v in (keys, value)]
            if case["group_score"] == "max":
                top = per[0].max(2)[0]
            else:
                top = torch.nan_to_num(per[1].topk(2, 2)[0], neginf=0.0).sum(2)
                top[torch.isneginf(per[1]).all(2)] = -math.inf
            kept = torch.zeros_like(top, dtype=torch.bool)
            for _ in range(case["group_topk"]):
                at = _first_largest(top)
                kept[rows, at] = True
                top[rows, at] = -math.inf
            per[0][~kept] = -math.inf                  # keys, through the view
        w, ids = torch.zeros((len(rows), case["k"]), dtype=torch.float64, device=x.device), []
        for j in range(case["k"]):
            at = _first_largest(keys)
            none = torch.isneginf(keys[rows, at])
            w[:, j] = s[rows, at].masked_fill(none, 0.0)
            ids.append(at.masked_fill(none, -1))
            keys[rows, at] = -math.inf
        if case["renormalize"]:
            w = w / (w.sum(1, keepdim=True) + RENORM_EPS)
        return torch.stack(ids, 1).to(torch.int32), w * case["scale"]
    if op == "dispatch":
        ids = st["ids"].flatten().long()
        T, k, E = case["tokens"], case["k"], case["experts"]
        ids[ids < 0] = E
        order = torch.argsort(ids * (T * k) + torch.arange(T * k, device=ids.device))
        x = st["x"].double()[order // k]
        x[ids[order] == E] = 0
        if case["form"] == "fp8":
            codes, scale = _quantize_64(x)
            return {"offsets": None, "row_of_slot": None, "codes": codes, "scale": scale}
        return {"offsets": None, "row_of_slot": None, "rows": x}
    if op == "combine":
        T, k, C = case["tokens"], case["k"], case["cols"]
        at = st["row_of_slot"].flatten().long()
        used = (at >= 0).reshape(T, k)
        w = used.double() if st["weights"] is None else st["weights"].double() * used
        at = torch.where(at < 0, -1 - at, at)
        if case["backward"]:
            g = st["grad"].double()
            gr = torch.zeros((T * k, C), dtype=torch.float64, device=g.device)
            gw = torch.zeros((T, k), dtype=torch.float64, device=g.device)
            for j in range(k):
                rows = at.reshape(T, k)[:, j]
                gr[rows] = g * w[:, j:j + 1]
                gw[:, j] = torch.linalg.vecdot(g, st["rows"][rows].double()) * used[:, j]
            return gr, gw
        y = torch.zeros((T, C), dtype=torch.float64, device=w.device)
        for j in range(k):
            y += st["rows"][at.reshape(T, k)[:, j]].double() * w[:, j:j + 1]
        return y
    F = case["half"]
    if not case["backward"]:
        x = st["x"].double()
        h = x[:, :F] * torch.sigmoid(x[:, :F]) * x[:, F:]
        out = {}
        if case["out"] == "fp8":
            out["codes"], out["scale"] = _quantize_64(h)
        else:
            out["h"] = h
        if case["checkpoint"]:
            out["checkpoint"], out["checkpoint_scale"] = _quantize_64(x)
        return out
    s = st["scale"].double().T.repeat_interleave(128, 1)
    x = st["codes"].view(torch.float8_e4m3fn).double() * s
    gate, up, g = x[:, :F], x[:, F:], st["grad"].double()
    sig = torch.sigmoid(gate)
    h = gate * sig * up
    grad_gate = g * up * (sig + gate * sig * torch.sigmoid(-gate))
    return {"grad_x": torch.cat((grad_gate, g * gate * sig), 1), "h": h}
