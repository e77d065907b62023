"""The cases of the router, the norm with 8-bit output, and the experts'
products on 8-bit rows.

A case's "op" is one of
  route      the router's scores to each token's experts and weights (and, with
             grad, the gradient of the scores)
  norm       the residual's addition and the root-mean-square norm: with grad
             the gradients of both inputs and of the weight; with bits = 8 the
             result in 8-bit microscaled values beside it, which are read back
  product    rows quantised to 8 bits, times each row's expert's 8-bit weights
  layer      a serving step in one: norm to 8 bits, route, plan, the 8-bit rows
             dispatched, product, combine
"""
import functools
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
MX8 = 1.0 + 1.0 / 32.0   # bytes of a value in 8 bits: its code, and its share of a block's scale


@functools.lru_cache(maxsize=1)
def _experts():
    """The framework's handle, which a program keeps."""
    import error_bounded_lossy_gb300 as ebc
    return ebc.Experts(0)


# ---- the cases ----
def listed():
    return [
        # one token of a decode step: latency only; sigmoid scores, a bias for balance, choices from four of eight groups
        dict(name="route one token", op="route", tokens=1, experts=256, top=8, score="sigmoid", bias=True, groups=8, keep=4, best=2,
             renorm=True, scale=2.5, type="f32", masked=0.0, grad=False),
        # a training batch of the repository's batch size, same router, with the gradient
        dict(name="route training batch", op="route", tokens=8192, experts=256, top=8, score="sigmoid", bias=True, groups=8, keep=4, best=2,
             renorm=True, scale=2.5, type="f32", masked=0.0, grad=True),
        # few experts, 16-bit scores with many ties, padding tokens and experts that are masked out, weights as the softmax has them
        dict(name="route odd bf16", op="route", tokens=1531, experts=10, top=2, score="softmax", bias=False, groups=1, keep=1, best=1,
             renorm=False, scale=1.0, type="bf16", masked=0.1, grad=True),
        # one token of a decode step, ahead of the experts: latency only
        dict(name="norm one token", op="norm", rows=1, width=4096, type="bf16", residual=True, bits=8, grad=False),
        # a training batch, both directions
        dict(name="norm training batch", op="norm", rows=8192, width=4096, type="bf16", residual=True, bits=16, grad=True),
        # rows that are not aligned to any vector, no residual
        dict(name="norm odd fp32", op="norm", rows=1531, width=1001, type="f32", residual=False, bits=32, grad=True),
        # prefill: 16-bit rows for the router and 8-bit rows for the experts in one pass
        dict(name="norm prefill", op="norm", rows=16384, width=4096, type="bf16", residual=True, bits=8, grad=False),
        # a decode step of a few tokens: the touched experts' weights are streamed once
        dict(name="product decode", op="product", rows=16, experts=32, outs=4096, width=2048, type="bf16"),
        # ragged segments, no size a multiple of a tile or of a scale block
        dict(name="product odd", op="product", rows=1531, experts=10, outs=1003, width=1001, type="f16"),
        # prefill: arithmetic counts
        dict(name="product prefill", op="product", rows=16384, experts=32, outs=4096, width=4096, type="bf16"),
        # the whole serving step, one token
        dict(name="layer one token", op="layer", tokens=1, experts=64, top=8, outs=2048, width=2048, score="sigmoid", bias=True, groups=8,
             keep=4, best=2, renorm=True, scale=2.5, type="bf16", masked=0.0),
        # the whole serving step, a prefill batch with padding
        dict(name="layer prefill", op="layer", tokens=4096, experts=32, top=4, outs=2048, width=2048, score="softmax", bias=False, groups=1,
             keep=1, best=1, renorm=True, scale=1.0, type="bf16", masked=0.05),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _router(rng, most):
    """A router's settings: groups of equal size, enough kept experts for the choices."""
    groups = rng.choice([1, 1, 1, 2, 4, 8])
    experts = groups * _log(rng, 2, most // groups)
    keep = rng.randint(1, groups)
    top = rng.randint(1, min(16, keep * (experts // groups)))
    return dict(experts=experts, top=top, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                keep=keep, best=rng.choice([1, 2]), renorm=top > 1 and rng.random() < 0.7,   # (a single choice's share is 1, whatever its score)
                scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.0, 0.1]))


def draw(rng):
    op = rng.choice(["route", "norm", "product", "layer"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "route":
        return dict(op=op, tokens=_log(rng, 1, 8192), type=kind, grad=rng.random() < 0.6, **_router(rng, 512))
    if op == "norm":
        rows, width = _log(rng, 1, 16384), _log(rng, 32, 16384)
        while rows * width * BYTES[kind] > 8192 * 4096 * 2:
            rows = max(1, rows // 2)
        bits = rng.choice([8, 8 * BYTES[kind]])
        return dict(op=op, rows=rows, width=width, type=kind, residual=rng.random() < 0.7, bits=bits, grad=bits != 8 and rng.random() < 0.7)
    kind = rng.choice(["bf16", "f16"])
    outs, width = _log(rng, 8, 4096), _log(rng, 32, 4096)
    if op == "product":
        return dict(op=op, rows=_log(rng, 1, 16384), experts=_log(rng, 1, 32), outs=outs, width=width, type=kind)
    r = _router(rng, 32)
    r["top"] = min(r["top"], 8)   # (more than one choice still)
    return dict(op=op, tokens=_log(rng, 1, 2048), outs=outs, width=width, type=kind, **r)


# ---- inputs ----
def _activations(g, rows, width, kind):
    """Hidden states: normal values, with a few channels that are much larger."""
    x = torch.randn(rows, width, generator=g, device="cuda")
    loud = 1.0 + 20.0 * (torch.rand(width, generator=g, device="cuda") < 0.01)
    return (x * loud).to(TYPES[kind])


def _weights(g, experts, outs, width):
    """The experts' weights [experts, outs, width] in 8 bits, as a program keeps them: codes and scales."""
    codes = torch.empty(experts, outs, -(-width // 32) * 32, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(experts, outs, -(-width // 512) * 16, dtype=torch.uint8, device="cuda")
    for e in range(experts):
        w = torch.randn(outs, width, generator=g, device="cuda") / math.sqrt(width)
        codes[e], scales[e, :, :-(-width // 32)] = _encode(w)
    return codes, scales


def _logits(g, case):
    """The router's scores: some experts are liked better than others; with `masked`, so many of them are masked out, and so
    many tokens (padding) have none left."""
    t, e = case["tokens"], case["experts"]
    l = torch.randn(t, e, generator=g, device="cuda") + 0.5 * torch.randn(e, generator=g, device="cuda")
    if case["masked"]:
        gone = torch.rand(t, e, generator=g, device="cuda") < case["masked"]
        gone |= torch.rand(t, 1, generator=g, device="cuda") < case["masked"] / 2
        l = torch.where(gone, -math.inf, l)
    return l.to(TYPES[case["type"] if case["op"] == "route" else "f32"])


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    op, kind = case["op"], case["type"]
    if op in ("route", "layer"):
        s["logits"] = _logits(g, case)
        # a bias as balancing leaves it, smaller than the scores' spread
        s["b"] = 0.05 * torch.randn(case["experts"], generator=g, device="cuda") if case["bias"] else None
        if case.get("grad"):
            s["dweights"] = torch.randn(case["tokens"], case["top"], generator=g, device="cuda")
    if op in ("norm", "layer"):
        rows = case["rows" if op == "norm" else "tokens"]
        s["x"] = _activations(g, rows, case["width"], kind)
        s["r"] = _activations(g, rows, case["width"], kind) if case.get("residual", True) else None
        s["gain"] = (1.0 + 0.1 * torch.randn(case["width"], generator=g, device="cuda")).to(TYPES[kind])
        if case.get("grad"):
            s["dy"] = torch.randn(rows, case["width"], generator=g, device="cuda").to(TYPES[kind])
            s["dh"] = torch.randn(rows, case["width"], generator=g, device="cuda").to(TYPES[kind]) if case["residual"] else None
            # the sum that the forward pass returned
            s["h"] = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(TYPES[kind])
    if op == "product":
        # rows of the experts in turn, as a plan leaves them: uneven segments, some of them empty
        share = torch.rand(case["experts"], generator=g, device="cuda") ** 2 + 1e-3
        pick = torch.multinomial(share, case["rows"], replacement=True, generator=g)
        s["offsets"] = torch.searchsorted(pick.sort().values, torch.arange(case["experts"] + 1, device="cuda")).to(torch.int32)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["x"] = _activations(g, case["rows"], case["width"], kind)
    if op == "layer":
        ids = _choose(s["logits"], s["b"], case)[0].reshape(-1)
        s["most"] = int(torch.bincount(ids[ids >= 0].long(), minlength=case["experts"]).max())
    if op in ("product", "layer"):
        s["codes"], s["scales"] = _weights(g, case["experts"], case["outs"], case["width"])
    return s


# ---- the plain forms: elementary torch operations in 32 bits, rounded once ----
def _choose(logits, bias, s):
    """Each token's experts (best first, ties to the lowest) and their weights.  In 64 bits: two experts' biased scores may be
    nearer to each other than 32 bits tell."""
    l = logits.double()
    if s["score"] == "softmax":
        top = l.amax(1, keepdim=True)
        p = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
        p = p / torch.where(top == -math.inf, 1.0, p.sum(1, keepdim=True))
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    c = p if bias is None else p + bias.double()
    c = torch.where(l == -math.inf, -math.inf, c)
    if s["groups"] > 1:
        each = c.view(c.shape[0], s["groups"], -1)
        best = torch.sort(each, dim=2, descending=True).values[..., :s["best"]]
        score = torch.where(best == -math.inf, 0.0, best).sum(2)
        score = torch.where(best[..., 0] == -math.inf, -math.inf, score)
        kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, kept, True)
        c = torch.where(keep[..., None], each, -math.inf).view(c.shape)
    order = torch.sort(c, dim=1, descending=True, stable=True)
    ids = order.indices[:, :s["top"]]
    none = order.values[:, :s["top"]] == -math.inf
    w = torch.where(none, 0.0, p.gather(1, ids))
    if s["renorm"]:
        w = w / torch.where(none[:, :1], 1.0, w.sum(1, keepdim=True))
    return torch.where(none, -1, ids).to(torch.int32), (w * s["scale"]).float()


def _choose_grad(dweights, logits, ids, s):
    """The gradient of the scores: of the chosen ones, and with a softmax that is not renormalised of all."""
    l, none = logits.float(), ids < 0
    at = ids.clamp(min=0).long()
    g = torch.where(none, 0.0, dweights) * s["scale"]
    if s["score"] == "softmax":
        top = l.amax(1, keepdim=True)
        p = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
        p = p / torch.where(top == -math.inf, 1.0, p.sum(1, keepdim=True))
        w, slope = torch.where(none, 0.0, p.gather(1, at)), 1.0
    else:
        w = torch.where(none, 0.0, torch.sigmoid(l.gather(1, at)))
        slope = torch.where(none, 0.0, torch.sigmoid(-l.gather(1, at)))
    if s["renorm"]:
        w = w / torch.where(none[:, :1], 1.0, w.sum(1, keepdim=True))
        d = w * (g - (w * g).sum(1, keepdim=True)) * slope
    else:
        d = w * g * slope
    out = torch.zeros_like(l).scatter_add_(1, at, d)
    if s["score"] == "softmax" and not s["renorm"]:
        out = out - p * d.sum(1, keepdim=True)
    return out.to(logits.dtype)


def _norm(x, r, gain):
    """The sum of both inputs, and its root-mean-square norm times the gain."""
    h = x.float() if r is None else x.float() + r.float()
    return h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * gain.float(), h


def _norm_grad(dy, h, gain, dh):
    h, dy = h.float(), dy.float()
    scale = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    unit, g = h * scale, dy * gain.float()
    dx = scale * (g - unit * (g * unit).mean(1, keepdim=True))
    return dx if dh is None else dx + dh.float(), (dy * unit).sum(0)


def _encode(x):
    """E4M3 codes and E8M0 scales of rows [n, k] in 32 bits, filled up with zeros to whole blocks of 32."""
    pad = -x.shape[1] % 32
    blocks = (torch.nn.functional.pad(x.float(), (0, pad)) if pad else x.float()).view(x.shape[0], -1, 32)
    top = blocks.abs().amax(2).view(torch.int32)
    scale = ((top >> 23) - 8 + ((top & 0x7FFFFF) > 0x600000).int()).clamp(0, 254)   # amax <= 448 * 2^(scale - 127)
    v = blocks * ((254 - scale) << 23).view(torch.float32)[..., None]
    return v.to(torch.float8_e4m3fn).view(torch.uint8).view(x.shape[0], -1), scale.to(torch.uint8)


def _decode(codes, scales):
    """The values of codes [n, k] and scales [n, >= k / 32]."""
    v = codes.view(torch.float8_e4m3fn).float().view(codes.shape[0], -1, 32)
    e = scales[:, :v.shape[1]].int()
    unit = torch.where(e == 0, 2.0 ** -127, (e << 23).view(torch.float32))
    return (v * unit[..., None]).view(codes.shape)


def _rounded(x):
    """Rows through 8 bits and back."""
    return _decode(*_encode(x))[:, :x.shape[1]]


def _product(x, codes, scales, offsets, most):
    """Each row times its expert's weights: the segments padded to the longest, one batched product."""
    e, n, k = codes.shape
    w = _decode(codes.view(e * n, k), scales.view(e * n, -1)).view(e, n, k)[..., :x.shape[1]]
    at = torch.arange(x.shape[0], device=x.device)
    mine = torch.searchsorted(offsets[1:], at, right=True).clamp(max=e - 1)
    inside = (at - offsets[mine]).clamp(max=max(most, 1) - 1)
    full = torch.zeros(e, max(most, 1), x.shape[1], device=x.device)
    live = at < offsets[-1]
    full[mine[live], inside[live]] = x[live]
    ys = torch.matmul(full, w.transpose(1, 2))[mine, inside]
    return torch.where(live[:, None], ys, 0.0)


def _run_plain(s):
    op, kind = s["op"], TYPES[s["type"]]
    if op == "route":
        ids, weights = _choose(s["logits"], s["b"], s)
        out = {"ids": ids, "weights": weights}
        if s["grad"]:
            out["dlogits"] = _choose_grad(s["dweights"], s["logits"], ids, s)
        return out
    if op == "norm":
        y, h = _norm(s["x"], s["r"], s["gain"])
        out = {"y": y.to(kind)}
        if s["residual"]:
            out["h"] = h.to(kind)
        if s["bits"] == 8:
            out["values"] = _rounded(y).to(torch.bfloat16)
        if s["grad"]:
            dx, dgain = _norm_grad(s["dy"], s["h"], s["gain"], s["dh"])
            out["dx"], out["dgain"] = dx.to(kind), dgain.to(kind)
        return out
    if op == "product":
        return {"ys": _product(_rounded(s["x"]), s["codes"], s["scales"], s["offsets"], s["most"]).to(kind)}
    y, h = _norm(s["x"], s["r"], s["gain"])
    ids, weights = _choose(s["logits"], s["b"], s)
    flat = torch.where(ids < 0, s["experts"], ids).reshape(-1)
    order = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(order.values, torch.arange(s["experts"] + 1, dtype=flat.dtype, device=flat.device)).to(torch.int32)
    ys = _product(_rounded(y)[order.indices // s["top"]], s["codes"], s["scales"], offsets, s["most"])
    back = torch.empty_like(ys)
    back[order.indices] = ys
    y = (back.view(*ids.shape, -1) * weights[..., None]).sum(1)
    return {"ids": ids, "h": h.to(kind), "y": y.to(kind)}


# ---- the framework's calls ----
def _run_own(s):
    import error_bounded_lossy_gb300 as ebc
    op, ex, kind = s["op"], _experts(), TYPES[s["type"]]
    if op == "route":
        ids, weights = ex.route(s["logits"], s["top"], s["score"], s["b"], s["groups"], s["keep"], s["best"], s["renorm"], s["scale"])
        out = {"ids": ids, "weights": weights}
        if s["grad"]:
            out["dlogits"] = ex.route_grad(s["dweights"], s["logits"], ids, s["score"], s["renorm"], s["scale"])
        return out
    if op == "norm":
        if s["bits"] == 8:
            q, y, h = ex.norm_mx8(s["x"], s["gain"], s["r"], EPS, wide=True)
            out = {"y": y, "values": ex.dequantize(q, torch.bfloat16)}
        else:
            y, h = ex.norm(s["x"], s["gain"], s["r"], EPS)
            out = {"y": y}
        if s["residual"]:
            out["h"] = h
        if s["grad"]:
            out["dx"], out["dgain"] = ex.norm_grad(s["dy"], s["h"], s["gain"], s["dh"], EPS)
        return out
    w = ebc.Mx8(s["codes"], s["scales"], s["width"])
    if op == "product":
        return {"ys": ex.product(ex.quantize_mx8(s["x"]), w, s["offsets"], kind)}
    q, _, h = ex.norm_mx8(s["x"], s["gain"], s["r"], EPS)
    ids, weights = ex.route(s["logits"], s["top"], s["score"], s["b"], s["groups"], s["keep"], s["best"], s["renorm"], s["scale"])
    plan = ex.plan(ids, s["experts"])
    # (in 32 bits until the weighted sum is rounded)
    ys = ex.product(ex.dispatch(q, plan), w, plan.offsets, torch.float32)
    return {"ids": ids, "h": h, "y": ex.combine(ys, weights, plan).to(kind)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ----
def _touched(experts, rows):
    """Experts that so many rows reach when spread evenly."""
    return experts * (1.0 - (1.0 - 1.0 / experts) ** rows)


def work(case):
    b, op = BYTES[case["type"]], case["op"]
    if op == "route":
        t, e, k, grad = case["tokens"], case["experts"], case["top"], case["grad"]
        return {"bytes": t * e * b + 4 * e * case["bias"] + 8 * t * k + grad * (2 * t * e * b + 8 * t * k), "flops": t * e * (4 + 4 * grad)}
    if op == "norm":
        n, more = case["rows"] * case["width"], 2 * case["residual"]
        total = n * b * (2 + more) + case["width"] * b
        if case["bits"] == 8:
            total += 2 * n * MX8 + 2 * n   # codes and scales written and read back, 16-bit values written
        if case["grad"]:
            total += n * b * (3 + case["residual"]) + 2 * case["width"] * b
        return {"bytes": total, "flops": n * (4 + 10 * case["grad"])}
    o, h = case["outs"], case["width"]
    if op == "product":
        n = case["rows"]
        return {"bytes": n * h * b + (2 * n + _touched(case["experts"], n) * o) * h * MX8 + n * o * b, "flops": 2 * n * o * h}
    t, n = case["tokens"], case["tokens"] * case["top"]
    live = n * (1.0 - case["masked"] / 2)
    return {"bytes": 4 * t * case["experts"] + 24 * n + 3 * t * h * b + (2 * t + 2 * live + _touched(case["experts"], live) * o) * h * MX8
            + (2 * live + t) * o * b, "flops": 2 * live * o * h}


# ---- the definitions in 64 bits ----
def _route64(s):
    """Of each token: its experts, one after the other the best that is left, and their weights without the scale."""
    l = s["logits"].double().cpu().numpy()
    t, e = l.shape
    dead = np.isneginf(l)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if s["score"] == "softmax":
            z = np.exp(l - np.where(dead.all(1), 0.0, l.max(1))[:, None])
            p = z / np.maximum(z.sum(1), 1e-300)[:, None]
        else:
            p = 0.5 * (1.0 + np.tanh(0.5 * l))
            p = np.where(l < -30, np.exp(l), p)
    c = np.where(dead, -np.inf, p + (0.0 if s["b"] is None else s["b"].double().cpu().numpy()))
    if s["groups"] > 1:
        size = e // s["groups"]
        total = np.full((t, s["groups"]), -np.inf)
        for j in range(s["groups"]):
            part = c[:, j * size:(j + 1) * size].copy()
            for i in range(min(s["best"], size)):
                at = part.argmax(1)
                v = part[np.arange(t), at]
                total[:, j] = np.where(np.isneginf(v), total[:, j], np.where(np.isneginf(total[:, j]), 0.0, total[:, j]) + v)
                part[np.arange(t), at] = -np.inf
        keep = np.zeros((t, s["groups"]), bool)
        for i in range(s["keep"]):
            at = total.argmax(1)
            keep[np.arange(t), at] = True
            total[np.arange(t), at] = -np.inf
        c = np.where(np.repeat(keep, size, 1), c, -np.inf)
    ids, w = np.full((t, s["top"]), -1), np.zeros((t, s["top"]))
    for j in range(s["top"]):
        at = c.argmax(1)
        good = ~np.isneginf(c[np.arange(t), at])
        ids[good, j], w[good, j] = at[good], p[np.arange(t), at][good]
        c[np.arange(t), at] = -np.inf
    if s["renorm"]:
        w = w / np.where(ids[:, 0] < 0, 1.0, w.sum(1))[:, None]
    return p, ids, w


def _route_grad64(s, p, ids, w):
    """dw_j / dl_i summed over j, from the weights' own derivatives."""
    g = s["dweights"].double().cpu().numpy() * s["scale"]
    d = np.zeros_like(p)
    rows = np.arange(len(p))
    total = np.where(ids >= 0, w * g, 0.0).sum(1)   # sum over j of g_j w_j
    for j in range(s["top"]):
        live, at = ids[:, j] >= 0, np.maximum(ids[:, j], 0)
        pj = p[rows, at]
        if s["renorm"]:     # dw_j = w_j (dlog s_j - sum_i w_i dlog s_i), dlog s = 1 - s for sigmoids, 1 for a softmax's numerators
            each = w[:, j] * (g[:, j] - total) * (1.0 - pj if s["score"] == "sigmoid" else 1.0)
        else:               # dw_j = w_j (1 - s_j) for sigmoids, w_j ([i = j] - p_i) for a softmax
            each = w[:, j] * g[:, j] * (1.0 - pj if s["score"] == "sigmoid" else 1.0)
        d[rows[live], at[live]] += each[live]
    if s["score"] == "softmax" and not s["renorm"]:
        d -= p * total[:, None]
    return d


def _power(e):
    """2^e in 64 bits, by its bits (exp2 may be an ulp off)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _nearest(x):
    """Rows through 8 bits in 64 bits: the least power of two X with max <= 448 X in each block, then the nearest value with
    three bits of fraction, down to steps of 2^-9, ties to even."""
    n, k = x.shape
    full = torch.zeros(n, -(-k // 32) * 32, dtype=torch.float64, device=x.device)
    full[:, :k] = x.double()
    blocks = full.view(n, -1, 32)
    m, e = torch.frexp(blocks.abs().amax(2, keepdim=True) / 448.0)
    unit = _power(torch.where(m == 0.5, e - 1, e).clamp(min=-127))
    v = blocks / unit
    step = _power(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return (torch.round(v / step) * step * unit).reshape(n, -1)[:, :k]


def _values64(codes, scales, k):
    c = torch.arange(256, device=codes.device, dtype=torch.float64)
    field, frac = torch.floor(c / 8) % 16, c % 8
    table = torch.where(field == 0, frac * 2.0 ** -9, (8 + frac) * _power(field - 10)) * torch.where(c >= 128, -1.0, 1.0)
    unit = _power(scales.int() - 127)
    return (table[codes.long()] * unit.repeat_interleave(32, -1)[..., :codes.shape[-1]])[..., :k]


def _norm64(s):
    h = s["x"].double()
    if s["r"] is not None:
        h = h + s["r"].double()
    rms = (torch.linalg.vecdot(h, h) / h.shape[1] + EPS).sqrt()
    return h / rms[:, None] * s["gain"].double(), h


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        p, ids, w = _route64(s)
        out = {"ids": None, "weights": torch.from_numpy(w * s["scale"]).cuda()}
        if case["grad"]:
            out["dlogits"] = torch.from_numpy(_route_grad64(s, p, ids, w)).cuda()
        return out
    if op == "norm":
        y, h = _norm64(s)
        out = {"y": y}
        if case["residual"]:
            out["h"] = h
        if case["bits"] == 8:
            out["values"] = _nearest(y)
        if case["grad"]:
            h, dy = s["h"].double(), s["dy"].double()
            ms = torch.linalg.vecdot(h, h)[:, None] / h.shape[1] + EPS
            inner = torch.linalg.vecdot(dy * s["gain"].double(), h)[:, None] / h.shape[1]
            out["dx"] = (dy * s["gain"].double() - h * inner / ms) / ms.sqrt() + (0.0 if s["dh"] is None else s["dh"].double())
            out["dgain"] = torch.einsum("nk,nk->k", dy, h / ms.sqrt())
        return out
    if op == "product":
        cut, x = s["offsets"].tolist(), _nearest(s["x"])
        ys = torch.zeros(case["rows"], case["outs"], dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            if cut[e + 1] > cut[e]:
                ys[cut[e]:cut[e + 1]] = x[cut[e]:cut[e + 1]] @ _values64(s["codes"][e], s["scales"][e], case["width"]).T
        return {"ys": ys}
    y, h = _norm64(s)
    p, ids, w = _route64(s)
    x, out = _nearest(y), torch.zeros(case["tokens"], case["outs"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        token, j = np.nonzero(ids == e)
        if len(token):
            at = torch.from_numpy(token).cuda()
            rows = x[at] @ _values64(s["codes"][e], s["scales"][e], case["width"]).T
            out.index_add_(0, at, rows * torch.from_numpy(w[token, j] * s["scale"]).cuda()[:, None])
    return {"ids": None, "h": h, "y": out}
