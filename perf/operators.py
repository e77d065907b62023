"""The expert-parallel operators' cases: tokens sorted by expert and back with
their gradients, 4-bit microscaled quantisation, and the experts' products on
4-bit operands.

A case's "op" is one of
  dispatch   plan of a batch's routing, then the tokens' rows sorted by expert
             (and, with grad, the gradient of the sorted rows brought back)
  combine    the experts' rows brought back and summed with the router's weights
             (and, with grad, the gradients of the rows and of the weights)
  quantize   rows quantised to 4 bits and read back
  product    rows quantised to 4 bits, times each row's expert's 4-bit weights
  experts    the serving path in one: plan, dispatch in 4 bits, product, combine
"""
import functools
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


@functools.lru_cache(maxsize=1)
def _experts():
    """The framework's handle, which a program keeps."""
    import error_bounded_lossy_gb300 as ebc
    return ebc.Experts(0)


# ---- the cases ----
def listed():
    return [
        # one token of a decode step: latency only
        dict(name="dispatch one token", op="dispatch", tokens=1, top=8, experts=64, width=2048, type="bf16", drop=0.0, grad=False),
        # a training batch of the repository's batch size, both directions
        dict(name="dispatch training batch", op="dispatch", tokens=8192, top=8, experts=64, width=4096, type="bf16", drop=0.0, grad=True),
        # an odd width (rows not aligned to any vector), padding tokens dropped
        dict(name="dispatch odd fp32", op="dispatch", tokens=1531, top=2, experts=10, width=1001, type="f32", drop=0.2, grad=True),
        # the way back of the training batch, and its gradients
        dict(name="combine training batch", op="combine", tokens=8192, top=8, experts=64, width=4096, type="bf16", drop=0.0, grad=True),
        # odd sizes, a capacity limit that dropped a third of the choices
        dict(name="combine odd fp16", op="combine", tokens=777, top=3, experts=13, width=1003, type="f16", drop=0.33, grad=True),
        # the repository's forward batch [8192, 26, 128], a fixed-rate alternative to its containers
        dict(name="quantize embeddings", op="quantize", rows=8192, width=3328, type="f32"),
        # the activations of a small serving batch
        dict(name="quantize small batch", op="quantize", rows=64, width=4096, type="bf16"),
        # a decode step of a few tokens: the touched experts' weights are streamed once
        dict(name="product decode", op="product", rows=16, experts=32, outs=4096, width=2048, type="bf16"),
        # ragged segments, neither size a multiple of a tile
        dict(name="product odd", op="product", rows=1531, experts=10, outs=1000, width=1056, type="f16"),
        # prefill: arithmetic counts
        dict(name="product prefill", op="product", rows=16384, experts=32, outs=4096, width=4096, type="bf16"),
        # the whole serving path, one token
        dict(name="experts one token", op="experts", tokens=1, top=8, experts=64, outs=2048, width=2048, type="bf16", drop=0.0),
        # the whole serving path, a prefill batch with padding
        dict(name="experts prefill", op="experts", tokens=4096, top=4, experts=32, outs=2048, width=2048, type="bf16", drop=0.05),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "quantize", "product", "experts"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize":
        rows, width = _log(rng, 1, 16384), _log(rng, 32, 8192)
        while rows * width > 8192 * 3328:
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, width=width, type=kind)
    if op in ("dispatch", "combine"):
        experts = _log(rng, 1, 256)
        top = rng.randint(1, min(8, experts))
        tokens, width = _log(rng, 1, 16384), _log(rng, 16, 8192)
        while tokens * top * width * BYTES[kind] > 8192 * 8 * 4096 * 2:
            tokens = max(1, tokens // 2)
        return dict(op=op, tokens=tokens, top=top, experts=experts, width=width, type=kind,
                    drop=rng.choice([0.0, 0.1, 0.5]), grad=rng.random() < 0.7)
    experts, outs = _log(rng, 1, 32), _log(rng, 8, 4096)
    width = 32 * _log(rng, 1, 128)
    kind = rng.choice(["bf16", "f16"])
    if op == "product":
        return dict(op=op, rows=_log(rng, 1, 16384), experts=experts, outs=outs, width=width, type=kind)
    top = rng.randint(1, min(8, experts))
    return dict(op=op, tokens=_log(rng, 1, 2048), top=top, experts=experts, outs=outs, width=width, type=kind,
                drop=rng.choice([0.0, 0.1, 0.5]))


# ---- inputs ----
def _route(g, tokens, top, experts, drop):
    """The router's choices of each token (distinct, skewed to some experts), their weights, and dropped choices (-1)."""
    logits = torch.randn(tokens, experts, generator=g, device="cuda") + 0.5 * torch.randn(experts, generator=g, device="cuda")
    p, ids = logits.softmax(1).topk(top, 1)
    weights = p / p.sum(1, keepdim=True)
    ids = ids.to(torch.int32)
    if drop:
        ids = torch.where(torch.rand(tokens, top, generator=g, device="cuda") < drop, -1, ids)
    return ids.contiguous(), weights.contiguous()


def _activations(g, rows, width, kind):
    """Hidden states: normal values, with a few channels that are much larger."""
    x = torch.randn(rows, width, generator=g, device="cuda")
    loud = 1.0 + 20.0 * (torch.rand(width, generator=g, device="cuda") < 0.01)
    return (x * loud).to(TYPES[kind])


def _weights(g, experts, outs, width):
    """The experts' weights [experts, outs, width] in 4 bits, as a program keeps them: codes and scales."""
    codes = torch.empty(experts, outs, width // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(experts, outs, -(-width // 512) * 16, dtype=torch.uint8, device="cuda")
    for e in range(experts):
        c, s = _encode(torch.randn(outs, width, generator=g, device="cuda") / math.sqrt(width))
        codes[e] = c[:, 0::2] | (c[:, 1::2] << 4)
        scales[e, :, :width // 32] = s
    return codes, scales


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "quantize":
        s["x"] = _activations(g, case["rows"], case["width"], case["type"])
        return s
    if op == "product":
        # rows of the experts in turn, as a plan leaves them: uneven segments, some of them empty
        share = torch.rand(case["experts"], generator=g, device="cuda") ** 2 + 1e-3
        pick = torch.multinomial(share, case["rows"], replacement=True, generator=g)
        s["offsets"] = torch.searchsorted(pick.sort().values, torch.arange(case["experts"] + 1, device="cuda")).to(torch.int32)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["x"] = _activations(g, case["rows"], case["width"], case["type"])
        s["codes"], s["scales"] = _weights(g, case["experts"], case["outs"], case["width"])
        return s
    s["ids"], s["weights"] = _route(g, case["tokens"], case["top"], case["experts"], case["drop"])
    n, width, kind = case["tokens"] * case["top"], case["width"], case["type"]
    if op == "dispatch":
        s["x"] = _activations(g, case["tokens"], width, kind)
        if case["grad"]:
            s["dxs"] = torch.randn(n, width, generator=g, device="cuda").to(TYPES[kind])
    elif op == "combine":
        s["ys"] = _activations(g, n, width, kind)
        # the plan that the dispatch of the same batch made
        s["rows"], s["place"], s["offsets"] = _plan(s["ids"], case["experts"])
        if case["grad"]:
            s["dy"] = torch.randn(case["tokens"], width, generator=g, device="cuda").to(TYPES[kind])
    else:
        s["x"] = _activations(g, case["tokens"], width, kind)
        s["codes"], s["scales"] = _weights(g, case["experts"], case["outs"], width)
        valid = s["ids"].reshape(-1)
        s["most"] = int(torch.bincount(valid[valid >= 0].long(), minlength=case["experts"]).max()) if n else 0
    return s


# ---- the plain forms: elementary torch operations in 32 bits, rounded once ----
def _plan(ids, experts):
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(order.values, torch.arange(experts + 1, dtype=key.dtype, device=key.device)).to(torch.int32)
    at = torch.arange(flat.numel(), device=flat.device)
    rows = torch.where(at < offsets[experts], order.indices, -1).to(torch.int32)
    place = torch.empty_like(rows).scatter_(0, order.indices, torch.where(at < offsets[experts], at, -1).to(torch.int32))
    return rows, place.view(ids.shape), offsets


def _dispatch(x, rows, top):
    return torch.where((rows >= 0)[:, None], x.float()[rows.clamp(min=0) // top], 0.0)


def _gather(ys, place, weights=None):
    """Sum over each token's choices of its rows, times their weights."""
    picked = torch.where((place >= 0)[..., None], ys.float()[place.clamp(min=0)], 0.0)
    return (picked if weights is None else picked * weights[..., None]).sum(1)


def _encode(x):
    """E2M1 codes and E8M0 scales of rows [n, k] in 32 bits, k a multiple of 32."""
    blocks = x.view(x.shape[0], -1, 32)
    top = blocks.abs().amax(2).view(torch.int32)
    scale = ((top >> 23) - 2 + ((top & 0x7FFFFF) > 0x400000).int()).clamp(0, 254)   # amax <= 6 * 2^(scale - 127)
    v = blocks.abs() * ((254 - scale) << 23).view(torch.float32)[..., None]
    code = ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0)
            + (blocks < 0).to(torch.uint8) * 8)
    return code.view(x.shape), scale.to(torch.uint8)


def _decode(code, scale):
    """The values of codes [n, k] (one a byte) and scales [n, >= k / 32]."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    v = table[(code & 7).int()] * (1.0 - 2.0 * (code >> 3).float())
    s = torch.exp2(scale[:, :code.shape[1] // 32].float() - 127.0)
    return (v.view(code.shape[0], -1, 32) * s[..., None]).view(code.shape)


def _rounded(x):
    """Rows through 4 bits and back, padded with zeros to whole blocks."""
    pad = -x.shape[1] % 32
    full = torch.nn.functional.pad(x.float(), (0, pad)) if pad else x.float()
    return _decode(*_encode(full))[:, :x.shape[1]]


def _unpacked(codes, scales):
    """The weights that codes [e, n, k / 2] and scales stand for."""
    e, n, half = codes.shape
    c = torch.stack((codes & 15, codes >> 4), 3).view(e * n, half * 2)
    return _decode(c, scales.view(e * n, -1)).view(e, n, half * 2)


def _product(x, w, offsets, most):
    """Each row times its expert's weights: the segments padded to the longest, one batched product."""
    at = torch.arange(x.shape[0], device=x.device)
    e = torch.searchsorted(offsets[1:], at, right=True).clamp(max=w.shape[0] - 1)
    inside = (at - offsets[e]).clamp(max=max(most, 1) - 1)
    full = torch.zeros(w.shape[0], max(most, 1), x.shape[1], device=x.device)
    live = at < offsets[-1]
    full[e[live], inside[live]] = x[live]
    ys = torch.matmul(full, w.transpose(1, 2))[e, inside]
    return torch.where(live[:, None], ys, 0.0)


def _run_plain(s):
    op = s["op"]
    kind = TYPES[s["type"]]
    if op == "dispatch":
        rows, place, offsets = _plan(s["ids"], s["experts"])
        out = {"rows": rows, "place": place, "offsets": offsets, "xs": _dispatch(s["x"], rows, s["top"]).to(kind)}
        if s["grad"]:
            out["dx"] = _gather(s["dxs"], place).to(kind)
        return out
    if op == "combine":
        out = {"y": _gather(s["ys"], s["place"], s["weights"]).to(kind)}
        if s["grad"]:
            w = torch.where(s["rows"] >= 0, s["weights"].reshape(-1)[s["rows"].clamp(min=0)], 0.0)
            out["dys"] = (_dispatch(s["dy"], s["rows"], s["top"]) * w[:, None]).to(kind)
            picked = torch.where((s["place"] >= 0)[..., None], s["ys"].float()[s["place"].clamp(min=0)], 0.0)
            out["dweights"] = (picked * s["dy"].float()[:, None, :]).sum(2)
        return out
    if op == "quantize":
        return {"values": _rounded(s["x"]).to(kind)}
    w = _unpacked(s["codes"], s["scales"])
    if op == "product":
        return {"ys": _product(_rounded(s["x"]), w, s["offsets"], s["most"]).to(kind)}
    rows, place, offsets = _plan(s["ids"], s["experts"])
    ys = _product(_dispatch(_rounded(s["x"]), rows, s["top"]), w, offsets, s["most"])
    return {"y": _gather(ys, place, s["weights"]).to(kind)}


# ---- the framework's calls ----
def _run_own(s):
    import error_bounded_lossy_gb300 as ebc
    op, ex, kind = s["op"], _experts(), TYPES[s["type"]]
    if op == "dispatch":
        plan = ex.plan(s["ids"], s["experts"])
        out = {"rows": plan.rows, "place": plan.place, "offsets": plan.offsets, "xs": ex.dispatch(s["x"], plan)}
        if s["grad"]:
            out["dx"] = ex.dispatch_grad(s["dxs"], plan)
        return out
    if op == "combine":
        plan = ebc.Plan(s["rows"], s["place"], s["offsets"])
        out = {"y": ex.combine(s["ys"], s["weights"], plan)}
        if s["grad"]:
            out["dys"], out["dweights"] = ex.combine_grad(s["dy"], s["ys"], s["weights"], plan)
        return out
    if op == "quantize":
        return {"values": ex.dequantize(ex.quantize(s["x"]), kind)}
    w = ebc.Mx4(s["codes"], s["scales"], s["width"])
    if op == "product":
        return {"ys": ex.product(ex.quantize(s["x"]), w, s["offsets"], kind)}
    plan = ex.plan(s["ids"], s["experts"])
    ys = ex.product(ex.dispatch_mx4(s["x"], plan), w, plan.offsets, kind)
    return {"y": ex.combine(ys, s["weights"], plan)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ----
def _touched(experts, rows):
    """Experts that so many rows reach when spread evenly."""
    return experts * (1.0 - (1.0 - 1.0 / experts) ** rows)


def work(case):
    b, op = BYTES[case["type"]], case["op"]
    if op == "quantize":
        n = case["rows"] * case["width"]
        return {"bytes": 2 * n * b + 2 * n * 17 / 32, "flops": 0}
    if op == "product":
        n, o, k = case["rows"], case["outs"], case["width"]
        return {"bytes": n * k * b + (2 * n + _touched(case["experts"], n) * o) * k * 17 / 32 + n * o * b, "flops": 2 * n * o * k}
    t, n, h = case["tokens"], case["tokens"] * case["top"], case["width"]
    live = n * (1.0 - case["drop"])
    if op == "dispatch":
        plan = 4 * n + 8 * n + 4 * (case["experts"] + 1)
        return {"bytes": plan + (t + n) * h * b + (live + t) * h * b * case["grad"], "flops": live * h * case["grad"]}
    if op == "combine":
        return {"bytes": 8 * n + (live + t) * h * b + ((t + live + n) * h * b + 4 * n) * case["grad"],
                "flops": 2 * live * h * (1 + 2 * case["grad"])}
    o = case["outs"]
    return {"bytes": 16 * n + t * h * b + (2 * live + _touched(case["experts"], live) * o) * h * 17 / 32 + (2 * live + t) * o * b,
            "flops": 2 * live * o * h}


# ---- the definitions in 64 bits ----
def _nearest(x):
    """Rows through 4 bits in 64 bits: the least power of two X with max <= 6 X in each block, then the nearest of the
    sixteen values, ties to the even code."""
    n, k = x.shape
    full = torch.zeros(n, -(-k // 32) * 32, dtype=torch.float64, device=x.device)
    full[:, :k] = x.double()
    blocks = full.view(n, -1, 32)
    m, e = torch.frexp(blocks.abs().amax(2, keepdim=True) / 6.0)
    unit = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e).clamp(min=-127))
    v = blocks / unit
    low = torch.floor(torch.log2(v.abs().clamp(min=1.0)))        # spacing: 1/2 below 2, 1 below 4, 2 from there
    step = torch.exp2(low - 1.0)
    return (torch.round(v / step) * step * unit).reshape(n, -1)[:, :k]


def _values64(codes, scales, k):
    table = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
    table = torch.from_numpy(table).to(codes.device)
    v = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    v[..., 0::2] = table[(codes % 16).long()]
    v[..., 1::2] = table[torch.div(codes, 16, rounding_mode="floor").long()]
    unit = torch.ldexp(torch.ones((), dtype=torch.float64, device=codes.device), scales[..., :k // 32].int() - 127)
    return v * unit.repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return {"values": _nearest(s["x"])}
    if op == "product":
        cut, x = s["offsets"].tolist(), _nearest(s["x"])
        ys = torch.zeros(case["rows"], case["outs"], dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            if cut[e + 1] > cut[e]:
                ys[cut[e]:cut[e + 1]] = x[cut[e]:cut[e + 1]] @ _values64(s["codes"][e], s["scales"][e], case["width"]).T
        return {"ys": ys}
    ids = s["ids"].cpu().numpy().reshape(-1)
    live = np.flatnonzero((ids >= 0) & (ids < case["experts"]))
    order = live[np.lexsort((live, ids[live]))]
    at = torch.from_numpy(order).cuda()          # slots by expert, then by place in the batch
    token, top, n = at // case["top"], case["top"], case["tokens"] * case["top"]
    if op == "dispatch":
        xs = torch.zeros(n, case["width"], dtype=torch.float64, device="cuda")
        xs[:len(order)] = s["x"].double()[token]
        out = {"rows": None, "place": None, "offsets": None, "xs": xs}
        if case["grad"]:
            out["dx"] = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda").index_add_(
                0, token, s["dxs"][:len(order)].double())
        return out
    w = s["weights"].double().reshape(-1)[at][:, None]
    if op == "combine":
        ys = s["ys"][:len(order)].double()
        out = {"y": torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda").index_add_(0, token, ys * w)}
        if case["grad"]:
            dy = s["dy"].double()[token]
            out["dys"] = torch.zeros(n, case["width"], dtype=torch.float64, device="cuda")
            out["dys"][:len(order)] = dy * w
            dw = torch.zeros(n, dtype=torch.float64, device="cuda")
            dw[at] = torch.linalg.vecdot(dy, ys)
            out["dweights"] = dw.view(case["tokens"], top)
        return out
    y, x = torch.zeros(case["tokens"], case["outs"], dtype=torch.float64, device="cuda"), _nearest(s["x"])
    mine = ids[order]
    for e in range(case["experts"]):
        here = torch.from_numpy(np.flatnonzero(mine == e)).cuda()
        if len(here):
            rows = x[token[here]] @ _values64(s["codes"][e], s["scales"][e], case["width"]).T
            y.index_add_(0, token[here], rows * w[here])
    return {"y": y}
