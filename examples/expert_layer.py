"""A mixture-of-experts layer with experts on several ranks, the operators as
they are used together: the router, tokens sorted by expert, the rows of each rank as an
error-bounded container, the experts' products on the received rows in 4 bits,
and the weighted sum on the way back; then a training step's gradients.

The ranks are run one after the other on one GPU, each with its share of the
experts; what a container would be sent to is the next rank's codec.

    python examples/expert_layer.py [--tokens 2048] [--width 1024] [--outs 1024] [--experts 16] [--top 4]
                                    [--ranks 4] [--bound 0.01]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import error_bounded_lossy_gb300 as ebc  # noqa: E402


def route(x, gate, top):
    """The router's definition in torch's operations: each token's experts and their weights."""
    p, ids = (x.float() @ gate).softmax(1).topk(top, 1)
    return ids, (p / p.sum(1, keepdim=True)).contiguous()


def exchange(codec, rows, bound):
    """The rows of one rank through a container: (the rows as received, container bytes, largest error)."""
    if rows.shape[0] == 0:
        return rows, 0, 0.0
    d = 512
    while rows.shape[1] % d:
        d //= 2
    x = rows.view(rows.shape[0], -1, d)          # [rows, tables, d]: the codec's shape
    box, nbytes = codec.compress(x, [bound] * x.shape[1])
    codec.check()
    back = codec.decompress(box, int(nbytes.item()), *x.shape)
    codec.check()
    worst = float((back - x.float()).abs().max())
    return back.view(rows.shape).to(rows.dtype), int(nbytes.item()), worst


def forward(ex, codec, x, gate, weights, top, ranks, bound):
    """The layer's result, and what its parts were."""
    ids, w = ex.route(x.float() @ gate, top)
    n_experts = gate.shape[1]
    plan = ex.plan(ids, n_experts)
    xs = ex.dispatch(x, plan)
    cut = plan.offsets.tolist()                  # an all-to-all needs its counts on the host
    ys = torch.zeros(xs.shape[0], weights.shape[1], dtype=x.dtype, device=x.device)
    each, sent, worst = n_experts // ranks, 0, 0.0
    for r in range(ranks):
        at = slice(cut[r * each], cut[(r + 1) * each])
        got, nbytes, off = exchange(codec, xs[at], bound)
        sent, worst = sent + nbytes, max(worst, off)
        if got.shape[0]:
            mine = ebc.Mx4(weights.codes[r * each:(r + 1) * each], weights.scales[r * each:(r + 1) * each], weights.width)
            local = plan.offsets[r * each:(r + 1) * each + 1] - cut[r * each]
            ys[at] = ex.product(ex.quantize(got), mine, local.contiguous(), x.dtype)
    y = ex.combine(ys, w, plan)
    ex.check()
    return y, dict(plan=plan, w=w, xs=xs, ys=ys, raw_bytes=xs.numel() * xs.element_size(), sent_bytes=sent, worst=worst)


def backward(ex, dy, weights, parts):
    """The gradients of the layer's input rows and of the router's weights for the
    gradient dy, through the experts' weights as their 4 bits stand for them."""
    plan = parts["plan"]
    dys, dw = ex.combine_grad(dy, parts["ys"], parts["w"], plan)
    dxs = torch.zeros_like(parts["xs"])
    cut = plan.offsets.tolist()
    for e in range(plan.n_experts):
        if cut[e + 1] > cut[e]:
            w = ex.dequantize(ebc.Mx4(weights.codes[e], weights.scales[e], weights.width), dy.dtype)
            dxs[cut[e]:cut[e + 1]] = dys[cut[e]:cut[e + 1]] @ w
    return ex.dispatch_grad(dxs, plan), dw


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 2048), ("width", 1024), ("outs", 1024), ("experts", 16), ("top", 4), ("ranks", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--bound", type=float, default=0.01)
    a = ap.parse_args(argv)
    if a.experts % a.ranks:
        ap.error("the ranks must divide the experts")
    g = torch.Generator("cuda").manual_seed(0)
    x = torch.randn(a.tokens, a.width, generator=g, device="cuda").to(torch.bfloat16)
    gate = torch.randn(a.width, a.experts, generator=g, device="cuda") / a.width ** 0.5
    full = torch.randn(a.experts, a.outs, a.width, generator=g, device="cuda") / a.width ** 0.5
    ex, codec = ebc.Experts(0), ebc.Codec(0)
    weights = ex.quantize(full)
    y, parts = forward(ex, codec, x, gate, weights, a.top, a.ranks, a.bound)
    dx, dw = backward(ex, torch.randn(y.shape, generator=g, device="cuda").to(y.dtype), weights, parts)
    ex.check()
    # the same layer without any loss
    ids, w = route(x, gate, a.top)
    want = torch.zeros(a.tokens, a.outs, device="cuda")
    for j in range(a.top):
        for e in range(a.experts):
            hit = ids[:, j] == e
            want[hit] += w[hit, j:j + 1] * (x[hit].float() @ full[e].T)
    off = float((y.float() - want).norm() / want.norm())
    print(f"{a.tokens} tokens x {a.top} of {a.experts} experts on {a.ranks} ranks: {parts['raw_bytes']} bytes of rows sent as "
          f"{parts['sent_bytes']} ({parts['raw_bytes'] / parts['sent_bytes']:.2f}x, largest error {parts['worst']:.4f} "
          f"under a bound of {a.bound}); result {off:.3f} off the full-precision layer; gradients {tuple(dx.shape)}, "
          f"{tuple(dw.shape)}")
    ex.close()
    codec.close()
    return dict(parts, y=y, dx=dx, dw=dw, off=off, want=want)


if __name__ == "__main__":
    main()
