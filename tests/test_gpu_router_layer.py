"""The norm, the router, the plan, the 8-bit rows, the experts' products and the
weighted sum as a layer uses them: served, captured into a graph, on several
streams and threads at once, and trained."""
import threading

import numpy as np
import pytest
import torch

import error_bounded_lossy_gb300 as ebc

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

U = 2.0 ** -24
ROUTER = dict(score="sigmoid", groups=4, keep_groups=2, group_top=2, scale=2.5)


@pytest.fixture(scope="module")
def ex():
    e = ebc.Experts(0)
    yield e
    e.check()
    e.close()


def weights(ex, experts, outs, width, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return dict(
        gain=(1 + 0.2 * torch.randn(width, generator=g, device="cuda")),
        gate=torch.randn(width, experts, generator=g, device="cuda") / width ** 0.5,
        bias=0.1 * torch.randn(experts, generator=g, device="cuda"),
        w=ex.quantize_mx8(torch.randn(experts, outs, width, generator=g, device="cuda") / width ** 0.5))


def serve(ex, x, r, p, top, kind="mx8"):
    """One layer: everything that it made on the way."""
    q, y, h = ex.norm_mx8(x, p["gain"], r, wide=True)
    ids, w = ex.route(y.float() @ p["gate"], top, bias=p["bias"], **ROUTER)
    plan = ex.plan(ids, p["gate"].shape[1])
    ys = ex.product(ex.dispatch(q, plan), p["w"], plan.offsets, torch.float32)
    return dict(q=q, y=y, h=h, ids=ids, w=w, plan=plan, ys=ys, out=ex.combine(ys, w, plan))


@pytest.mark.parametrize("tokens", [1, 3, 130, 700])
@pytest.mark.parametrize("width,outs", [(256, 128), (250, 70)])
def test_a_layer_is_served(ex, tokens, width, outs):
    """Each token's sum over its experts of weight times product, in 64 bits from the rows and weights that the calls
    before it gave: width additions in 32 bits for a product, and 9 for the sum and the weights' products."""
    experts, top = 16, 4
    p = weights(ex, experts, outs, width, tokens)
    g = torch.Generator("cuda").manual_seed(width)
    x, r = (torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(2))
    s = serve(ex, x, r, p, top)
    ex.check()
    rows, full = ex.dequantize(s["q"]).double(), ex.dequantize(p["w"]).double()
    terms = lambda f: torch.einsum("tj,tjok,tk->to", f(s["w"].double()), f(full)[s["ids"].long()], f(rows))  # noqa: E731
    off = (s["out"].double() - terms(lambda v: v)).abs()
    assert bool((off <= 2 * (width + 9) * U * terms(torch.abs)).all())
    # what the router saw is what the norm gave, and each token has `top` experts of two groups
    assert bool((s["ids"] >= 0).all()) and bool(((s["ids"] // 4).sort(1).values.diff(dim=1) != 0).sum(1).le(1).all())
    assert torch.equal(s["plan"].offsets.diff(), torch.bincount(s["ids"].flatten(), minlength=experts).int())
    assert torch.equal(s["h"], ex.norm(x, p["gain"], r)[1])


def test_padding_tokens_take_no_part(ex):
    """Tokens whose scores are all masked out are dropped: no rows, a zero result, and a zero gradient."""
    p = weights(ex, 16, 64, 128, 0)
    x = torch.randn(50, 128, device="cuda")
    logits = torch.randn(50, 16, device="cuda")
    pad = torch.arange(50, device="cuda") % 3 == 0
    logits[pad] = -torch.inf
    ids, w = ex.route(logits, 4, bias=p["bias"], **ROUTER)
    plan = ex.plan(ids, 16)
    assert int(plan.offsets[-1]) == 4 * int((~pad).sum())
    q = ex.dispatch(ex.norm_mx8(x, p["gain"])[0], plan)
    out = ex.combine(ex.product(q, p["w"], plan.offsets, torch.float32), w, plan)
    assert not out[pad].any() and bool((out[~pad] != 0).any(1).all())
    d = ex.route_grad(torch.ones_like(w), logits, ids, "sigmoid", True, 2.5)
    assert not d[pad].any() and bool(torch.isfinite(d).all())
    ex.check()


def test_a_layer_in_a_graph_and_on_two_streams_at_once(ex):
    p = weights(ex, 16, 96, 320, 1)
    g = torch.Generator("cuda").manual_seed(3)
    batches = [tuple(torch.randn(n, 320, generator=g, device="cuda").bfloat16() for _ in range(2)) for n in (40, 40, 300)]
    want = [serve(ex, *b, p, 4)["out"] for b in batches]
    graph, given = torch.cuda.CUDAGraph(), [t.clone() for t in batches[0]]
    with torch.cuda.graph(graph):
        got = serve(ex, *given, p, 4)["out"]
    for i in (0, 1, 0):
        for t, b in zip(given, batches[i]):
            t.copy_(b)
        graph.replay()
        assert torch.equal(got, want[i])
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(20):
        outs = []
        for s, b in zip(streams, batches):
            with torch.cuda.stream(s):
                outs.append(serve(ex, *b, p, 4)["out"])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_two_threads_with_a_context_each():
    failed = []
    x, l = torch.randn(200, 520, device="cuda").bfloat16(), torch.randn(200, 64, device="cuda")
    gain = torch.ones(520, device="cuda")
    torch.cuda.synchronize()

    def work(k):
        e, s = ebc.Experts(0), torch.cuda.Stream()
        try:
            first = None
            for _ in range(200):
                with torch.cuda.stream(s):
                    q, y, h = e.norm_mx8(x, gain, x, wide=True)
                    ids, w = e.route(l, 6, "sigmoid", None, 8, 2 + k, 2)
                    got = (q.codes, q.scales, y, h, ids, w, e.norm_grad(x, h, gain)[1], e.route_grad(w, l, ids, "sigmoid"))
                s.synchronize()
                if first is None:
                    first = got
                if not all(torch.equal(a, b) for a, b in zip(first, got)):
                    failed.append(k)
            e.check()
        except Exception as err:   # noqa: BLE001
            failed.append(repr(err))
        e.close()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_a_layer_is_trained(ex, score, renormalize):
    """norm, route, dispatch and combine recorded together, with plain fp32 experts between them, against the
    definition's recorded gradients in 64 bits for the same choice.  A gradient is a sum of chains of some hundred
    fp32 operations whose terms may cancel to a tenth: 1e-4 of its norm covers 100 units of 2^-24 (6e-6) each."""
    tokens, width, experts, top, outs = 60, 96, 8, 3, 40
    g = torch.Generator("cuda").manual_seed(5)
    make = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x0, r0, gain0, gate0, w0 = make(tokens, width), make(tokens, width), 1 + 0.1 * make(width), make(width, experts) / 10, make(experts, outs, width) / 10
    dy, dh = make(tokens, outs), make(tokens, width)
    x, r, gain, gate, w = (t.clone().requires_grad_() for t in (x0, r0, gain0, gate0, w0))
    y, h = ex.norm(x, gain, r)
    ids, p = ex.route(y @ gate, top, score, renormalize=renormalize)
    plan = ex.plan(ids, experts)
    cut = plan.offsets.tolist()
    xs = ex.dispatch(y, plan)
    ys = torch.cat([xs[cut[e]:cut[e + 1]] @ w[e].T for e in range(experts)])
    out = ex.combine(ys, p, plan)
    torch.autograd.backward((out, h), (dy, dh))
    x64, r64, gain64, gate64, w64 = (t.double().clone().requires_grad_() for t in (x0, r0, gain0, gate0, w0))
    h64 = x64 + r64
    y64 = h64 / ((h64 * h64).mean(1, keepdim=True) + 1e-6).sqrt() * gain64
    l64 = y64 @ gate64
    s64 = (l64.softmax(1) if score == "softmax" else l64.sigmoid()).gather(1, ids.long())
    p64 = s64 / s64.sum(1, keepdim=True) if renormalize else s64
    out64 = torch.einsum("tj,tjok,tk->to", p64, w64[ids.long()], y64)
    torch.autograd.backward((out64, h64), (dy.double(), dh.double()))
    for a, b in ((out, out64), (x.grad, x64.grad), (r.grad, r64.grad), (gain.grad, gain64.grad), (gate.grad, gate64.grad), (w.grad, w64.grad)):
        assert float((a.detach().double() - b.detach()).norm() / b.detach().norm()) < 1e-4
    assert torch.equal(x.grad, r.grad)
    ex.check()


def test_a_training_pass_in_a_graph(ex):
    """Forward and backward captured together and replayed on other inputs: the bits of an eager pass.  (Outputs of
    eager passes over the same leaves are gone by then, as torch asks.)"""
    tokens, width, experts, top = 70, 200, 16, 4
    g = torch.Generator("cuda").manual_seed(9)
    make = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    leaves = [t.requires_grad_() for t in (make(tokens, width), make(tokens, width), 1 + 0.1 * make(width), make(width, experts) / 10)]
    inputs = [[make(tokens, width) for _ in range(4)] for _ in range(3)]   # x, residual, dy, dh
    bias = 0.1 * make(experts)

    def step(dy, dh):
        x, r, gain, gate = leaves
        y, h = ex.norm(x, gain, r)
        ids, p = ex.route(y @ gate, top, bias=bias, **ROUTER)
        plan = ex.plan(ids, experts)
        out = ex.combine(ex.dispatch(y, plan), p, plan)
        return torch.autograd.grad((out, h), leaves, (dy, dh))

    def eager(x, r, dy, dh):
        with torch.no_grad():
            leaves[0].copy_(x)
            leaves[1].copy_(r)
        return step(dy, dh)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [[t.clone() for t in eager(*i)] for i in inputs]
    torch.cuda.synchronize()
    graph, dy, dh = torch.cuda.CUDAGraph(), inputs[0][2].clone(), inputs[0][3].clone()
    with torch.cuda.graph(graph):
        got = step(dy, dh)
    for k in (1, 0, 2, 1):
        with torch.no_grad():
            for t, i in zip((leaves[0], leaves[1], dy, dh), inputs[k]):
                t.copy_(i)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want[k])), k
    ex.check()


def test_8_bit_rows_of_several_ranks_to_one_product(ex):
    """Pieces of several senders, each sorted by expert, are sorted together by a plan of one choice a row."""
    width, experts, outs = 200, 6, 40
    g = torch.Generator("cuda").manual_seed(7)
    w = ex.quantize_mx8(torch.randn(experts, outs, width, generator=g, device="cuda"))
    pieces, owners = [], []
    for r in range(3):
        plan = ex.plan(torch.randint(0, experts, (30 + r, 2), generator=g, device="cuda"), experts)
        pieces.append(ex.dispatch(ex.quantize_mx8(torch.randn(30 + r, width, generator=g, device="cuda")), plan))
        owners.append(torch.repeat_interleave(torch.arange(experts, device="cuda"), plan.offsets.diff()))
    got = ebc.Mx8(torch.cat([q.codes for q in pieces]), torch.cat([q.scales for q in pieces]), width)
    e = torch.cat(owners)
    plan = ex.plan(e[:, None], experts)
    back = ex.combine(ex.product(ex.dispatch(got, plan), w, plan.offsets, torch.float32), None, plan)
    rows, full = ex.dequantize(got).double(), ex.dequantize(w).double()[e]
    off = (back.double() - torch.einsum("rk,rok->ro", rows, full)).abs()
    assert bool((off <= 2 * (width + 1) * U * torch.einsum("rk,rok->ro", rows.abs(), full.abs())).all())
    ex.check()
