"""dispatch and combine recorded for gradients, against the definition's recorded
gradients in 64 bits.

Values are multiples of 1/8 below 4, so that products of three of them are
multiples of 1/512 below 64; sums of less than 2^9 of those are exact in 24
bits, whatever their order, and results are compared for equality."""
import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import error_bounded_lossy_gb300 as ebc

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(scope="module")
def ex():
    e = ebc.Experts(0)
    yield e
    e.check()
    e.close()


def grid(g, *shape):
    return torch.randint(-31, 32, shape, generator=g, device="cuda").float() / 8


def batch(tokens, top, experts, width, drop, seed):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, experts, (tokens, top))
    ids[rng.random(ids.shape) < drop] = -1
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.from_numpy(ids).cuda(), grid(g, tokens, width), grid(g, tokens, top), grid(g, tokens * top, width), grid(g, tokens, width)


def defined(x, w, scale, plan):
    """sum over j of w[t, j] * (x[t] * scale[place[t, j]]) over the kept choices, in 64 bits."""
    place = plan.place.long()
    kept = (place >= 0)[..., None]
    rows = x[:, None, :] * scale[place.clamp(min=0)]
    return torch.where(kept, w[..., None] * rows, 0.0).sum(1)


@pytest.mark.parametrize("tokens,top,experts,width,drop", [(1, 1, 1, 1, 0.0), (1, 8, 64, 33, 0.0), (37, 3, 5, 130, 0.3), (6, 2, 3, 8, 1.0), (0, 2, 3, 8, 0.0)])
@pytest.mark.parametrize("side", [False, True])
def test_a_layer_is_recorded(ex, tokens, top, experts, width, drop, side):
    ids, x0, w0, scale, dy = batch(tokens, top, experts, width, drop, tokens + width)
    plan = ex.plan(ids, experts)
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    x, w = x0.clone().requires_grad_(), w0.clone().requires_grad_()
    torch.cuda.synchronize()
    xs = ex.dispatch(x, plan, stream=stream)
    with torch.cuda.stream(stream):
        rows = xs * scale
    y = ex.combine(rows, w, plan, stream=stream)
    assert xs.requires_grad and y.requires_grad
    torch.cuda.synchronize()
    y.backward(dy)
    torch.cuda.synchronize()
    x64, w64 = x0.double().requires_grad_(), w0.double().requires_grad_()
    y64 = defined(x64, w64, scale.double(), plan)
    y64.backward(dy.double())
    assert torch.equal(y.double(), y64) and torch.equal(x.grad.double(), x64.grad) and torch.equal(w.grad.double(), w64.grad)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_the_recorded_gradients_are_the_calls(ex, dtype):
    ids, x0, w0, _, dy = batch(50, 4, 7, 96, 0.2, 3)
    plan = ex.plan(ids, 7)
    x = x0.to(dtype).requires_grad_()
    dxs = torch.randn(200, 96, device="cuda").to(dtype)
    ex.dispatch(x, plan).backward(dxs)
    assert torch.equal(x.grad, ex.dispatch_grad(dxs, plan))
    ys, w = dxs.clone().requires_grad_(), w0.clone().requires_grad_()
    dy = dy.to(dtype)
    ex.combine(ys, w, plan).backward(dy)
    dys, dw = ex.combine_grad(dy, ys, w, plan)
    assert torch.equal(ys.grad, dys) and torch.equal(w.grad, dw)
    ys.grad = None
    ex.dispatch_grad(ys, plan).backward(dy)
    assert torch.equal(ys.grad, ex.dispatch(dy, plan))


def test_gradients_of_any_strides(ex):
    """A sum's gradient is one value expanded; a transposed use gives transposed rows."""
    ids, x0, w0, _, _ = batch(20, 2, 3, 24, 0.2, 4)
    plan = ex.plan(ids, 3)
    x, ys, w = x0.clone().requires_grad_(), torch.ones(40, 24, device="cuda", requires_grad=True), w0.clone().requires_grad_()
    ex.dispatch(x, plan).sum().backward()
    assert torch.equal(x.grad, (plan.place >= 0).sum(1, keepdim=True).float().expand(20, 24))
    ex.combine(ys, w, plan).sum().backward()
    assert torch.equal(w.grad, torch.where(plan.place >= 0, 24.0, 0.0))
    x.grad = None
    t = torch.randint(-4, 5, (24, 40), device="cuda").float()
    (ex.dispatch(x, plan).t() * t).sum().backward()
    assert torch.equal(x.grad, ex.dispatch_grad(t.t().contiguous(), plan))


def test_only_what_is_asked_for_is_recorded(ex):
    ids, x0, w0, _, dy = batch(9, 2, 3, 16, 0.2, 5)
    plan = ex.plan(ids, 3)
    x = x0.clone().requires_grad_()
    with torch.no_grad():
        assert not ex.dispatch(x, plan).requires_grad
    assert not ex.dispatch(x0, plan).requires_grad
    ys = ex.dispatch(x0, plan)
    w = w0.clone().requires_grad_()
    y = ex.combine(ys, w, plan)
    y.backward(dy)
    assert torch.equal(w.grad, ex.combine_grad(dy, ys, w0, plan)[1])
    assert not any(t.requires_grad for t in ex.combine_grad(dy, ys, w, plan))
    # 4 bits: integers, as from any rounding
    assert not ex.dequantize(ex.quantize(x)).requires_grad
    ids_w = torch.randn(9, 2, device="cuda", requires_grad=True)
    assert ex.combine(ys, ids_w, plan).requires_grad


def test_second_derivatives(ex):
    """dispatch is linear, so its gradient is recorded in turn; combine's gradients refuse."""
    ids, x0, w0, _, dy = batch(9, 2, 3, 16, 0.2, 6)
    plan = ex.plan(ids, 3)
    x = x0.clone().requires_grad_()
    (dx,) = torch.autograd.grad((ex.dispatch(x, plan) ** 2).sum() / 2, x, create_graph=True)
    v = torch.randint(-4, 5, x.shape, device="cuda").float()
    (hv,) = torch.autograd.grad((dx * v).sum(), x)
    assert torch.equal(hv, (plan.place >= 0).sum(1, keepdim=True) * v)
    ys, w = torch.ones(18, 16, device="cuda", requires_grad=True), w0.clone().requires_grad_()
    (dw,) = torch.autograd.grad((ex.combine(ys, w, plan) ** 2).sum(), w, create_graph=True)
    with pytest.raises(RuntimeError):
        dw.sum().backward()


def test_forward_mode_is_refused(ex):
    ids, x0, w0, _, dy = batch(9, 2, 3, 16, 0.2, 7)
    plan = ex.plan(ids, 3)
    ys = ex.dispatch(x0, plan)
    with forward_ad.dual_level():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        for call in (lambda: ex.dispatch(dual(x0), plan), lambda: ex.combine(dual(ys), w0, plan),
                     lambda: ex.combine(ys, dual(w0), plan), lambda: ex.combine_grad(dual(dy), ys, w0, plan)):
            with pytest.raises(ValueError, match="forward"):
                call()


def test_a_gradient_after_the_operators_were_closed_is_refused():
    e = ebc.Experts(0)
    x = torch.randn(4, 8, device="cuda", requires_grad=True)
    xs = e.dispatch(x, e.plan(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 3))
    torch.cuda.synchronize()
    e.close()
    with pytest.raises(ValueError, match="closed"):
        xs.sum().backward()
