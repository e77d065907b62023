"""The example that runs the expert-parallel operators, the 4-bit products and
the codec together, on small sizes."""
import importlib.util
import os

import pytest
import torch

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("tokens,width,outs,experts,top,ranks", [(300, 256, 200, 8, 2, 4), (5, 128, 64, 6, 3, 2)])
def test_expert_layer(example, tokens, width, outs, experts, top, ranks):
    r = example.main(["--tokens", str(tokens), "--width", str(width), "--outs", str(outs), "--experts", str(experts),
                      "--top", str(top), "--ranks", str(ranks), "--bound", "0.01"])
    assert r["worst"] <= torch.tensor(0.01)
    assert 0 < r["sent_bytes"] < r["raw_bytes"]
    # 4-bit values are within a sixth of their magnitude or a twelfth of the block's largest on both sides; for normal
    # values that is about 0.1 of a row's norm, so the products are about 0.16 off, and far from unrelated
    assert r["off"] < 0.3
    assert r["y"].shape == (tokens, outs) and r["dx"].shape == (tokens, width) and r["dw"].shape == (tokens, top)
    assert all(bool(torch.isfinite(r[k].float()).all()) for k in ("y", "dx", "dw"))


def test_the_gradients_of_the_layer(example):
    """Against the layer's definition in 64 bits, the experts' weights as their 4 bits stand for them and the rows as
    they arrived.  In fp32: a product with the router's weight and a sum over outs (or over the choices) are within
    2^-23 a term of the sum of the magnitudes."""
    import error_bounded_lossy_gb300 as ebc
    tokens, width, outs, experts, top = 90, 64, 130, 6, 2
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(tokens, width, generator=g, device="cuda")
    gate = torch.randn(width, experts, generator=g, device="cuda") / width ** 0.5
    ex, codec = ebc.Experts(0), ebc.Codec(0)
    weights = ex.quantize(torch.randn(experts, outs, width, generator=g, device="cuda") / width ** 0.5)
    dy = torch.randn(tokens, outs, generator=g, device="cuda")
    y, parts = example.forward(ex, codec, x, gate, weights, top, 3, 0.01)
    dx, dw = example.backward(ex, dy, weights, parts)
    ex.check()
    ids, w = example.route(x, gate, top)
    w64, dy64, full = w.double(), dy.double(), ex.dequantize(weights).double()[ids]   # [tokens, top, outs, width]
    terms = lambda f: torch.einsum("tj,to,tjok->tk", f(w64), f(dy64), f(full))  # noqa: E731
    assert bool(((dx.double() - terms(lambda v: v)).abs() <= (outs + top + 2) * 2.0 ** -23 * terms(torch.abs)).all())
    ys = parts["ys"].double()[parts["plan"].place.long()]                             # [tokens, top, outs]
    dots = lambda f: torch.einsum("to,tjo->tj", f(dy64), f(ys))  # noqa: E731
    assert bool(((dw.double() - dots(lambda v: v)).abs() <= (outs + 1) * 2.0 ** -23 * dots(torch.abs)).all())
    # the same from the definition's own recorded gradients
    x64, p64 = x.double().requires_grad_(), w64.clone().requires_grad_()
    y64 = torch.einsum("tj,tjok,tk->to", p64, full, x64)
    y64.backward(dy64)
    assert float((dx.double() - x64.grad).norm() / x64.grad.norm()) < 1e-5
    # rows lose a bound of 0.01 and 4 bits on the way (about 0.1 of their norm), and so do the weights' gradients
    assert float((dw.double() - p64.grad).norm() / p64.grad.norm()) < 0.3
    ex.close()
    codec.close()
