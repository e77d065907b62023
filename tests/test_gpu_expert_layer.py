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
