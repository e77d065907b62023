"""The expert-parallel and 4-bit calls on a machine without a GPU: declared and
exported, refusing what is wrong before any device work; the torch layer checks
its tensors."""
import os
import re

import pytest
import torch

import error_bounded_lossy_gb300 as ebc
from error_bounded_lossy_gb300 import build as ebc_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    ebc_build.build()
    return ebc.lib()


def test_a_null_context_is_refused():
    bad = ebc.EBC_ERR_INVALID_ARG
    assert ebc.ebc_moe_plan(None, None, 4, 0, 1, 1, None, None, None, None) == bad
    assert ebc.ebc_moe_dispatch(None, None, 8, 0, 0, 1, 8, None, None, 1, None, None) == bad
    assert ebc.ebc_moe_combine(None, None, 8, 0, 0, 1, 8, None, None, None, None) == bad
    assert ebc.ebc_moe_combine_grad(None, None, 8, None, 8, 0, 0, 1, 8, None, None, 1, None, None, None, None) == bad
    assert ebc.ebc_mx4_quantize(None, None, 8, 0, 0, 8, None, None, None) == bad
    assert ebc.ebc_mx4_dequantize(None, None, None, 0, 8, 0, None, None) == bad
    assert ebc.ebc_moe_dispatch_mx4(None, None, 8, 0, 0, 1, 8, None, None, 1, None, None, None) == bad
    assert ebc.ebc_mx4_product(None, None, None, 0, 8, None, None, 8, 1, None, 0, None, None) == bad


def test_the_torch_types_refuse_other_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ebc.Plan(i, i.view(2, 2), i)
    with pytest.raises(ValueError, match="offsets"):
        ebc.Plan(i, i, i)
    b = torch.zeros(3, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        ebc.Mx4(b, torch.zeros(3, 16, dtype=torch.uint8), 64)
    with pytest.raises(ValueError, match="do not hold"):
        ebc.Mx4(b, torch.zeros(3, 16, dtype=torch.uint8), 65)
    with pytest.raises(ValueError, match="do not hold"):
        ebc.Mx4(b, torch.zeros(4, 16, dtype=torch.uint8), 64)


def test_no_context_without_a_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    with pytest.raises(ebc.EbcError):
        ebc.Experts(0)


@pytest.mark.parametrize("name", ["ebc_experts.cu", "ebc_mx4.cu", "ebc_mx4_product.cu"])
def test_kernels_that_start_early_read_with_ordinary_loads(name):
    """Read-only loads are for memory that nobody writes while the kernel runs; these kernels start before their
    producers have ended."""
    text = open(os.path.join(ebc_build.CSRC, name)).read()
    assert "pdl_enter();" in text
    assert not re.findall(r"const\s+\w+\s*\*\s*__restrict__|__ldg|ld\.global\.nc", text)


def test_the_compiled_calls_are_kept_apart_by_torch_and_python(monkeypatch):
    names = {ebc_build.torch_module()}
    monkeypatch.setattr(torch, "__version__", "0.1")
    names.add(ebc_build.torch_module())
    config = ebc_build.sysconfig.get_config_var
    monkeypatch.setattr(ebc_build.sysconfig, "get_config_var", lambda k: "cpython-00-none" if k == "SOABI" else config(k))
    names.add(ebc_build.torch_module())
    assert len(names) == 3
