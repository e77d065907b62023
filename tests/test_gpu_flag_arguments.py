"""A flag that has no truth value (more numbers than one) is that value's own error, and the call is not made."""
import pytest
import torch

import error_bounded_lossy_gb300 as ebc

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def test_flags_without_a_truth_value():
    ex = ebc.Experts(0)
    l, w, x, gain = (torch.ones(*s, device="cuda") for s in ((3, 8), (3, 2), (3, 64), (64,)))
    ids, _ = ex.route(l, 2)
    both = torch.ones(2)
    for call in (lambda f: ex.route(l, 2, renormalize=f), lambda f: ex.route_grad(w, l, ids, renormalize=f),
                 lambda f: ex.norm_mx8(x, gain, wide=f), lambda f: ex.norm_mx8(x.view(3, 1, 64), gain, wide=f)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call(both)
        call(both[:1])
        call(None)
    ex.set_profiling(True)
    with pytest.raises(RuntimeError):
        ex.route(l, 2, renormalize=both)
    assert not ex.profile()
    ex.check()
    ex.close()
