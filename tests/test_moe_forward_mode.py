"""The routed-expert layer's operators under forward-mode differentiation, on the
CPU: the kernels' calls are replaced, so what is tested is which way a tensor
with a tangent takes.  None of the operators has a forward-mode derivative, and
none may answer as if it were zero."""

import pytest
import torch
from torch.autograd import forward_ad

import nvfp4_quantization_grouped_amd as mxq
from nvfp4_quantization_grouped_amd import moe


@pytest.fixture(autouse=True)
def without_kernels(monkeypatch):
    monkeypatch.setattr(moe, "_need_cuda", lambda *ts: ts[0].device)
    monkeypatch.setattr(moe, "_call", lambda *args: None)


def operators():
    plan = mxq.MoEPlan(torch.zeros(2, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32),
                       torch.zeros(8, dtype=torch.int32))
    x, y, w = torch.randn(4, 64), torch.randn(8, 64), torch.randn(4, 2)
    return {"route": (lambda t: mxq.moe_route(t, 2), x), "dispatch": (lambda t: mxq.moe_dispatch(t, plan), x),
            "combine, rows": (lambda t: mxq.moe_combine(t, w, plan), y),
            "combine, weights": (lambda t: mxq.moe_combine(y, t, plan), w),
            "swiglu": (lambda t: mxq.swiglu(t), x), "swiglu, whole": (lambda t: mxq.swiglu(t, checkpoint=None), x)}


@pytest.mark.parametrize("name", list(operators()))
@pytest.mark.parametrize("grad", [True, False])
def test_a_tangent_is_refused(name, grad):
    call, t = operators()[name]
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        with pytest.raises(NotImplementedError, match="forward mode"):
            call(forward_ad.make_dual(t, torch.ones_like(t)))
        call(t)                                           # an open level alone changes nothing
    call(t)


@pytest.mark.parametrize("activations", ["fp8", "mxfp4"])
def test_low_bit_activations_refuse_a_tangent(activations):
    x, w = torch.zeros(4, 512, dtype=torch.bfloat16), torch.zeros(4, 2)
    e = torch.zeros(4, 2, dtype=torch.int32)
    weights = (torch.zeros(1, 1, 1),) * 4
    with forward_ad.dual_level():
        for args in ((forward_ad.make_dual(x, x + 1), w), (x, forward_ad.make_dual(w, w + 1))):
            with pytest.raises(ValueError, match="no gradient"):
                mxq.mxfp4_moe(*args, e, *weights, activations=activations)
