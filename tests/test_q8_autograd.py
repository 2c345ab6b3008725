"""Inputs of the 8-bit block products that autograd tracks, without a GPU: they
are refused while gradients are recorded, before anything else is looked at."""

import pytest
import torch

nsd = pytest.importorskip("newton_schulz_dmuon_amd")
from newton_schulz_dmuon_amd import _lib  # noqa: E402


def message(fn, *a, **kw):
    with pytest.raises(nsd.DmuonError) as e:
        fn(*a, **kw)
    assert e.value.status == _lib.ERR_INVALID_ARG
    return str(e.value)


def tracked(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, requires_grad=True)


CALLS = [lambda x: nsd.q8_quantize(x), lambda x: nsd.q8_quantize(x * 2),
         lambda x: nsd.q8_weight_grad(x, nsd.Q8Rows.empty(4, 256, "cpu")),
         lambda x: nsd.q8_quantize_weights([x * 2]), lambda x: nsd.q8_quantize_weights([x.detach(), x * 2])]


@pytest.mark.parametrize("call", CALLS)
def test_tracked_inputs_are_refused(call):
    x = tracked(4, 256)
    assert "gradient" in message(call, x)
    with torch.no_grad():
        assert "gradient" not in message(call, x)  # refused as a host tensor


def test_a_parameter_may_be_quantised():
    assert "gradient" not in message(nsd.q8_quantize_weights, [torch.nn.Parameter(torch.zeros(128, 256))])
    assert "gradient" not in message(nsd.q8_quantize, tracked(4, 256).detach())


def test_inside_an_autograd_function():
    """Neither its forward pass nor its backward pass records gradients."""
    seen = []

    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            seen.append(message(nsd.q8_quantize, x))
            return x.clone()

        @staticmethod
        def backward(ctx, dy):
            seen.append(message(nsd.q8_weight_grad, dy, nsd.Q8Rows.empty(4, 256, "cpu")))
            return dy

    x = tracked(4, 256)
    Layer.apply(x).sum().backward()
    assert len(seen) == 2 and not any("gradient" in s for s in seen)
