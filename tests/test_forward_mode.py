"""Inputs of the block products that forward-mode differentiation tracks, without a
GPU: a tangent would leave without a word, so they are refused, before anything else
is looked at."""

import pytest
import torch
from torch.autograd import forward_ad

nsd = pytest.importorskip("newton_schulz_dmuon_amd")
from newton_schulz_dmuon_amd import _lib  # noqa: E402


def message(fn, *a, **kw):
    with pytest.raises(nsd.DmuonError) as e:
        fn(*a, **kw)
    assert e.value.status == _lib.ERR_INVALID_ARG
    return str(e.value)


def plain():
    return torch.zeros(4, 256, dtype=torch.bfloat16)


CALLS = {
    "q8_quantize": lambda x: nsd.q8_quantize(x),
    "q8_quantize_weights": lambda x: nsd.q8_quantize_weights([plain(), x]),
    "q8_weight_grad": lambda x: nsd.q8_weight_grad(x, nsd.Q8Rows.empty(4, 256, "cpu")),
    "q4_quantize": lambda x: nsd.q4_quantize(x),
    "q4_quantize_weights": lambda x: nsd.q4_quantize_weights([plain(), x]),
}


@pytest.mark.parametrize("name", CALLS)
def test_tangents_are_refused(name):
    call = CALLS[name]
    with forward_ad.dual_level():
        x = forward_ad.make_dual(plain(), torch.ones(4, 256, dtype=torch.bfloat16))
        assert "tangent" in message(call, x) and "tangent" in message(call, x * 2)
        with torch.no_grad():  # which forward mode does not heed
            assert "tangent" in message(call, x)
        # refused as host tensors, the level open
        assert "tangent" not in message(call, plain())
        assert "tangent" not in message(call, forward_ad.unpack_dual(x).primal)
        with torch.inference_mode():
            assert "tangent" not in message(call, x)
    assert "tangent" not in message(call, plain())


@pytest.mark.parametrize("name", CALLS)
def test_a_parameter_with_a_tangent_is_refused(name):
    p = torch.nn.Parameter(plain())
    with forward_ad.dual_level(), torch.no_grad():
        assert "tangent" in message(CALLS[name], forward_ad.make_dual(p, torch.ones_like(p)))


@pytest.mark.parametrize("name", CALLS)
def test_inside_an_autograd_function(name):
    """Which carries its tangents on itself."""
    seen = []

    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            seen.append(message(CALLS[name], x))
            return x.clone()

        @staticmethod
        def jvp(ctx, tangent):
            seen.append(message(CALLS[name], tangent))
            return tangent.clone()

    with forward_ad.dual_level():
        y = Layer.apply(forward_ad.make_dual(plain(), torch.ones(4, 256, dtype=torch.bfloat16)))
        assert forward_ad.unpack_dual(y).tangent is not None
    assert len(seen) == 2 and not any("tangent" in s for s in seen)


def test_under_a_functional_transform():
    def fn(x):
        assert "tangent" in message(nsd.q4_quantize, x)
        return x * 2

    torch.func.jvp(fn, (plain(),), (plain(),))
