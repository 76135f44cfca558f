"""Inputs with a forward-mode tangent: an operator's result drops it, and the operators say so as they do
of inputs that require grad (no GPU: the check itself)."""
import warnings

import pytest

torch = pytest.importorskip("torch")

import torch.autograd.forward_ad as forward_ad  # noqa: E402

from nearest_centroid_assignment_amd import experts, layers  # noqa: E402


def _say(name, module, *inputs):
    if module is layers:
        return layers._module().unrecorded(name, *inputs)
    return experts._module().unrecorded(name, *inputs)


@pytest.mark.parametrize("module,name", [(layers, "embed"), (experts, "linear")])
def test_a_tangent_is_not_dropped_silently(module, name):
    plain, leaf = torch.ones(3, 4), torch.ones(3, 4, requires_grad=True)
    said = f"{module.__name__.split('.')[-1]}.{name}.*not recorded"
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(torch.ones(3, 4), torch.ones(3, 4))
        for inputs in ((dual,), (plain, None, dual)):
            with pytest.warns(UserWarning, match=said + ".*tangent"):
                _say(name, module, *inputs)
            with torch.no_grad(), pytest.warns(UserWarning, match=said):  # no_grad keeps tangents
                _say(name, module, *inputs)
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with torch.inference_mode():  # which keeps none
                _say(name, module, dual)
            with forward_ad._set_fwd_grad_enabled(False):
                _say(name, module, dual)
            _say(name, module, forward_ad.unpack_dual(dual).primal, plain, None)
            with pytest.raises(UserWarning):
                _say(name, module, dual)
        with pytest.warns(UserWarning, match=said + ".*requires grad"):
            _say(name, module, leaf)
    with warnings.catch_warnings():  # a level that has ended leaves no tangent
        warnings.simplefilter("error")
        _say(name, module, dual, plain)
