"""The helpers have no forward-mode derivative: dual tensors are refused, on the host before anything of the library is
called, instead of losing their tangents."""
import pytest
import torch
from torch.autograd import forward_ad

import test_abi_rows as rows
import test_layer_forward_only as layer
from test_abi_rows import lib  # noqa: F401  (the fixture)

CASES = [(h, lambda h=h: rows._args()[h], q) for h, q in rows.TENSORS if rows._args()[h][q].is_floating_point()]
CASES += layer.CASES
IDS = ["%s-%s" % (c[0], c[2]) for c in CASES]


@pytest.mark.parametrize("grad", [True, False], ids=["grad", "no_grad"])
@pytest.mark.parametrize("helper,make,name", CASES, ids=IDS)
def test_dual_inputs(lib, helper, make, name, grad):  # noqa: F811
    kw = make()
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        dual = {**kw, name: forward_ad.make_dual(kw[name], torch.ones_like(kw[name]))}
        with pytest.raises(ValueError, match="forward-mode"):
            getattr(lib, helper)(**dual)
        with pytest.raises(ValueError, match="CUDA device"):  # as far as a host tensor comes
            getattr(lib, helper)(**{**kw, name: dual[name].detach()})


@pytest.mark.parametrize("transform", [
    lambda f, x: torch.func.jvp(f, (x,), (x,)), lambda f, x: torch.func.jacfwd(f)(x)], ids=["jvp", "jacfwd"])
def test_transforms(lib, transform):  # noqa: F811
    with pytest.raises(ValueError, match="forward-mode"):
        transform(lambda x: lib.dropout(x, 0.0, None), torch.ones(4, 32))
