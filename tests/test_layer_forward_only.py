"""The helpers of the layer behind the router have no backward pass: inputs that ask for a gradient are refused, on the
host before anything of the library is called."""
import pytest
import torch

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    from top_gating_expert_row_gb300 import build

    build.build()
    import top_gating_expert_row_gb300 as m

    return m


def _experts():
    return dict(x=torch.ones(4, 64).to(BF16), topk_idx=torch.zeros(4, 2, dtype=torch.int32), topk_w=torch.ones(4, 2),
                w13=torch.ones(3, 64, 64).to(BF16), w2=torch.ones(3, 64, 32).to(BF16))


def _layer():
    v = _experts()
    return dict(x=v["x"], logits=torch.ones(4, 3), topk=2, w13=v["w13"], w2=v["w2"], bias=torch.ones(3), score_fn=1)


def _adapter():
    return dict(x=torch.ones(4, 64).to(BF16), w=torch.ones(8, 64).to(BF16), a=torch.ones(2, 8, 64).to(BF16),
                b=torch.ones(2, 8, 8).to(BF16), adapter=torch.zeros(4, dtype=torch.int32), scale=torch.ones(2))


CASES = [("experts", _experts, n) for n in ("x", "topk_w", "w13", "w2")]
CASES += [("layer", _layer, n) for n in ("x", "logits", "w13", "w2", "bias")]
CASES += [("adapter_proj", _adapter, n) for n in ("x", "w", "a", "b", "scale")]


@pytest.mark.parametrize("helper,make,name", CASES, ids=["%s-%s" % (c[0], c[2]) for c in CASES])
def test_inputs_that_ask_for_a_gradient(lib, helper, make, name):
    kw = make()
    kw[name].requires_grad_()
    with pytest.raises(ValueError, match="no backward"):
        getattr(lib, helper)(**kw)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):  # as far as a host tensor comes
        getattr(lib, helper)(**kw)
