"""The rows' calls at the edges of what they accept, on the GPU against their definitions in 64 bits."""
import pytest
import torch

import rows_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 2.0 ** -24  # half a step of fp32


@pytest.mark.parametrize("p", [0.0, 0.1, 0.25, 0.4])
@pytest.mark.parametrize("kind", [0, 1], ids=["silu", "gelu"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("n,I", [(2048, 1024), (1500, 1001)])
def test_h_again_is_the_forward_h(mr, n, I, dtype, kind, p):
    """The gradient of w2 takes the h that the product took, bit for bit."""
    gen = torch.Generator(device="cuda").manual_seed(I)
    gu = torch.randn(n, 2 * I, generator=gen, device="cuda").to(dtype)
    gh = torch.randn(n, I, generator=gen, device="cuda").to(dtype)
    rng = torch.tensor([17, 3], device="cuda")
    h = mr.expert_act(gu, act=kind, p=p, rng=rng)
    assert torch.equal(mr.expert_act_bwd(gh, gu, act=kind, p=p, rng=rng)["h"], h)
