"""Sizes past what the tensor-core kernels count in 32 bits, on the host without a GPU: the workspace that a call asks
for shows which kernels it takes (the plain ones need the pairs' h alone)."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from top_gating_expert_row_gb300 import build

    build.build()
    import top_gating_expert_row_gb300 as m

    return m


H = I = 8
ROWS = 2 ** 30  # of the sorted layout: a grid's stride past them, or twice them, still fits an int


def experts_bytes(lib, T, E, topk):
    return lib.moe_experts_workspace_bytes(lib.mr_expert_params(T, H, I, E, topk, lib.MR_BF16, lib.MR_SILU))


@pytest.mark.parametrize("T,E,topk", [(ROWS + 1, 1, 1), (2 ** 31 - 2, 1, 1), (2 ** 31 - 2 ** 18, 4096, 1),
                                      (2 ** 28 + 1, 4, 4), (ROWS - 64, 4, 1), (2 ** 30 - 2 ** 12, 4096, 1)])
def test_rows_past_32_bits_take_the_plain_kernels(lib, T, E, topk):
    pairs = T * topk
    assert 0 < experts_bytes(lib, T, E, topk) <= pairs * I * 4 + 256
    if T * E > 2 ** 31 - 1:
        return  # the router refuses such logits
    routed = lib.moe_layer_workspace_bytes(lib.RouterParams(T, E, topk), H, I)
    assert 0 < routed <= pairs * (I * 4 + 8) + 3 * 256


@pytest.mark.parametrize("T,E,topk", [(ROWS - 2 ** 17, 1, 1), (2 ** 29, 8, 1), (2 ** 28, 4096, 2)])
def test_rows_below_take_the_tensor_cores(lib, T, E, topk):
    pairs = T * topk
    assert experts_bytes(lib, T, E, topk) >= pairs * (4 + 2 * I + 2 * H + 4 * H)  # ids, h, x in sorted order, y


@pytest.mark.parametrize("T,E,topk,H,I", [(9, 5, 3, 33, 17), (9, 5, 3, 64, 37), (9, 5, 3, 37, 64)])
def test_odd_rows_take_the_plain_kernels(lib, T, E, topk, H, I):
    p = lib.mr_expert_params(T, H, I, E, topk, lib.MR_BF16, lib.MR_SILU)
    assert 0 < lib.moe_experts_workspace_bytes(p) <= T * topk * I * 4 + 256
