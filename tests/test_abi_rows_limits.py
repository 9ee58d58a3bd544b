"""Sizes past 32 bits, which would pass for small ones in the library's fields, are refused by the helpers on the host."""
import pytest
import torch

from test_abi_rows import _args, lib  # noqa: F401  (the fixture)

BIG = (1 << 32) + 5  # 5 in 32 bits


@pytest.mark.parametrize("plan,sizes", [
    ("_rows_plan", 4), ("_act_plan", 2), ("_experts_plan", 5), ("_adapter_plan", 5), ("_layer_plan", 2)])
def test_plans(lib, plan, sizes):  # noqa: F811
    rest = dict(_rows_plan=[0], _act_plan=[0, 0], _experts_plan=[0], _adapter_plan=[False],
                _layer_plan=[0, 4, 4, 2, 0, 0, 0, 0, 0, 0, 1.0, 1.0])[plan]
    for i in range(sizes):
        args = [8] * sizes + rest
        args[i] = BIG
        with pytest.raises(ValueError, match="2\\^31"):
            getattr(lib, plan)(*args)
    if plan == "_layer_plan":
        for i in range(3):
            options = rest[1:]
            options[i] = BIG
            with pytest.raises(ValueError, match="2\\^31"):
                lib._layer_plan(8, 8, 0, *options)


@pytest.mark.parametrize("shape", [(BIG, 1), (1, BIG)])
def test_dropout(lib, shape):  # noqa: F811
    x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    for call in (lambda: lib.dropout(x, 0.0, None), lambda: lib.dropout_bwd(x, 0.0, None)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_number_of_experts(lib):  # noqa: F811
    with pytest.raises(ValueError, match="2\\^31"):
        lib.permute(**{**_args()["permute"], "E_tot": BIG})
