"""Refusals of the rows' entry points and helpers, on the host without a GPU: every call here fails its checks (or has
nothing to do) before any CUDA call."""
import ctypes

import pytest
import torch

FAKE = 0x10000  # never dereferenced
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    from top_gating_expert_row_gb300 import build

    build.build()
    import top_gating_expert_row_gb300 as m

    return m


POINTERS = dict(
    moe_permute_fwd=["x", "topk_idx", "sorted_token_ids", "num_tokens_post_pad", "rows", "pair_row", "status"],
    moe_permute_bwd=["grad_rows", "pair_row", "grad_x", "status"],
    moe_combine_fwd=["rows", "pair_row", "topk_w", "residual", "p", "rng", "out", "status"],
    moe_combine_bwd=["grad_out", "rows", "pair_row", "topk_w", "sorted_token_ids", "num_tokens_post_pad", "p", "rng",
                     "grad_rows", "grad_w", "status"],
    moe_expert_act_fwd=["gu", "num_rows", "p", "rng", "h"],
    moe_expert_act_bwd=["grad_h", "gu", "num_rows", "p", "rng", "grad_gu", "h"],
    moe_dropout_fwd=["x", "residual", "p", "rng", "y"],
    moe_dropout_bwd=["grad_y", "p", "rng", "grad_x"],
)
NULLABLE = {("moe_expert_act_bwd", "h")} | {(n, q) for n in POINTERS for q in ("status", "residual", "num_rows")}
CASES = [(n, q) for n, names in POINTERS.items() for q in names if q != "p"]


def call(lib, name, ptr=None, p=0.25, E_tot=8, **kw):
    a = {q: FAKE for q in POINTERS[name]}
    a["p"] = p
    a.update(ptr or {})
    args = [a[q] for q in POINTERS[name]]
    if "act" in name:
        f = dict(n_rows=4, I=32, act=0, dtype=1)
        f.update(kw)
        args.insert(0, ctypes.byref(lib.mr_act_params(**f)))
    elif "dropout" in name:
        f = dict(T=4, H=32, dtype=1)
        f.update(kw)
        args = [f["T"], f["H"], f["dtype"]] + args
    else:
        f = dict(T=4, H=32, topk=2, n_rows=16, dtype=1)
        f.update(kw)
        args.insert(0, ctypes.byref(lib.mr_rows_params(**f)))
        if name == "moe_permute_fwd":
            args.insert(1, E_tot)
    return getattr(lib._lib, name)(*args, None)


def empty(name):
    return dict(n_rows=0) if "act" in name else dict(T=0)


@pytest.mark.parametrize("name,q", CASES)
def test_null_and_misaligned(lib, name, q):
    assert call(lib, name, {q: FAKE + 1}) == 1
    if (name, q) not in NULLABLE:
        assert call(lib, name, {q: None}) == 1
    if q == "rng":
        assert call(lib, name, {q: FAKE + 4}) == 1


@pytest.mark.parametrize("name", POINTERS)
def test_sizes(lib, name):
    width = "I" if "act" in name else "H"
    rows = "n_rows" if "act" in name else "T"
    for kw, code in ((({width: 0}), 1), ({width: -5}, 1), ({rows: -1}, 1), (dict(dtype=2), 1), (dict(dtype=-1), 1),
                     ({width: (1 << 20) + 1}, 2)):
        assert call(lib, name, **kw) == code, kw
    if "act" in name:
        assert call(lib, name, act=2) == 1 and call(lib, name, act=-1) == 1
    if rows == "T" and "dropout" not in name:
        assert call(lib, name, topk=0) == 1 and call(lib, name, n_rows=-1) == 1
        assert call(lib, name, T=1 << 30, topk=2) == 1
    if name == "moe_permute_fwd":
        assert call(lib, name, E_tot=0) == 1
    if "p" in POINTERS[name]:
        for p in (-0.01, 1.01, float("nan"), float("inf")):
            assert call(lib, name, p=p) == 1
    assert call(lib, name, {q: None for q in POINTERS[name] if q not in ("p", "rng")}, **empty(name)) == 0


def test_null_options(lib):
    for name in ("moe_permute_fwd", "moe_permute_bwd", "moe_combine_fwd", "moe_combine_bwd"):
        args = [1] if name == "moe_permute_fwd" else []
        args += [0.0 if q == "p" else FAKE for q in POINTERS[name]]
        assert getattr(lib._lib, name)(None, *args, None) == 1
    for name in ("moe_expert_act_fwd", "moe_expert_act_bwd"):
        assert getattr(lib._lib, name)(None, *[0.0 if q == "p" else FAKE for q in POINTERS[name]], None) == 1


# ---- the helpers' refusals ---------------------------------------------------


def _args():
    i32 = dict(dtype=torch.int32)
    rows, pair_row, w = torch.ones(10, 32).to(BF16), torch.zeros(4, 2, **i32), torch.ones(4, 2)
    x, ids, n, rng = torch.ones(4, 32).to(BF16), torch.zeros(10, **i32), torch.ones(1, **i32), torch.zeros(2, dtype=torch.int64)
    return dict(
        permute=dict(x=x, topk_idx=pair_row, E_tot=3, sorted_token_ids=ids, num_tokens_post_pad=n, rows=rows),
        permute_bwd=dict(grad_rows=rows, pair_row=pair_row),
        combine=dict(rows=rows, pair_row=pair_row, topk_w=w, residual=x, p=0.5, rng=rng),
        combine_bwd=dict(grad_out=x, rows=rows, pair_row=pair_row, topk_w=w, sorted_token_ids=ids,
                         num_tokens_post_pad=n, p=0.5, rng=rng, grad_rows=rows.clone()),
        expert_act=dict(gu=rows, num_rows=n, p=0.5, rng=rng, h=torch.ones(10, 16).to(BF16)),
        expert_act_bwd=dict(grad_h=torch.ones(10, 16).to(BF16), gu=rows, num_rows=n, p=0.5, rng=rng,
                            grad_gu=rows.clone(), h=torch.ones(10, 16).to(BF16)),
        dropout=dict(x=x, p=0.5, rng=rng, residual=x.clone()),
        dropout_bwd=dict(grad_y=x, p=0.5, rng=rng),
    )


TENSORS = [(h, q) for h, kw in _args().items() for q, v in kw.items() if isinstance(v, torch.Tensor)]


@pytest.mark.parametrize("helper,q", TENSORS)
def test_helpers_refuse(lib, helper, q):
    def go(**change):
        with torch.no_grad():
            getattr(lib, helper)(**{**_args()[helper], **change})

    t = _args()[helper][q]
    with pytest.raises(ValueError, match="CUDA device"):  # as far as host tensors come
        go()
    with pytest.raises(TypeError):
        go(**{q: t.to(torch.float16)})
    with pytest.raises(ValueError):
        go(**{q: t[None]})  # another rank
    if t.numel() > 1:
        with pytest.raises(ValueError, match="contiguous"):
            go(**{q: torch.stack([t, t], -1)[..., 0]})
    if t.is_floating_point():
        with pytest.raises(ValueError, match="gradients are computed by"):
            getattr(lib, helper)(**{**_args()[helper], q: t.clone().requires_grad_()})


@pytest.mark.parametrize("helper", ["combine", "combine_bwd", "expert_act", "expert_act_bwd", "dropout", "dropout_bwd"])
def test_helpers_refuse_dropout(lib, helper):
    for change in (dict(p=-0.1), dict(p=1.5), dict(p=float("nan")), dict(p=0.5, rng=None)):
        with pytest.raises(ValueError):
            getattr(lib, helper)(**{**_args()[helper], **change})


def test_odd_gated_width(lib):
    with pytest.raises(ValueError, match="gu"):
        lib.expert_act(torch.ones(4, 33).to(BF16))
