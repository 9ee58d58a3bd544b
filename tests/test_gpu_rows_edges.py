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


STALE = ["-1", "0", "last", "behind", "lowest", "highest", "any", "whole"]


@pytest.mark.parametrize("missing", ["behind the buffer", "padding's id", "id too large", "negative id"])
@pytest.mark.parametrize("T,k,E,H,block,dropped", [
    (1, 2, 4, 8, 1, 0.0), (16, 2, 8, 64, 16, 0.0), (333, 5, 20, 1001, 16, 0.2), (9000, 4, 32, 16, 64, 0.1)])
def test_pairs_without_a_row(mr, T, k, E, H, block, dropped, missing):
    """Every pair has its row or -1, whatever pair_row held before: where rows lie behind the buffer, and where ids are
    missing from sorted_token_ids. What follows takes such pairs as none."""
    gen = torch.Generator().manual_seed(T)
    P, code = T * k, mr.MR_F32
    idx = torch.argsort(torch.rand(T, E, generator=gen), 1)[:, :k].to(torch.int32)
    idx[torch.rand(T, k, generator=gen) < dropped] = -1
    full, n, pair_row = ref.sort(idx, E, block)
    used, ids = n, torch.tensor(full, dtype=torch.int32)
    if missing == "behind the buffer":
        ids = ids[: max(1, n * 2 // 3)].clone()
    else:
        gone = torch.rand(n, generator=gen) < 0.1
        gone[pair_row.max()] = True
        ids[gone & (ids < P)] = {"padding's id": P, "id too large": P + 3, "negative id": -2}[missing]
    n_rows = len(ids)
    want = torch.full((P,), -1, dtype=torch.int32)
    real = (ids >= 0) & (ids < P)
    want[ids[real].long()] = torch.arange(n_rows, dtype=torch.int32)[real]
    assert (want.view(T, k) != pair_row).any()  # some pair has lost its row
    x = torch.randn(T, H, generator=gen)
    want_rows = torch.where(real[:, None], x[(ids.clamp(0, P - 1) // k).long()], torch.zeros(()))

    dev = "cuda"
    xg, ig, sg = x.to(dev), idx.to(dev), ids.to(dev)
    npp = torch.tensor([used], dtype=torch.int32, device=dev)
    rows = torch.empty(n_rows, H, device=dev)
    p = mr.mr_rows_params(T, H, k, n_rows, code)
    for stale in STALE:
        held = {"-1": -1, "0": 0, "last": n_rows - 1, "behind": n_rows, "lowest": -(1 << 31), "highest": (1 << 31) - 1}
        if stale in held:
            got = torch.full((T, k), held[stale], dtype=torch.int32, device=dev)
        elif stale == "any":
            got = torch.randint(-3, n_rows + 3, (T, k), generator=gen, dtype=torch.int32).to(dev)
        else:
            got = pair_row.to(torch.int32).to(dev)  # what the same call gave before rows went missing
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        mr.moe_permute_fwd(p, E, xg, ig, sg, npp, rows, got, status)
        assert torch.equal(got.cpu(), want.view(T, k)), stale
        assert torch.equal(rows.cpu(), want_rows), stale
        assert int(status) == (0 if missing == "padding's id" else mr.MR_ERANGE)

    w = torch.rand(T, k, generator=gen)
    mine = ref.gathered(want_rows, want.view(T, k))
    terms = mine * w.double()[:, :, None]
    out = mr.combine(rows, got, w.to(dev))
    assert ((out.cpu().double() - terms.sum(1)).abs() <= (k + 1) * EPS * terms.abs().sum(1)).all()
    back = mr.combine_bwd(xg, rows, got, w.to(dev), sg, npp)
    assert (back["grad_w"].cpu()[want.view(T, k) < 0] == 0).all()
    want_grad = torch.zeros(n_rows, H)
    want_grad[want[want >= 0].long()] = (x[:, None] * w[:, :, None]).view(P, H)[want >= 0]
    assert torch.equal(back["grad_rows"].cpu(), want_grad)


def test_as_many_rows_as_the_type_counts(mr):
    """n_rows = 2^31 - 1, the most that is accepted, all of them in use: one column, so 4 GB a buffer."""
    n, dev, i32 = (1 << 31) - 1, "cuda", torch.int32
    T, k = 1400, 3  # with dropout a token's rows share its factors from 4096 pairs on
    P = T * k
    at = torch.randperm(n // 1000, generator=torch.Generator().manual_seed(1))[:P] * 999
    at[:3] = torch.tensor([n - 1, n - 33, 0])  # the last row among them
    assert at.unique().numel() == P
    at = at.to(dev)
    ids = torch.full((n,), P, dtype=i32, device=dev)
    ids[at] = torch.arange(P, dtype=i32, device=dev)
    npp = torch.tensor([n], dtype=i32, device=dev)
    pair_row = at.view(T, k).to(i32)
    rows = torch.zeros(n, 1, dtype=BF16, device=dev)
    vals = torch.randn(P, 1, device=dev).to(BF16)
    rows[at] = vals
    w, x = torch.rand(T, k, device=dev), torch.randn(T, 1, device=dev).to(BF16)
    rng = torch.tensor([5, 6], device=dev)
    padding = torch.ones(n, dtype=torch.bool, device=dev)
    padding[at] = False
    for p in (0.0, 0.5):
        grad = torch.full((n, 1), float("nan"), dtype=BF16, device=dev)
        got = mr.combine_bwd(x, rows, pair_row, w, ids, npp, p=p, rng=rng, grad_rows=grad)
        g = x.float() * ref.factors(T, 1, p, rng.tolist()).float().to(dev)
        assert torch.equal(got["grad_w"], g * vals.view(T, k).float())  # one product in fp32
        assert torch.equal(grad[at], (g * w).view(P, 1).to(BF16))
        assert int(torch.count_nonzero(grad.view(torch.int16)[:, 0][padding])) == 0
    got = mr.permute(x, torch.zeros(T, k, dtype=i32, device=dev), 1, ids, npp, rows=grad)
    assert torch.equal(got["pair_row"], pair_row)
    assert torch.equal(grad[at], x.expand(T, k).reshape(P, 1))
    assert int(torch.count_nonzero(grad.view(torch.int16)[:, 0][padding])) == 0
