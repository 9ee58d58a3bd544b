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


@pytest.mark.parametrize("up", [1.0, 2.0 ** 60])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("kind", [0, 1], ids=["silu", "gelu"])
def test_far_gates_keep_their_values(mr, kind, dtype, up):
    """Gates so low that the exponentials are subnormal, as long as there is anything left of the results in their type.

    Relative errors as for other gates: an exponential's argument and its rounded square (GELU: 1.5 g^2 EPS, with the
    polynomial 2 g^2), some EPS besides. fp32: exponents to 150 are kept, so that less than |g| 2^-150 of a result is lost;
    GELU's products with the exponential are rounded to half a subnormal step, 2^-150, before they are multiplied by g, and
    its polynomial, taken at 14 for gates beyond, is 0.2 of such a step off: (2 |g| + 4) 2^-150 in all. bf16: exponents to
    142 are kept, |g| + 1 is below 100 there, and less than 2^-135 of act and act' is lost (half of bf16's least number
    is 2^-134). Results may be subnormal in their own type.
    """
    lo, hi = ((-112.0, -80.0), (-14.5, -12.0))[kind]
    g = torch.linspace(lo, hi, 64 * 512).view(64, 512).to(dtype)
    d = g.double()
    a, da = ref.act(d, kind)
    flat = (2 * d.abs() + 4) * 2.0 ** -150 + (2.0 ** -135 if dtype is BF16 else 0.0)
    if kind == 0:
        rel = (d.abs() + 12) * EPS
        ta = rel * a.abs() + flat
        tda = (rel + 3 * EPS) * (a.abs() + torch.sigmoid(d)) + flat
    else:
        pdf = torch.exp(-0.5 * d * d) * (2 * torch.pi) ** -0.5
        rel = (2 * d * d + 10) * EPS
        ta = rel * a.abs() + flat
        tda = rel * (a / d).abs() + (1.5 * d * d + 10) * EPS * (d * pdf).abs() + flat
    step = {F32: 2.0 ** -150, BF16: 2.0 ** -134}[dtype]
    half = torch.finfo(dtype).eps / 2 * (1 + 2.0 ** -7)  # of the value before it was rounded
    gu = torch.cat([g, torch.full_like(g, up)], 1).cuda()
    h = mr.expert_act(gu, act=kind).cpu().double()
    assert ((h - a * up).abs() <= up * (ta + 2 * EPS * a.abs()) + half * (a * up).abs() + step).all()
    out = mr.expert_act_bwd(torch.ones_like(g).cuda(), gu, act=kind)
    got = out["grad_gu"].cpu().double()
    assert ((got[:, 512:] - a).abs() <= ta + EPS * a.abs() + half * a.abs() + step).all()
    assert ((got[:, :512] - up * da).abs() <= up * (tda + 2 * EPS * da.abs()) + half * (up * da).abs() + step).all()
    assert torch.equal(out["h"].cpu().double(), h)


def test_far_gates_that_leave_nothing(mr):
    """Where nothing is left results are 0, not NaN; a NaN stays one."""
    g = torch.tensor([[-200.0, -1e4, -1e30, -3.4e38, float("nan"), -1.0, 1e30, 0.0]], device="cuda")
    for kind in (0, 1):
        gu = torch.cat([g, torch.ones_like(g)], 1)
        for t in (mr.expert_act(gu, act=kind), mr.expert_act_bwd(torch.ones_like(g), gu, act=kind)["grad_gu"][:, :8]):
            assert (t[0, :4] == 0).all() and t[0, 4].isnan() and t[0, 5:].isfinite().all(), (kind, t)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("T,k,H", [(7, 2, 264), (7, 5, 257), (1400, 3, 520), (1100, 4, 257)])
def test_dropped_gradients_are_zero_whatever_they_meet(mr, T, k, H, dtype):
    """A dropped element's gradient is 0 in grad_w's sums and in grad_rows, although the row holds an infinity or NaN there
    or the weight is one: out does not depend on them. Kept elements follow the formula. Pairs alone and, from 4096 on,
    tokens whose rows share their factors."""
    gen = torch.Generator().manual_seed(H + T)
    P, p, dev = T * k, 0.5, "cuda"
    pair_row = torch.randperm(P, generator=gen).view(T, k)
    ids = torch.empty(P, dtype=torch.int32)
    ids[pair_row.view(-1)] = torch.arange(P, dtype=torch.int32)
    rng = torch.tensor([21, 22])
    f = ref.factors(T, H, p, rng.tolist())
    go = torch.randn(T, H, generator=gen).to(dtype)
    rows = torch.randn(P, H, generator=gen).to(dtype)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")]).to(dtype)
    which = torch.randint(0, 6, (T, k, H), generator=gen)
    which = torch.where((f == 0)[:, None].expand(T, k, H), which, 5)
    mine = rows[pair_row]
    mine = torch.where(which < 3, bad[which.clamp(max=2)], mine)
    rows[pair_row.view(-1)] = mine.view(P, H)
    w = torch.rand(T, k, generator=gen)
    w[0, 0], w[T // 2, 1], w[T - 1, 0] = float("inf"), float("nan"), -float("inf")
    out = mr.combine_bwd(go.to(dev), rows.to(dev), pair_row.to(torch.int32).to(dev), w.to(dev), ids.to(dev),
                         torch.tensor([P], dtype=torch.int32, device=dev), p=p, rng=rng.to(dev))
    g = go.double() * f
    kept = (f != 0)[:, None].expand(T, k, H)
    terms = torch.where(kept, g[:, None] * mine.double(), 0.0)
    assert ((out["grad_w"].cpu().double() - terms.sum(2)).abs()
            <= ((H + 255) // 256 * 8 + 7) * EPS * terms.abs().sum(2)).all()  # a lane's chain, lanes, the scale
    want = torch.where(kept, g[:, None] * w.double()[:, :, None], 0.0).view(P, H)
    got = out["grad_rows"].cpu()[pair_row.view(-1)].double()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
    fine = want.isfinite()
    assert (got[~fine & ~want.isnan()] == want[~fine & ~want.isnan()]).all()
    half = torch.finfo(dtype).eps / 2 * (1 + 2.0 ** -7)
    assert ((got - want).abs()[fine] <= (3 * EPS + half) * want.abs()[fine]).all()  # the scale, two products, the output's


@pytest.mark.parametrize("p", [0.0, 0.5])
def test_gradients_and_padding_past_32_bits(mr, p):
    """Pairs and padding rows whose elements lie past 2^31, a gradient of 4.4 GB that holds NaN before; with dropout in the
    kernel whose tokens share their factors."""
    n, H, T, k, dev = 270001, 8192, 1400, 3, "cuda"
    P = T * k
    gen = torch.Generator().manual_seed(3)
    at = torch.randperm(n - 1, generator=gen)[:P]
    at[0] = n - 1
    assert (at * H >= 1 << 31).sum() > 100
    at = at.to(dev)
    ids = torch.full((n,), P, dtype=torch.int32, device=dev)
    ids[at] = torch.arange(P, dtype=torch.int32, device=dev)
    rows = torch.full((n, H), float("nan"), dtype=BF16, device=dev)  # the padding is not read
    vals = torch.randn(P, H, generator=gen).to(BF16).to(dev)
    rows[at] = vals
    go, w = torch.randn(T, H, generator=gen).to(BF16).to(dev), torch.rand(T, k, generator=gen).to(dev)
    rng = torch.tensor([8, 9], device=dev)
    npp = torch.tensor([n], dtype=torch.int32, device=dev)
    grad = torch.full((n, H), float("nan"), dtype=BF16, device=dev)
    got = mr.combine_bwd(go, rows, at.view(T, k).to(torch.int32), w, ids, npp, p=p, rng=rng, grad_rows=grad)
    g = go.float() * ref.factors(T, H, p, rng.tolist()).float().to(dev)  # factors of 0, 1 and 2: exact
    assert torch.equal(grad[at], (g[:, None] * w[:, :, None]).to(BF16).view(P, H))
    terms = g.double()[:, None] * vals.view(T, k, H).double()
    # a lane's chain, lanes, the four warps of a token
    assert ((got["grad_w"] - terms.sum(2)).abs() <= (H // 32 + 10) * EPS * terms.abs().sum(2)).all()
    padding = torch.ones(n, dtype=torch.bool, device=dev)
    padding[at] = False
    for first in range(0, n, 30000):
        part = grad[first : first + 30000].view(torch.int16)
        assert not (part != 0).any(1)[padding[first : first + 30000]].any(), first


@pytest.mark.parametrize("score_fn,renorm,shared", [(0, 0, 0), (0, 1, 1), (1, 0, 1), (1, 1, 0)])
def test_from_logits_to_gradients(mr, score_fn, renorm, shared):
    """A layer's training pass from the router's logits to their gradient: route, sort, permute, products by torch,
    expert_act, combine, and back, where combine_bwd's grad_w goes to route_bwd by a scatter into zeros [T, E], the shared
    experts' columns left out (their weights are constants). Against the whole in 64 bits with the selection held fixed.

    d = 1.5e-3 bounds the error of grad_w as it does in the test of a layer's gradients. A weight's gradient enters ds with
    scaling / A, once as itself and once in their mean, A > 1/2 being the sum of the winners' scores (or 1): 2 * 1.5 * 2 d;
    dx = s (ds - sum s ds) doubles that: 12 d.
    """
    from test_gpu_rows import _layer

    T, k, E, H, I, block, p, d = 29, 3, 7, 48, 20, 4, 0.25, 1.5e-3
    gen = torch.Generator().manual_seed(6)
    x, logits = torch.randn(T, H, generator=gen), torch.randn(T, E, generator=gen)
    all_e = E + shared
    w13, w2 = torch.randn(all_e, 2 * I, H, generator=gen) * H ** -0.5, torch.randn(all_e, H, I, generator=gen) * I ** -0.5
    go, rng = torch.randn(T, H, generator=gen), torch.tensor([[12, 0], [12, 1]])
    options = dict(score_fn=score_fn, renorm=renorm, n_shared=shared, scaling=1.5, shared_weight=0.5)
    back = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        r = mr.route(logits.cuda(), k + shared, **options)
        out, backward, _ = _layer(mr, x.cuda(), r["topk_idx"], r["topk_w"], w13.cuda(), w2.cuda(), rng.cuda(), p, block, 0)
        got = backward(go.cuda())
        idx = r["topk_idx"][:, :k].long()
        grad_probs = torch.zeros(T, E, device="cuda").scatter_(1, idx, got["w"][:, :k])
        grad_logits = mr.route_bwd(mr.params_for(logits, k + shared, **options), grad_probs, r["intermediate"], r["routing_map"])
    finally:
        torch.backends.cuda.matmul.allow_tf32 = back

    idx = r["topk_idx"].cpu()
    assert (idx[:, k:] == torch.arange(E, all_e)).all()
    _, n, pair_row = ref.sort(idx, all_e, block)
    f_row, f_out = ref.factors(n, I, p, rng[0].tolist()), ref.factors(T, H, p, rng[1].tolist())
    leaf = logits.double().requires_grad_()
    s = torch.softmax(leaf, 1) if score_fn == 0 else torch.sigmoid(leaf)
    win = s.gather(1, idx[:, :k].long())
    total = win.sum(1, keepdim=True)
    assert not renorm or (total > 0.5).all()
    w = torch.cat([1.5 * (win / total if renorm else win), torch.full((T, shared), 0.5, dtype=torch.float64)], 1)
    x64, w13, w2 = x.double(), w13.double(), w2.double()
    y = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k + shared):
            gu = w13[idx[t, j]] @ x64[t]
            h = f_row[pair_row[t, j]] * ref.act(gu[:I], 0)[0] * gu[I:]
            y[t] = y[t] + w[t, j] * (w2[idx[t, j]] @ h)
    want = x64 + f_out * y
    assert ((out.cpu().double() - want).abs() < d).all()
    want.backward(go.double())
    assert ((grad_logits.cpu().double() - leaf.grad).abs() < 12 * d).all()
    assert leaf.grad.abs().max() > 1


def test_rows_of_pairs_that_topk_idx_drops(mr):
    """Sorted for more experts than E_tot says: the pairs beyond have -1 each time, and the status word says so."""
    T, k, E, H = 3000, 4, 12, 16
    gen = torch.Generator().manual_seed(4)
    idx = torch.argsort(torch.rand(T, E, generator=gen), 1)[:, :k].to(torch.int32)
    srt = mr.sort(idx.cuda(), torch.ones(T, k, device="cuda"), E, 16)
    ids, n = srt["sorted_token_ids"], srt["num_tokens_post_pad"]
    _, _, pair_row = ref.sort(idx, E, 16)
    x = torch.randn(T, H, generator=gen).cuda()
    for E_tot, code in ((E, 0), (E - 2, mr.MR_ERANGE)):
        want = torch.where(idx < E_tot, pair_row, -1)
        for _ in range(4):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = mr.permute(x, idx.cuda(), E_tot, ids, n, status=status)
            assert torch.equal(out["pair_row"].cpu().long(), want) and int(status) == code
            assert torch.equal(out["rows"][pair_row.view(-1).cuda()], x.repeat_interleave(k, 0))
