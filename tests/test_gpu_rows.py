"""The rows' permutation, weighted sum, gated activation and dropout on the GPU against their definitions in 64 bits.

Tolerances. EPS = 2^-24 is half a step of fp32; an output in type t adds half a step of its own, finfo(t).eps / 2 of its
value. A sum of n fused products is off by at most n EPS of the sum of the terms' magnitudes, every further product or sum
by EPS of its value.
"""
import pytest
import torch

import rows_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 2.0 ** -24
TINY = 2.0 ** -120  # results of a flushed exponential


def check(got, want, tol, what):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    assert torch.equal(got.isnan(), want.isnan()), what
    bad = (got - want).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), (got - want).abs()[bad].max().item())


def half_step(want, dtype):
    return want.abs() * (torch.finfo(dtype).eps / 2) * (1 + 2.0 ** -7)  # of the value before it was rounded


def make_pairs(gen, T, k, E, dropped):
    idx = torch.argsort(torch.rand(T, max(E, k), generator=gen), 1)[:, :k].to(torch.int32) % E
    if dropped:
        gone = torch.rand(T, k, generator=gen) < dropped
        gone[T // 2] = True
        idx[gone] = torch.where(torch.rand(int(gone.sum()), generator=gen) < 0.5, -1, E).to(torch.int32)
    return idx.contiguous()


def offset_view(t, shift):
    """t's values on the GPU, `shift` elements behind an aligned base."""
    flat = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
    v = flat[shift:].view(t.shape)
    v.copy_(t)
    return v


def setup(mr, T, k, E, H, block, dtype, dropped=0.0, shift=0, seed=0):
    gen = torch.Generator().manual_seed(seed + 1000 * T + H)
    idx = make_pairs(gen, T, k, E, dropped)
    ids, n, pair_row = ref.sort(idx, E, block)
    srt = mr.sort(idx.cuda(), torch.ones(T, k, device="cuda"), E, block)
    n_rows = len(srt["sorted_token_ids"])
    assert int(srt["num_tokens_post_pad"]) == n
    x = torch.randn(T, H, generator=gen).to(dtype)
    rows = torch.randn(n_rows, H, generator=gen).to(dtype)
    rows[n:] = float("nan")  # not to be read
    w = torch.rand(T, k, generator=gen)
    return dict(gen=gen, idx=idx, ids=ids, n=n, n_rows=n_rows, pair_row=pair_row, srt=srt, x=x, rows=rows, w=w,
                rng=torch.tensor([0x1234567890ABCDEF + seed, 0x0FEDCBA987654321]), T=T, k=k, E=E, H=H,
                g=lambda t: offset_view(t, shift))


SIZES = [  # T, topk, E, H, block, dropped, shift
    (1, 1, 1, 1, 1, 0.0, 0),
    (1, 8, 256, 2048, 16, 0.0, 0),
    (3, 2, 5, 8, 4, 0.0, 0),
    (16, 2, 8, 512, 16, 0.0, 0),
    (37, 5, 100, 1000, 16, 0.3, 0),
    (37, 5, 100, 1001, 16, 0.3, 0),
    (33, 9, 384, 257, 64, 0.0, 1),
    (20, 33, 40, 264, 8, 0.1, 0),
    (9, 40, 64, 31, 1, 0.0, 3),
    (64, 4, 7, 2304, 32, 0.5, 1),
    (200, 1, 3, 776, 128, 1.0, 0),
    (130, 3, 16, 4096, 64, 0.0, 0),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_permute(mr, size, dtype):
    T, k, E, H, block, dropped, shift = size
    s = setup(mr, T, k, E, H, block, dtype, dropped, shift)
    buf = s["g"](torch.full((s["n_rows"], H), float("nan")).to(dtype))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mr.permute(s["g"](s["x"]), s["idx"].cuda(), E, s["srt"]["sorted_token_ids"], s["srt"]["num_tokens_post_pad"],
                     rows=buf, status=status)
    assert out["rows"] is buf and int(status) == 0
    want = ref.permute(s["x"], s["ids"], s["n"], s["n_rows"], k)
    check(buf, want, torch.zeros_like(want), "rows")  # NaN behind the rows in use: left as they were
    assert torch.equal(out["pair_row"].cpu().long(), s["pair_row"])

    # its gradient: k - 1 sums of rows
    rows = s["g"](s["rows"])
    got = mr.permute_bwd(rows, out["pair_row"], status=status)
    mine = ref.gathered(s["rows"], s["pair_row"])
    want = mine.sum(1)
    check(got, want, k * EPS * mine.abs().sum(1) + half_step(want, dtype), "grad_x")
    assert int(status) == 0 and torch.equal(got, mr.permute_bwd(rows, out["pair_row"]))


@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_combine(mr, size, dtype, p):
    T, k, E, H, block, dropped, shift = size
    s = setup(mr, T, k, E, H, block, dtype, dropped, shift)
    rows, w, pair_row, rng = s["g"](s["rows"]), s["w"].cuda(), s["pair_row"].to(torch.int32).cuda(), s["rng"].cuda()
    mine = ref.gathered(s["rows"], s["pair_row"]) * s["w"].double()[:, :, None]
    f = ref.factors(T, H, p, s["rng"].tolist())
    size_of = mine.abs().sum(1) * f
    for residual in (None, s["x"]):
        want = f * mine.sum(1) + (0 if residual is None else residual.double())
        # k products, the scale and the product with it, the residual
        tol = (k + 2) * EPS * size_of + EPS * want.abs() + half_step(want, dtype)
        got = mr.combine(rows, pair_row, w, None if residual is None else s["g"](residual), p=p, rng=rng)
        check(got, want, tol, "out")
    # in place of the residual
    res = s["g"](s["x"])
    code = mr.MR_F32 if dtype is F32 else mr.MR_BF16
    mr.moe_combine_fwd(mr.mr_rows_params(T, H, k, s["n_rows"], code), rows, pair_row, w, res, p, rng, res)
    assert torch.equal(res, got)

    # the gradient
    go = torch.randn(T, H, generator=s["gen"]).to(dtype)
    buf = s["g"](torch.full((s["n_rows"], H), float("nan")).to(dtype))
    out = mr.combine_bwd(s["g"](go), rows, pair_row, w, s["srt"]["sorted_token_ids"], s["srt"]["num_tokens_post_pad"],
                         p=p, rng=rng, grad_rows=buf)
    assert out["grad_rows"] is buf
    g = go.double() * f
    want = torch.full((s["n_rows"], H), float("nan"), dtype=torch.float64)
    want[: s["n"]] = 0
    has = s["pair_row"] >= 0
    want[s["pair_row"][has]] = (g[:, None] * s["w"].double()[:, :, None])[has]
    # the scale, two products
    check(buf, want, 3 * EPS * want.abs() + half_step(want, dtype), "grad_rows")
    plain = ref.gathered(s["rows"], s["pair_row"])
    terms = g[:, None] * plain
    # a lane's chain, five steps across lanes, the scale and the product with it
    check(out["grad_w"], terms.sum(2), ((H + 255) // 256 * 8 + 7) * EPS * terms.abs().sum(2), "grad_w")
    again = mr.combine_bwd(s["g"](go), rows, pair_row, w, s["srt"]["sorted_token_ids"],
                           s["srt"]["num_tokens_post_pad"], p=p, rng=rng)
    assert torch.equal(again["grad_w"], out["grad_w"])
    assert torch.equal(again["grad_rows"][: s["n"]], buf[: s["n"]])


MANY = [  # T, topk, E, H, block, dropped, shift: more pairs and rows than the GPU takes at a time
    (1400, 3, 16, 257, 16, 0.2, 0),
    (1030, 4, 64, 2304, 32, 0.0, 0),
    (130, 33, 40, 264, 8, 0.1, 1),
    (9000, 4, 32, 40, 16, 0.1, 0),
    (2500, 9, 384, 64, 1, 0.0, 0),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("size", MANY, ids=str)
def test_many_pairs(mr, size, dtype):
    """The same checks where CTAs take several rows, and where a token's rows share its dropout factors."""
    test_permute(mr, size, dtype)
    test_combine(mr, size, dtype, 0.3)


def gate_tolerance(g, kind):
    """Relative error of act(g), absolute error of act'(g), in 64 bits.

    The exponential's argument is rounded once and its base-2 exponent (|x| log2 e) EPS off, its result 2 units (4 EPS)
    besides; sums and a reciprocal of 2 units follow. GELU's Phi(-a) = exp(-a^2 / 2) R(s): the square's rounding and the
    exponent's enter a^2 / 2 times each, the exponential adds 4 EPS; R's polynomial is within 0.25 EPS of its function
    and off by at most 2.1 EPS below a = 0.5, 3.5 below 1, 7.1 below 2, 13 below 4, 35 below 8, 69 below 14 (in fp32,
    with a unit's error in s, tried at 400,001 points), one product's EPS: below (2 a^2 + 10) EPS throughout.
    """
    a, da = ref.act(g, kind)
    if kind == 0:
        s = torch.sigmoid(g)
        rel = (g.abs() + 12) * EPS
        # s, 1 - s (s's error and a rounding, absolute), a (1 - s), the sum
        return (rel + EPS) * a.abs() + TINY * g.abs(), rel * s + a.abs() * (rel * s + EPS) + (rel + 3 * EPS) * (a * (1 - s)).abs() + EPS * da.abs() + TINY
    cdf = 0.5 * torch.special.erfc(-g / 2 ** 0.5)
    pdf = torch.exp(-0.5 * g * g) * (2 * torch.pi) ** -0.5
    rel = (2 * g * g + 10) * EPS
    # the exponential of -g^2 / 2: two roundings of its argument, its own, the constant's and two products
    erel = (1.5 * g * g + 9) * EPS
    return (rel + EPS) * a.abs() + TINY * g.abs(), rel * cdf + erel * (g * pdf).abs() + 2 * EPS * da.abs() + EPS * (g * pdf).abs() + TINY


ACT_SIZES = [  # rows, used, I, shift
    (1, 1, 1, 0), (1, 0, 8, 0), (5, 5, 7, 0), (40, 37, 344, 0), (64, 64, 768, 1), (33, 20, 257, 0), (300, 299, 1001, 0),
    (128, 100, 2048, 0), (17, 40, 520, 0),
]


@pytest.mark.parametrize("p", [0.0, 0.4])
@pytest.mark.parametrize("kind", [0, 1], ids=["silu", "gelu"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("size", ACT_SIZES, ids=str)
def test_expert_act(mr, size, dtype, kind, p):
    n, used, I, shift = size
    gen = torch.Generator().manual_seed(n * I)
    gu = (torch.randn(n, 2 * I, generator=gen) * 3).to(dtype)
    gh = torch.randn(n, I, generator=gen).to(dtype)
    m = min(n, used)
    gu[m:], gh[m:] = float("nan"), float("nan")
    rng = torch.tensor([-5, 1 << 40])
    f = ref.factors(n, I, p, rng.tolist())
    g, u, d = gu[:, :I].double(), gu[:, I:].double(), gh.double() * f
    a, da = ref.act(g, kind)
    ta, tda = gate_tolerance(g, kind)
    h = f * a * u
    grad = torch.cat([d * u * da, d * a], 1)
    # products with u, the scale, the scale's own rounding
    tol_h = f * u.abs() * (ta + 3 * EPS * a.abs()) + half_step(h, dtype)
    tol = torch.cat([(d * u).abs() * (tda + 4 * EPS * da.abs()), d.abs() * (ta + 3 * EPS * a.abs())], 1) + half_step(grad, dtype)
    nan = float("nan")
    h[m:], grad[m:] = nan, nan

    def put(t):
        return offset_view(t, shift)

    num = torch.tensor([used], dtype=torch.int32, device="cuda")
    nans = lambda w: put(torch.full((n, w), nan).to(dtype))  # noqa: E731
    got = mr.expert_act(put(gu), num, act=kind, p=p, rng=rng.cuda(), h=nans(I))
    check(got, h, tol_h, "h")
    out = mr.expert_act_bwd(put(gh), put(gu), num, act=kind, p=p, rng=rng.cuda(), grad_gu=nans(2 * I), h=nans(I))
    check(out["grad_gu"], grad, tol, "grad_gu")
    check(out["h"], h, tol_h, "h again")
    less = mr.expert_act_bwd(put(gh), put(gu), num, act=kind, p=p, rng=rng.cuda(), need_h=False)
    assert set(less) == {"grad_gu"} and torch.equal(less["grad_gu"][:m], out["grad_gu"][:m])
    if m == n:  # without a count: all rows
        assert torch.equal(mr.expert_act(put(gu), act=kind, p=p, rng=rng.cuda()), got)


@pytest.mark.parametrize("kind", [0, 1], ids=["silu", "gelu"])
def test_activation_everywhere(mr, kind):
    """act and act' in fp32 at 2^19 gates from -16 to 16, up and grad_h being 1."""
    g = torch.linspace(-16, 16, 1 << 19).view(512, 1024)
    gu = torch.cat([g, torch.ones_like(g)], 1)
    a, da = ref.act(g.double(), kind)
    ta, tda = gate_tolerance(g.double(), kind)
    check(mr.expert_act(gu.cuda(), act=kind), a, ta, "h")
    out = mr.expert_act_bwd(torch.ones_like(g).cuda(), gu.cuda(), act=kind)
    check(out["grad_gu"], torch.cat([da, a], 1), torch.cat([tda, ta], 1), "grad_gu")


@pytest.mark.parametrize("p", [0.0, 2.0 ** -18, 0.1, 0.999, 1.0])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("T,H,shift", [(1, 1, 0), (3, 8, 0), (7, 31, 0), (50, 256, 1), (19, 1001, 0), (5, 9000, 0), (300, 520, 0)])
def test_dropout(mr, T, H, shift, dtype, p):
    gen = torch.Generator().manual_seed(T)
    x, res = torch.randn(T, H, generator=gen).to(dtype), torch.randn(T, H, generator=gen).to(dtype)
    rng = torch.tensor([1 << 62, -1])
    f = ref.factors(T, H, p, rng.tolist())
    xg, rg = offset_view(x, shift), rng.cuda()
    for residual in (None, res):
        want = x.double() * f + (0 if residual is None else residual.double())
        tol = 2 * EPS * (x.double() * f).abs() + EPS * want.abs() + half_step(want, dtype)
        check(mr.dropout(xg, p, rg, None if residual is None else offset_view(res, shift)), want, tol, "y")
    want = x.double() * f
    check(mr.dropout_bwd(xg, p, rg), want, 2 * EPS * want.abs() + half_step(want, dtype), "grad_x")
    # in place, of x and of the residual
    code = mr.MR_F32 if dtype is F32 else mr.MR_BF16
    want = mr.dropout(xg, p, rg, offset_view(res, shift))
    y, z = offset_view(x, shift), offset_view(res, shift)
    mr.moe_dropout_fwd(T, H, code, y, z, p, rg, y)
    mr.moe_dropout_fwd(T, H, code, xg, z, p, rg, z)
    assert torch.equal(y, want) and torch.equal(z, want)


@pytest.mark.parametrize("H", [264, 257])
def test_dropped_elements_are_zero_whatever_they_held(mr, H):
    rng = torch.tensor([3, 4])
    f = ref.factors(6, H, 0.5, rng.tolist())
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")])[torch.arange(6 * H) % 3].view(6, H)
    for dtype in (F32, BF16):
        x = bad.to(dtype).cuda()
        drop = (f == 0).cuda()
        assert (mr.dropout(x, 0.5, rng.cuda())[drop] == 0).all()
        assert (mr.expert_act(torch.cat([x, x], 1), p=0.5, rng=rng.cuda())[drop] == 0).all()
        out = mr.expert_act_bwd(x, torch.cat([x, x], 1), p=0.5, rng=rng.cuda())
        assert (out["h"][drop] == 0).all() and (out["grad_gu"][torch.cat([drop, drop], 1)] == 0).all()


def test_infinities_and_nan_pass(mr):
    """What is not dropped keeps the formula's infinities and NaN; a pair without a row adds nothing, not even NaN."""
    inf, nan = float("inf"), float("nan")
    rows = torch.tensor([[inf, nan, 1.0], [-inf, 1.0, 2.0], [nan, nan, nan]]).cuda()
    pair_row = torch.tensor([[0, 1], [0, -1], [-1, 1]], dtype=torch.int32, device="cuda")
    out = mr.combine(rows, pair_row, torch.ones(3, 2, device="cuda")).cpu()
    assert out[0, 0].isnan() and out[0, 1].isnan() and out[0, 2] == 3
    assert out[1, 0] == inf and out[2].tolist() == [-inf, 1.0, 2.0]
    big = torch.tensor([[100.0, -100.0, 1e30, -1e30]], device="cuda")
    for kind in (0, 1):
        h = mr.expert_act(torch.cat([big, torch.ones_like(big)], 1), act=kind).cpu()
        assert h[0, 0] == 100 and h[0, 2] == 1e30 and h[0, 1].abs() < 1e-30 and h[0, 3] == 0
        gr = mr.expert_act_bwd(torch.ones_like(big), torch.cat([big, torch.ones_like(big)], 1), act=kind)["grad_gu"].cpu()
        assert gr[0, 0] == 1 and gr[0, 2] == 1 and gr[0, 1].abs() < 1e-30 and gr[0, 3] == 0


def test_empty_and_nothing_kept(mr):
    z = lambda *s, d=F32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    i32 = torch.int32
    out = mr.permute(z(0, 16), z(0, 2, d=i32), 4, z(0, d=i32), z(1, d=i32))
    assert out["pair_row"].shape == (0, 2)
    assert mr.combine(z(8, 16), z(0, 2, d=i32), z(0, 2)).shape == (0, 16)
    assert mr.expert_act(z(0, 32)).shape == (0, 16) and mr.dropout(z(0, 8), 0.0, None).shape == (0, 8)
    # no row at all: tokens get their residual, or 0
    none = torch.full((5, 3), -1, dtype=i32, device="cuda")
    res = torch.randn(5, 16, device="cuda")
    assert torch.equal(mr.combine(z(0, 16), none, z(5, 3), residual=res), res)
    assert (mr.permute_bwd(z(0, 16), none) == 0).all()
    out = mr.permute(res, none, 4, z(0, d=i32), z(1, d=i32))
    assert out["rows"].shape == (0, 16) and (out["pair_row"] == -1).all()
    got = mr.combine_bwd(res, z(0, 16), none, z(5, 3), z(0, d=i32), z(1, d=i32))
    assert (got["grad_w"] == 0).all()


def test_rows_out_of_range_are_reported(mr):
    """Pair rows past the buffer count as none, rows past it are left out; both raise the status word."""
    dev, i32 = "cuda", torch.int32
    status = lambda: torch.zeros(1, dtype=i32, device=dev)  # noqa: E731
    rows, w = torch.randn(4, 64, device=dev), torch.ones(2, 2, device=dev)
    good = torch.tensor([[0, -1], [3, -1]], dtype=i32, device=dev)
    for bad in (4, 1 << 30, -2, -(1 << 31)):
        pr = good.clone()
        pr[1, 1] = bad
        s = status()
        assert torch.equal(mr.combine(rows, pr, w, status=s), mr.combine(rows, good, w)) and int(s) == mr.MR_ERANGE
        s = status()
        assert torch.equal(mr.permute_bwd(rows, pr, status=s), mr.permute_bwd(rows, good)) and int(s) == mr.MR_ERANGE
        s = status()
        ids = torch.tensor([0, 4, 4, 2], dtype=i32, device=dev)
        n = torch.tensor([4], dtype=i32, device=dev)
        a = mr.combine_bwd(rows[:2].contiguous(), rows, pr, w, ids, n, status=s)
        b = mr.combine_bwd(rows[:2].contiguous(), rows, good, w, ids, n)
        assert torch.equal(a["grad_rows"], b["grad_rows"]) and torch.equal(a["grad_w"], b["grad_w"]) and int(s) == mr.MR_ERANGE
    idx = torch.tensor([[0, 7], [1, 7]], dtype=i32, device=dev)
    x = torch.randn(2, 64, device=dev)
    for ids, n in (([0, 4, 2, 9], 4), ([0, -3, 2, 4], 4), ([0, 4, 2, 4], 5)):
        s = status()
        out = mr.permute(x, idx, 2, torch.tensor(ids, dtype=i32, device=dev), torch.tensor([n], dtype=i32, device=dev), status=s)
        assert int(s) == mr.MR_ERANGE
        assert torch.equal(out["rows"], torch.stack([x[0], x[0] * 0, x[1], x[0] * 0]))
        assert out["pair_row"].tolist() == [[0, -1], [2, -1]]


def test_same_expert_twice(mr):
    idx = torch.tensor([[2, 2], [1, 2]], dtype=torch.int32, device="cuda")
    srt = mr.sort(idx, torch.ones(2, 2, device="cuda"), 4, 4)
    x = torch.randn(2, 40, device="cuda")
    out = mr.permute(x, idx, 4, srt["sorted_token_ids"], srt["num_tokens_post_pad"])
    assert out["pair_row"].tolist() == [[4, 5], [0, 6]]
    assert torch.equal(mr.permute_bwd(out["rows"], out["pair_row"]), 2 * x)


def _layer(mr, x, idx, w, w13, w2, rng, p, block, kind):
    """A layer's forward pass and its gradients by hand, products per expert by torch."""
    E = len(w13)
    srt = mr.sort(idx, w, E, block)
    ids, n = srt["sorted_token_ids"], srt["num_tokens_post_pad"]
    per = mr.permute(x, idx, E, ids, n, rows=x.new_zeros(len(ids), x.shape[1]))
    owner = srt["expert_ids"].long().clamp(0, E - 1).repeat_interleave(block)[: len(ids)]
    owner = torch.where(torch.arange(len(ids), device=x.device) < n, owner, 0)  # rows behind are zeros
    gu = torch.einsum("rh,rih->ri", per["rows"], w13[owner])
    h = mr.expert_act(gu, n, act=kind, p=p, rng=rng[0], h=x.new_zeros(len(ids), w2.shape[2]))
    y = torch.einsum("ri,rhi->rh", h, w2[owner])
    out = mr.combine(y, per["pair_row"], w, residual=x, p=p, rng=rng[1])

    def backward(go):
        c = mr.combine_bwd(go, y, per["pair_row"], w, ids, n, p=p, rng=rng[1], grad_rows=torch.zeros_like(y))
        a = mr.expert_act_bwd(torch.einsum("rh,rhi->ri", c["grad_rows"], w2[owner]), gu, n, act=kind, p=p, rng=rng[0],
                              grad_gu=torch.zeros_like(gu), h=torch.zeros_like(h))
        sel = torch.nn.functional.one_hot(owner, E).to(x.dtype)
        gw2 = torch.einsum("re,rh,ri->ehi", sel, c["grad_rows"], a["h"])
        gw13 = torch.einsum("re,ri,rh->eih", sel, a["grad_gu"], per["rows"])
        gx = mr.permute_bwd(torch.einsum("ri,rih->rh", a["grad_gu"], w13[owner]), per["pair_row"]) + go
        return dict(x=gx, w=c["grad_w"], w13=gw13, w2=gw2)

    return out, backward, (srt, per)


@pytest.mark.parametrize("kind", [0, 1], ids=["silu", "gelu"])
@pytest.mark.parametrize("dropped", [False, True])
def test_a_layer_and_its_gradients(mr, kind, dropped):
    """Sort, permutation, activation and weighted sum as a training step uses them, between products by torch, against
    the whole layer in 64 bits with gradients by autograd (which are checked against differences). Sums of up to 48
    products follow one another six times, each off by less than 64 EPS of its terms' sizes, which these inputs keep
    below 64: 6 * 64 * 64 * EPS = 1.5e-3, taken as the bound."""
    T, k, E, H, I, block, p = 23, 3, 6, 48, 20, 4, 0.25
    gen = torch.Generator().manual_seed(5)
    x, w = torch.randn(T, H, generator=gen), torch.rand(T, k, generator=gen)
    w13, w2 = torch.randn(E, 2 * I, H, generator=gen) * H ** -0.5, torch.randn(E, H, I, generator=gen) * I ** -0.5
    idx = make_pairs(gen, T, k, E, 0.3 if dropped else 0.0)
    go = torch.randn(T, H, generator=gen)
    rng = torch.tensor([[11, 0], [11, 1]])
    back = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        c = [t.cuda() for t in (x, idx, w, w13, w2, rng)]
        out, backward, (srt, per) = _layer(mr, *c, p, block, kind)
        got = backward(go.cuda())
    finally:
        torch.backends.cuda.matmul.allow_tf32 = back

    _, n, pair_row = ref.sort(idx, E, block)
    f_row = ref.factors(n, I, p, rng[0].tolist())
    f_out = ref.factors(T, H, p, rng[1].tolist())

    def whole(x, w, w13, w2):
        total = torch.zeros(T, H, dtype=torch.float64)
        for t in range(T):
            for j in range(k):
                e, r = int(idx[t, j]), int(pair_row[t, j])
                if r >= 0:
                    gu = w13[e] @ x[t]
                    h = f_row[r] * ref.act(gu[:I], kind)[0] * gu[I:]
                    total[t] = total[t] + w[t, j] * (w2[e] @ h)
        return x + f_out * total

    leaves = [t.double().requires_grad_() for t in (x, w, w13, w2)]
    want = whole(*leaves)
    want.backward(go.double())
    check(out, want.detach(), torch.full_like(want, 1.5e-3), "out")
    for name, leaf in zip(("x", "w", "w13", "w2"), leaves):
        check(got[name], leaf.grad, torch.full_like(leaf.grad, 1.5e-3), name)
        step = torch.randn(leaf.shape, generator=gen, dtype=torch.float64)
        args = [t.detach() for t in leaves]
        i = [id(t) for t in leaves].index(id(leaf))
        up, down = (whole(*args[:i], args[i] + e * step, *args[i + 1:]) for e in (1e-5, -1e-5))
        slope = ((up - down) * go.double()).sum() / 2e-5
        assert abs(slope - (leaf.grad * step).sum()) < 1e-6 * (leaf.grad * step).abs().sum() + 1e-6


@pytest.mark.parametrize("overlap", [True, False])
def test_captured_and_replayed(mr, overlap):
    """A captured step gives what an eager one gives; the generator's state is read when the graph runs."""
    T, k, E, H, block = 70, 4, 16, 512, 16
    s = setup(mr, T, k, E, H, block, BF16)
    x, idx, w = s["x"].cuda(), s["idx"].cuda(), s["w"].cuda()
    rng = torch.tensor([5, 0], device="cuda")

    def step():
        srt = mr.sort(idx, w, E, block)
        ids, n = srt["sorted_token_ids"], srt["num_tokens_post_pad"]
        per = mr.permute(x, idx, E, ids, n)
        h = mr.expert_act(per["rows"], n, p=0.3, rng=rng)
        y = mr.expert_act_bwd(h, per["rows"], n, p=0.3, rng=rng)["grad_gu"]
        out = mr.dropout(mr.combine(y, per["pair_row"], w, residual=x, p=0.3, rng=rng), 0.3, rng)
        c = mr.combine_bwd(out, y, per["pair_row"], w, ids, n, p=0.3, rng=rng)
        return out, c["grad_w"], mr.permute_bwd(c["grad_rows"], per["pair_row"])

    mr.moe_router_set_launch_overlap(overlap)
    try:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            eager = []
            for o in (0, 1, 2):
                rng[1] = o
                eager.append([t.clone() for t in step()])
            rng[1] = 0
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out = step()
            rng[1] += 1
        for o in (0, 1, 2):
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, eager[o]):
                assert torch.equal(a, b), o
        assert not torch.equal(eager[0][0], eager[1][0])
    finally:
        mr.moe_router_set_launch_overlap(True)


def test_another_stream(mr):
    T, H = 4000, 1024
    st = torch.cuda.Stream()
    rng = torch.tensor([1, 2], device="cuda")
    x = torch.randn(T, H, device="cuda").to(BF16)
    want = mr.dropout(x, 0.5, rng)
    torch.cuda.synchronize()
    outs = [mr.dropout(x, 0.5, rng, stream=st) for _ in range(8)] + [mr.dropout(x, 0.5, rng, stream=st.cuda_stream)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_offsets_past_32_bits(mr):
    """Rows, tokens and activations whose elements lie past 2^31 (bf16, about 5 GB a buffer)."""
    n, H = 270001, 8192  # 2.2e9 elements
    rows = torch.zeros(n, H, dtype=BF16, device="cuda")
    at = [0, 1, 131072, 262144, 262145, 270000]
    vals = torch.randn(len(at), H).to(BF16)
    rows[at] = vals.cuda()
    pair_row = torch.tensor([at], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, 2.0, 4.0, 8.0, 16.0, 32.0]], device="cuda")
    terms = vals.double() * w.cpu().double().t()
    want = terms.sum(0, keepdim=True)
    check(mr.combine(rows, pair_row, w), want, 6 * EPS * terms.abs().sum(0) + half_step(want, BF16), "out")
    x = torch.randn(1, H).to(BF16)
    ids = torch.full((n,), 6, dtype=torch.int32, device="cuda")
    ids[at] = torch.arange(6, dtype=torch.int32, device="cuda")
    npp = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = mr.combine_bwd(x.cuda(), rows, pair_row, w, ids, npp)
    terms = vals.double() * x.double()
    check(got["grad_w"], terms.sum(1)[None], (H // 32 + 7) * EPS * terms.abs().sum(1)[None], "grad_w")
    assert torch.equal(got["grad_rows"][at].cpu(), (x.float() * w.cpu().t()).to(BF16))
    mask = torch.ones(n, dtype=torch.bool, device="cuda")
    mask[at] = False
    assert int(torch.count_nonzero(got["grad_rows"].view(torch.int16).view(n, H).amax(1)[mask])) == 0
    idx = torch.zeros(1, 6, dtype=torch.int32, device="cuda")
    out = mr.permute(x.cuda(), idx, 1, ids, npp, rows=got["grad_rows"])
    assert out["pair_row"].tolist() == [at] and torch.equal(out["rows"][at].cpu(), x.expand(6, H))
    rng = torch.tensor([1, 2], device="cuda")
    y = mr.dropout(out["rows"].fill_(1.0), 0.5, rng)
    f = ref.factors(at, H, 0.5, [1, 2])
    assert torch.equal(y[at].cpu().double(), f)
    h = mr.expert_act(rows.fill_(1.0), p=0.5, rng=rng)
    f = ref.factors(at, H // 2, 0.5, [1, 2])
    a = ref.act(torch.ones(1, dtype=torch.float64), 0)[0]
    check(h[at], f * a, 20 * EPS * f * a + half_step(f * a, BF16), "h")
