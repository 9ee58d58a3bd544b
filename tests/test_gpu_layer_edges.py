"""Edges of the experts' products, the layer and the adapter projection on the GPU: values far from the usual, the bits
that intermediate values keep, sizes at which rings wrap and units follow one another."""
import pytest
import torch

from layer_reference import assert_within, experts64
from test_gpu_layer import make_adapters, make_experts, shifted

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# ---- infinite weights ---------------------------------------------------------------------------------------------

# a few pairs, narrow blocks (16, 32 and 64 pairs), blocks of 128 and 256, rows for the plain kernels
INFINITE = [(1, 4, 2, 64, 32), (16, 64, 2, 128, 64), (40, 16, 2, 128, 64), (40, 8, 2, 128, 64), (100, 8, 2, 128, 64),
            (700, 4, 2, 128, 64), (40, 8, 2, 33, 17)]


@pytest.mark.parametrize("size", INFINITE, ids=lambda s: "T%d_E%d_k%d_H%d_I%d" % s)
def test_an_infinite_weight_gives_an_infinity(mr, size):
    """One infinite element of w2: h_i * inf + (finite) is an infinity of h_i's sign, on every path."""
    x, idx, w, w13, w2 = make_experts(*size, seed=11)
    T, E, k, H, I = size
    e, row, i = int(idx[0, 0]), 3, 5
    clean = mr.experts(*[t.cuda() for t in (x, idx, w, w13, w2)]).cpu()
    w2[e, row, i] = float("inf")
    got = mr.experts(*[t.cuda() for t in (x, idx, w, w13, w2)]).cpu()
    gu = x.double() @ w13[e].double().t()
    sign = torch.sign(gu[:, i] * gu[:, I + i])  # of h: SiLU has its argument's sign
    hit = (idx == e).any(1)
    assert (sign != 0).all()
    want = clean.clone()
    want[hit, row] = (sign[hit] * float("inf")).to(BF16)
    assert torch.equal(got, want)


# T, K, N, rank, adapters, out: one token, tiles of at most 64 tokens, wide tiles of one adapter, the plain kernels
INFINITE_ADAPTERS = [(1, 64, 40, 8, 2, F32), (20, 256, 128, 16, 2, BF16), (300, 128, 72, 24, 2, F32),
                     (20000, 64, 128, 64, 1, BF16), (40000, 64, 128, 40, 1, BF16), (20, 33, 17, 9, 2, F32)]


@pytest.mark.parametrize("case", INFINITE_ADAPTERS, ids=lambda c: "T%d_K%d_N%d_r%d_n%d" % c[:5])
def test_an_infinite_element_of_b_gives_an_infinity(mr, case):
    *size, out = case
    x, w, a, b, _, sc = make_adapters(*size, seed=12)
    ad = torch.zeros(size[0], dtype=torch.int32)
    clean = mr.adapter_proj(*[t.cuda() for t in (x, w, a, b, ad, sc)], out_dtype=out).cpu()
    row, q = 5, 7
    b[0, row, q] = float("inf")
    got = mr.adapter_proj(*[t.cuda() for t in (x, w, a, b, ad, sc)], out_dtype=out).cpu()
    low = x.double() @ a[0, q].double()
    # a sum over K in fp32 has the sign of the exact one unless it is next to zero
    sure = low.abs() > size[1] * 2.0 ** -23 * (x.double().abs() @ a[0, q].double().abs())
    assert sure.double().mean() > 0.999
    want = clean.clone()
    want[:, row] = (torch.sign(low) * float("inf")).to(out)
    assert torch.equal(got[sure], want[sure])


# ---- gates far below zero -----------------------------------------------------------------------------------------


@pytest.mark.parametrize("size", [(1, 2, 1, 64, 40), (12, 4, 1, 64, 40), (90, 4, 2, 64, 40), (9, 3, 2, 33, 41)],
                         ids=lambda s: "T%d_E%d_k%d_H%d_I%d" % s)
def test_gelu_of_gates_below_zero(mr, size):
    """g * Phi(g) for g in [-6, -2] to bf16's precision: 1 + erf(g / sqrt 2) would leave 10 bits at -4 and none at -6.

    x picks one column of w13, so g and u are exact, and w2 is the identity, so out is h rounded to bf16 (half a step:
    2^-8 relative) once, or twice in blocks of more than 64 pairs. h itself: erfc to 2^-20 and its argument to 2^-23,
    which |g|^2 <= 36 times enters the value: 2^-17.5; two parts: 2^-16. In all below 2^-7 + 2^-13."""
    T, E, k, H, I = size
    x, idx, w, w13, w2 = make_experts(*size, seed=13)
    x = torch.zeros_like(x)
    x[:, 2] = 1
    w13[:, :I, 2] = torch.linspace(-6, -2, I).to(BF16)
    w13[:, I:, 2] = 1
    n = min(H, I)
    w2 = torch.zeros_like(w2)
    w2[:, range(n), range(n)] = 1
    idx = idx[:, :1].contiguous()
    w = torch.ones_like(w[:, :1])
    got = mr.experts(*[t.cuda() for t in (x, idx, w, w13, w2)], act=mr.MR_GELU).cpu().double()
    g = w13[0, :n, 2].double()
    want = (0.5 * g * torch.special.erfc(-g * 0.5 ** 0.5)).expand(T, n)
    off = ((got[:, :n] - want) / want).abs().max().item()
    assert off <= 2.0 ** -7 + 2.0 ** -13, off
    assert not got[:, n:].any()


# ---- the bits that intermediate values keep -------------------------------------------------------------------------


def cancelling_experts(T, E, k, H, I, seed):
    """h's values two and two almost alike (gate rows that differ by one bf16 step of one element, the same up rows),
    and w2 takes their differences: about 2^-9 of the values. Eight elements of x, so that sums over H are short."""
    x, idx, w, w13, w2 = make_experts(T, E, k, H, I, seed)
    x[:, 8:] = 0
    w13 = w13 * 2
    n = min(I // 2, H)
    gate, up = w13[:, :I], w13[:, I:]
    gate[:, 1:2 * n:2] = gate[:, 0:2 * n:2]
    up[:, 1:2 * n:2] = up[:, 0:2 * n:2]
    first = gate[:, 1:2 * n:2, 0].contiguous()
    gate[:, 1:2 * n:2, 0] = (first.view(torch.int16) + 1).view(BF16)
    w2 = torch.zeros_like(w2)
    w2[:, range(n), range(0, 2 * n, 2)] = 1
    w2[:, range(n), range(1, 2 * n, 2)] = -1
    return x, idx, w, w13, w2


def experts_by_pair(x, idx, w, w13, w2, unit):
    """In 64 bits (value, bound for h off by at most `unit` of itself, the value with h rounded to bf16)."""
    x, w, w13, w2 = x.double(), w.double(), w13.double(), w2.double()
    T, H = x.shape
    I = w2.shape[2]
    out, err, short = [torch.zeros(T, H, dtype=torch.float64) for _ in range(3)]
    for t in range(T):
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            gu, mag = w13[e] @ x[t], w13[e].abs() @ x[t].abs()
            g, u = gu[:I], gu[I:]
            d = 8 * 2.0 ** -23 * mag  # fp32 sums of eight products
            h = g * torch.sigmoid(g) * u
            dh = 1.13 * d[:I] * (u.abs() + d[I:]) + g.abs() * d[I:] + (2.0 ** -20 + unit) * h.abs()
            out[t] += w[t, j] * (w2[e] @ h)
            short[t] += w[t, j] * (w2[e] @ h.to(BF16).double())
            # sums of a few values of |h| in fp32
            err[t] += w[t, j] * (w2[e].abs() @ (dh + 8 * 2.0 ** -23 * h.abs()))
    return out, err + 2.0 ** -8 * (out.abs() + err) + 1e-30, short


# a few pairs; blocks of 16, 32 and 64 pairs; odd rows (plain kernels)
@pytest.mark.parametrize("size", [(1, 4, 2, 64, 32), (20, 64, 1, 64, 32), (30, 8, 2, 64, 32), (60, 8, 2, 128, 64),
                                  (3, 4, 2, 33, 18), (60, 8, 2, 65, 30)], ids=lambda s: "T%d_E%d_k%d_H%d_I%d" % s)
def test_h_keeps_sixteen_bits(mr, size):
    v = cancelling_experts(*size, seed=14)
    got = mr.experts(*[t.cuda() for t in v])
    want, bound, short = experts_by_pair(*v, unit=2.0 ** -16)
    assert ((short - want).abs() > 2 * bound).any()  # eight bits are told from sixteen
    assert_within(got, want, bound, "out")


def test_h_keeps_sixteen_bits_at_unaligned_bases(mr):
    v = cancelling_experts(5, 4, 2, 64, 32, seed=15)
    want, bound, _ = experts_by_pair(*v, unit=2.0 ** -16)
    assert_within(mr.experts(*[shifted(t.cuda(), 1) for t in v]), want, bound, "out")


# K shared by a cluster, and K in one CTA
@pytest.mark.parametrize("T,N", [(8, 512), (100, 512), (32, 10240), (100, 6000), (300, 2048)])
def test_fp32_projection_of_4096(mr, T, N):
    """The tensor cores' sum loses last bits: 4.4e-6 of the output's norm when it runs over all of K = 4096 and 4.7e-7
    over parts of 512, against 2.4e-7 with the parts of 256 that fp32 outputs take."""
    x, w, *_ = make_adapters(T, 4096, N, 8, 1, seed=16)
    want = x.double() @ w.double().t()
    got = mr.adapter_proj(x.cuda(), w.cuda(), out_dtype=F32).cpu().double()
    assert ((got - want).norm() / want.norm()).item() <= 3.5e-7


# ---- rings that wrap, accumulators handed back, units one after another -----------------------------------------------


# pairs of CTAs with 16 and more steps of K a unit and several units a pair, the last row tile without a second one;
# single CTAs with as many; one token below and above what the CUDA cores take
@pytest.mark.parametrize("size", [(6000, 4, 2, 2048, 1024), (5000, 3, 2, 1096, 1160), (3000, 40, 2, 1536, 1024),
                                  (800, 60, 4, 1024, 1024), (48, 200, 8, 1032, 1160), (1, 32, 8, 2048, 1024), (1, 8, 4, 2560, 2048)],
                         ids=lambda s: "T%d_E%d_k%d_H%d_I%d" % s)
def test_experts_of_real_sizes(mr, size):
    """Against the definition in 64 bits, by the norm of each token's row: rounding the output and h to bf16
    (2^-8 at most, 2^-8 / sqrt 3 in the mean, each) stays below 2^-8 over a row of a thousand; a lost or stale step of
    K is a tenth or more."""
    T, E, k, H, I = size
    x, idx, w, w13, w2 = [t.cuda() for t in make_experts(*size, seed=17)]
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            gu = x[t].double() @ w13[e].double().t()
            h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
            want.index_add_(0, t, (h @ w2[e].double().t()) * w[t, j, None].double())
    first = mr.experts(x, idx, w, w13, w2)
    off = (first.double() - want).norm(dim=1) / want.norm(dim=1)
    assert off.max().item() <= 2.0 ** -8
    for _ in range(3):
        assert torch.equal(mr.experts(x, idx, w, w13, w2), first)


def whole_adapters(T, K, N, r, n, segment, seed=18):
    """Small whole numbers: every sum is exact in fp32, and the rank-space values fit 16 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(top, *shape):
        return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(BF16)

    x, w, a, b = rand(2, T, K), rand(2, N, K), rand(1, n, r, K), rand(1, n, N, r)
    scale = 2.0 ** torch.randint(-1, 2, (n,), generator=g, device="cuda").float()
    ad = torch.randint(-1, n, (-(-T // segment),), generator=g, device="cuda", dtype=torch.int32)
    ad[0] = n - 1
    ad = ad.repeat_interleave(segment)[:T].contiguous()
    want = x.double() @ w.double().t()
    for i in range(n):
        t = (ad == i).nonzero()[:, 0]
        low = x[t].double() @ a[i].double().t() * scale[i].double()
        assert not len(t) or low.abs().max().item() < 2 ** 15  # halves among them
        want[t] += low @ b[i].double().t()
    assert want.abs().max().item() < 2 ** 22
    return (x, w, a, b, ad, scale), want


WHOLE = [
    # T, K, N, rank, adapters, segment, out
    # wide tiles (256 and 128 tokens) with many steps of K and several slices of the rank-space values: one adapter a
    # tile, requests that end inside tiles, one a token
    (4096, 1024, 4096, 64, 8, 512, BF16), (4096, 1024, 4096, 64, 8, 300, BF16), (4096, 1096, 4100, 128, 5, 4096, BF16),
    (2048, 1544, 1536, 40, 6, 500, BF16), (2000, 1024, 1536, 64, 30, 1, BF16), (4096, 2048, 2304, 8, 3, 256, BF16),
    # rank-space values on the tensor cores in tiles of 16, 32 and 64 tokens
    (16, 40960, 256, 128, 3, 1, F32), (32, 20480, 200, 128, 40, 1, F32), (64, 8200, 256, 128, 64, 1, BF16),
    (700, 2048, 512, 64, 9, 100, F32), (3600, 1104, 512, 32, 16, 29, F32), (3600, 1104, 256, 32, 4, 600, F32),
    # a K for each CTA of a cluster, and units one after another without one
    (40, 4096, 1024, 16, 40, 1, F32), (64, 1024, 20000, 16, 5, 7, F32), (2500, 520, 2048, 24, 6, 111, F32),
]


@pytest.mark.parametrize("case", WHOLE, ids=lambda c: "T%d_K%d_N%d_r%d_n%d_s%d" % c[:6])
def test_adapter_sums_of_whole_numbers_are_exact(mr, case):
    *size, out = case
    v, want = whole_adapters(*size)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = mr.adapter_proj(*v, out_dtype=out, status=status)
    assert torch.equal(first, want.to(out))
    assert int(status.item()) == 0
    for _ in range(3):
        assert torch.equal(mr.adapter_proj(*v, out_dtype=out), first)


def test_layer_with_bias_and_groups_against_the_oracle(mr, orc):
    T, E, k, H, I = 50, 64, 9, 128, 64
    x, _, _, w13, w2 = make_experts(T, E, k, H, I, seed=19, E_tot=E + 1)
    g = torch.Generator().manual_seed(20)
    logits, bias = torch.randn(T, E, generator=g), torch.rand(E, generator=g) - 0.5
    for opts in (dict(n_shared=1, renorm=1, scaling=2.5), dict(n_shared=1, n_group=8, topk_group=4, renorm=1)):
        got = mr.layer(x.cuda(), logits.cuda(), k, w13.cuda(), w2.cuda(), score_fn=mr.MR_SIGMOID, bias=bias.cuda(), **opts)
        ref = orc.router_fwd(logits.numpy(), k, 1, 1, opts.get("n_group", 0), opts.get("topk_group", 0), 1,
                             opts.get("scaling", 1.0), 1.0, bias.numpy())
        assert torch.equal(got["topk_idx"].cpu(), torch.from_numpy(ref["topk_idx"]).to(torch.int32))
        weights = torch.from_numpy(ref["topk_w"])
        assert torch.allclose(got["topk_w"].cpu().double(), weights.double(), rtol=1e-6, atol=1e-7)
        want, bound = experts64(x, got["topk_idx"].cpu(), got["topk_w"].cpu(), w13, w2)
        assert_within(got["out"], want, bound, "out")
