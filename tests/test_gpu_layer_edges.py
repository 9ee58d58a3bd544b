"""Edges of the experts' products, the layer and the adapter projection on the GPU: values far from the usual, the bits
that intermediate values keep, sizes at which rings wrap and units follow one another."""
import pytest
import torch

from layer_reference import assert_within
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
