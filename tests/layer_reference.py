"""The experts' products and the adapter projection in 64 bits, element by element bounds included.

Each function returns (value, bound): the definition's value in double precision and how far a right bf16 kernel
may be from it. The bounds count roundings:

* u(bf16) = 2^-8 relative, for each rounding to bf16 (the stored h, the stored output);
* an fp32 sum of n products of bf16 values (the products are exact) is off by at most n * 2^-23 times the sum of
  the products' magnitudes (2^-23 an addition: the tensor cores may cut a sum off instead of rounding it);
* the activation and its product add a few fp32 roundings and errors of the exponential: 2^-20 relative;
* |d act / dg| <= 1.13 for SiLU and GELU, and |act(g)| <= |g|.
"""
import torch

U16, U32 = 2.0 ** -8, 2.0 ** -23


def act64(g, act):
    return g * torch.sigmoid(g) if act == 0 else 0.5 * g * (1 + torch.erf(g * 0.5 ** 0.5))


def experts64(x, idx, w, w13, w2, act=0):
    """x [T, H], idx / w [T, topk], w13 [E, 2I, H], w2 [E, H, I]: CPU tensors of any type."""
    x, w, w13, w2 = x.double(), w.double(), w13.double(), w2.double()
    (T, H), E, I, k = x.shape, w13.shape[0], w2.shape[2], idx.shape[1]
    out, err = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    mag = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        gu, ab = x[t] @ w13[e].t(), x[t].abs() @ w13[e].abs().t()
        d = H * U32 * ab
        g, u, dg, du = gu[:, :I], gu[:, I:], d[:, :I], d[:, I:]
        h = act64(g, act) * u
        dh = 1.13 * dg * (u.abs() + du) + g.abs() * du + 2.0 ** -20 * h.abs()
        dh = dh + U16 * (h.abs() + dh)
        wt = w[t, j][:, None]
        out.index_add_(0, t, (h @ w2[e].t()) * wt)
        top = (h.abs() + dh) @ w2[e].abs().t()
        err.index_add_(0, t, (dh @ w2[e].abs().t()) * wt.abs())
        mag.index_add_(0, t, top * wt.abs())
    err = err + (I + 2 * k) * U32 * mag
    return out, err + U16 * (out.abs() + err) + 1e-30


def adapter64(x, w, a, b, adapter, scale, bf16_out):
    x, w = x.double(), w.double()
    T, K = x.shape
    out, mag = x @ w.t(), x.abs() @ w.abs().t()
    err = torch.zeros_like(out)
    if a is not None:
        a, b = a.double(), b.double()
        n, r = a.shape[:2]
        for i in range(n):
            t = (adapter == i).nonzero()[:, 0]
            if len(t) == 0:
                continue
            sc = 1.0 if scale is None else float(scale[i].double())
            low, lmag = x[t] @ a[i].t() * sc, x[t].abs() @ a[i].abs().t() * abs(sc)
            # the rank-space values: an fp32 sum over K in parts, then 16 significant bits
            dlow = (K + 40) * U32 * lmag + 2.0 ** -16 * low.abs()
            out[t] += low @ b[i].t()
            err[t] += dlow @ b[i].abs().t()
            mag[t] += (low.abs() + dlow) @ b[i].abs().t()
        err = err + 3 * r * U32 * mag
    err = err + K * U32 * mag
    return out, (err + U16 * (out.abs() + err) if bf16_out else err + 2.0 ** -24 * out.abs()) + 1e-30


def assert_within(got, want, bound, what):
    g = got.detach().cpu().double()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    off = (g - want).abs()
    bad = ~(off <= bound)  # NaN counts as bad
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; first at {i}: "
                             f"{g[i].item()!r} against {want[i].item()!r}, bound {bound[i].item():.3e}")
