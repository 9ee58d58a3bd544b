"""The steps of a mixture-of-experts layer's training pass around the experts' matrix products, as they are measured.

Four operators, each with its gradient: ``permute`` (tokens to rows sorted by expert), ``combine`` (the rows back to
tokens, weighted, with dropout and a residual), ``act`` (the gated activation of the rows, with expert dropout) and
``dropout`` (of hidden states, with a residual). Dropout's masks come from a counter-based generator and are never
stored. Every case is a dict of sizes; the plain forms here are elementary torch operations in fp32, the framework's
own calls run where ``own`` is true.
"""
import math

import numpy
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


def _rows(name, op, T, E, topk, H, **kw):
    c = dict(op=op, bwd=False, T=T, E=E, topk=topk, H=H, block=64, dropped=0.0, zipf=0.0, dtype="bf16")
    if op == "combine":
        c.update(p=0.0, residual=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _act(name, rows, used, I, **kw):
    c = dict(op="act", bwd=False, rows=rows, used=used, I=I, gelu=False, p=0.0, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def _dropout(name, T, H, **kw):
    c = dict(op="dropout", bwd=False, T=T, H=H, p=0.1, residual=False, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # 16 tokens of a toy-sized layer (the repository's 8 experts, top-2): nothing but latency
        _rows("permute_T16_E8_k2", "permute", 16, 8, 2, 512, block=16, dtype="fp32"),
        # a training batch of 8192 tokens to 64 experts, eight each: every token's row is written eight times
        _rows("permute_T8192_E64_k8", "permute", 8192, 64, 8, 2048),
        # the gradient of 4096 tokens from the rows of 128 experts, skewed load
        _rows("permute_bwd_T4096_E128_k4", "permute", 4096, 128, 4, 2048, bwd=True, zipf=1.1),
        # one token's eight rows back, as a single decoding step does it
        _rows("combine_T1_E256_k8", "combine", 1, 256, 8, 2048, block=16),
        # a training batch's rows back to 8192 tokens, with the block's dropout and residual
        _rows("combine_T8192_E64_k8", "combine", 8192, 64, 8, 2048, p=0.1, residual=True),
        # gradients at odd sizes, some slots dropped (ids of -1) and some tokens left with none
        _rows("combine_bwd_T333_E100_k5", "combine", 333, 100, 5, 1001, bwd=True, block=16, dropped=0.3),
        # gradients of a training batch of wide tokens, with dropout
        _rows("combine_bwd_T8192_E64_k4", "combine", 8192, 64, 4, 4096, bwd=True, p=0.1),
        # the rows of a few tokens through GELU in fp32
        _act("act_R40_I344", 40, 37, 344, gelu=True, dtype="fp32"),
        # a training batch's rows with expert dropout; the buffer has room for more rows than are in use
        _act("act_R32768_I1024", 32768, 30016, 1024, p=0.4),
        # its gradient, with the activation computed again for the weights' gradient
        _act("act_bwd_R32768_I2048", 32768, 32000, 2048, bwd=True, p=0.1),
        # an odd hidden size: rows that start at any alignment
        _dropout("dropout_T1000_H1001", 1000, 1001, residual=True),
        # the gradient of a batch's hidden states
        _dropout("dropout_bwd_T16384_H4096", 16384, 4096, bwd=True),
    ]


def _logu(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(c):
    return work(c)["bytes"]


def _width(rng, lo, hi):
    """Widths of layers are multiples of 8 mostly, and anything sometimes."""
    n = _logu(rng, lo, hi)
    return n if rng.random() < 0.25 else max(8, n // 8 * 8)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["permute", "combine", "act", "dropout"])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        bwd, p = rng.random() < 0.5, rng.choice([0.0, 0.1, 0.4])
        if op == "act":
            rows = _logu(rng, 1, 32768)
            c = _act(None, rows, rows - int(rows * rng.uniform(0.0, 0.2)), _width(rng, 64, 4096), bwd=bwd, p=p,
                     gelu=rng.random() < 0.5, dtype=dtype)
        elif op == "dropout":
            c = _dropout(None, _logu(rng, 1, 16384), _width(rng, 64, 4096), bwd=bwd, p=p or 0.05,
                         residual=not bwd and rng.random() < 0.5, dtype=dtype)
        else:
            T, E = _logu(rng, 1, 16384), _logu(rng, 4, 384)
            c = _rows(None, op, T, E, min(E, rng.randint(1, 9)), _width(rng, 64, 4096), bwd=bwd, dtype=dtype,
                      block=rng.choice([1, 16, 32, 64, 128]), zipf=rng.choice([0.0, 1.1]),
                      dropped=rng.choice([0.0, 0.0, 0.3]) if T >= 16 else 0.0)
            if op == "combine":
                c.update(p=p, residual=not bwd and rng.random() < 0.5)
        if _cost(c) <= most:
            return c


# ---- inputs ----------------------------------------------------------------------------------------------------


def _sorted(idx, E, block):
    """The router's sort: pairs by expert in blocks of `block` rows. Ids (T * topk at padding), their number, and each
    pair's row (-1 where its expert is none of ours)."""
    P = idx.numel()
    e = idx.reshape(-1).long()
    e = torch.where((e >= 0) & (e < E), e, torch.full_like(e, E))
    order = torch.argsort(e, stable=True)
    count = torch.bincount(e, minlength=E + 1)[:E]
    pad = (count + block - 1) // block * block
    first, start = count.cumsum(0) - count, pad.cumsum(0) - pad
    kept = order[: int(count.sum())]
    row = start[e[kept]] + torch.arange(len(kept), device=idx.device) - first[e[kept]]
    cap = P + min(P, E) * (block - 1)
    ids = torch.full((cap,), P, dtype=torch.int32, device=idx.device)
    ids[row] = kept.to(torch.int32)
    pair_row = torch.full((P,), -1, dtype=torch.int32, device=idx.device)
    pair_row[kept] = row.to(torch.int32)
    return ids, pad.sum().to(torch.int32).reshape(1), pair_row.view(idx.shape)


def prepare(case, seed):
    c, gen = dict(case), torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = F32 if c["dtype"] == "fp32" else BF16

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    s = dict(case=c)
    # the generator's key and the step's counter
    s["rng"] = torch.randint(-(1 << 62), 1 << 62, (2,), generator=gen, device="cuda")
    if c["op"] == "dropout":
        s["x"] = rand(c["T"], c["H"])
        s["residual"] = rand(c["T"], c["H"]) if c["residual"] else None
        return s
    if c["op"] == "act":
        s["gu"] = rand(c["rows"], 2 * c["I"])
        s["used"] = torch.tensor([c["used"]], dtype=torch.int32, device="cuda")
        if c["bwd"]:
            s["grad_h"] = rand(c["rows"], c["I"])
            s["grad_gu"] = torch.zeros_like(s["gu"])
        s["h"] = torch.zeros(c["rows"], c["I"], dtype=dtype, device="cuda")
        return s
    T, E, k, H = c["T"], c["E"], c["topk"], c["H"]
    logits = torch.randn(T, E, generator=gen, device="cuda")
    if c["zipf"]:
        rank = torch.randperm(E, generator=gen, device="cuda") + 1
        logits = logits - c["zipf"] * torch.log(rank.float())
    top = logits.topk(k, dim=1)
    idx = top.indices.to(torch.int32)
    if c["dropped"]:
        gone = torch.rand(T, k, generator=gen, device="cuda") < c["dropped"]
        gone[1 :: max(2, T // 8)] = True  # tokens whose experts all live elsewhere
        idx = torch.where(gone, torch.full_like(idx, -1), idx)
    s["topk_idx"], s["topk_w"] = idx.contiguous(), torch.softmax(top.values, dim=1).contiguous()
    s["ids"], s["used"], s["pair_row"] = _sorted(idx, E, c["block"])
    if c["op"] == "permute" and not c["bwd"]:
        s["x"] = rand(T, H)
        s["rows"] = torch.zeros(len(s["ids"]), H, dtype=dtype, device="cuda")
        return s
    s["rows"] = rand(len(s["ids"]), H)  # the experts' outputs, or the gradients of their inputs
    if c["op"] == "combine" and c["bwd"]:
        s["grad_out"] = rand(T, H)
        s["grad_rows"] = torch.zeros_like(s["rows"])
    elif c["op"] == "combine":
        s["residual"] = rand(T, H) if c["residual"] else None
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------


def _bits(rows, cols, rng):
    """16 random bits for each element: Philox 4x32 with 10 rounds (Salmon et al., "Parallel random numbers: as easy as
    1, 2, 3"); its key is the seed, its counter (column / 8, row, offset), eight elements to a block."""
    low = 0xFFFFFFFF
    a = torch.arange((cols + 7) // 8, device=rng.device)[None, :].expand(rows, -1)
    b = torch.arange(rows, device=rng.device)[:, None].expand(-1, a.shape[1])
    key, more = rng[0], rng[1]
    c, d = (more & low).expand_as(a), (more >> 32 & low).expand_as(a)
    k0, k1 = key & low, key >> 32 & low
    for _ in range(10):
        x, y = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (y >> 32 & low) ^ b ^ k0, y & low, (x >> 32 & low) ^ d ^ k1, x & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    words = torch.stack([a, b, c, d], 2)
    return torch.stack([words & 0xFFFF, words >> 16], 3).view(rows, -1)[:, :cols]


def _drop(x, p, rng):
    """Dropout of fp32 x [rows, cols]: elements whose 16 bits are below p * 2^16 become 0, the others grow to match."""
    cut = int(p * 65536 + 0.5)
    if cut == 0:
        return x
    keep = _bits(x.shape[0], x.shape[1], rng) >= cut
    return torch.where(keep, x * (65536 / (65536 - cut)), torch.zeros_like(x))


def _plain_permute(s):
    c, x = s["case"], s["x"]
    P = c["T"] * c["topk"]
    at = torch.arange(len(s["ids"]), device=x.device)
    real = (at < s["used"]) & (s["ids"] < P)
    take = x.float()[torch.where(real, s["ids"] // c["topk"], torch.zeros_like(s["ids"])).long()]
    rows = torch.where(real[:, None], take, torch.zeros_like(take)).to(x.dtype)
    pair_row = torch.full((P + 1,), -1, dtype=torch.int32, device=x.device)
    pair_row[torch.where(real, s["ids"], torch.full_like(s["ids"], P)).long()] = at.to(torch.int32)
    return dict(rows=rows, pair_row=pair_row[:P].view(c["T"], c["topk"]))


def _mine(s):
    """The rows of each token's pairs [T, topk, H] in fp32, zeros for dropped pairs."""
    got = s["rows"].float()[s["pair_row"].clamp(min=0).long()]
    return torch.where((s["pair_row"] >= 0)[:, :, None], got, torch.zeros_like(got))


def _plain_combine(s):
    c = s["case"]
    out = _drop((_mine(s) * s["topk_w"][:, :, None]).sum(1), c["p"], s["rng"])
    if c["residual"]:
        out = out + s["residual"].float()
    return out.to(s["rows"].dtype)


def _plain_combine_bwd(s):
    c = s["case"]
    P = c["T"] * c["topk"]
    g = _drop(s["grad_out"].float(), c["p"], s["rng"])
    grad_w = (_mine(s) * g[:, None, :]).sum(2)
    pairs = (s["topk_w"][:, :, None] * g[:, None, :]).view(P, -1)
    at = torch.arange(len(s["ids"]), device=g.device)
    real = (at < s["used"]) & (s["ids"] < P)
    take = pairs[torch.where(real, s["ids"], torch.zeros_like(s["ids"])).long()]
    grad_rows = torch.where(real[:, None], take, torch.zeros_like(take)).to(s["rows"].dtype)
    return dict(grad_rows=grad_rows, grad_w=grad_w)


def _gate(g, gelu):
    """act(g) and its derivative."""
    if gelu:
        cdf = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    sig = 1 / (1 + torch.exp(-g))
    return g * sig, sig * (1 + g * (1 - sig))


def _plain_act(s):
    c, gu = s["case"], s["gu"]
    g, u = gu[:, : c["I"]].float(), gu[:, c["I"] :].float()
    used = (torch.arange(len(gu), device=gu.device) < s["used"])[:, None]
    a, da = _gate(g, c["gelu"])
    h = torch.where(used, _drop(a * u, c["p"], s["rng"]), torch.zeros_like(g)).to(gu.dtype)
    if not c["bwd"]:
        return h
    d = torch.where(used, _drop(s["grad_h"].float(), c["p"], s["rng"]), torch.zeros_like(g))
    return dict(grad_gu=torch.cat([d * u * da, d * a], 1).to(gu.dtype), h=h)


def _plain_dropout(s):
    c = s["case"]
    y = _drop(s["x"].float(), c["p"], s["rng"])
    if c["residual"]:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def run(s):
    c = s["case"]
    if own:
        import top_gating_expert_row_gb300 as mr

        if c["op"] == "permute":
            if c["bwd"]:
                return mr.permute_bwd(s["rows"], s["pair_row"])
            return mr.permute(s["x"], s["topk_idx"], c["E"], s["ids"], s["used"], rows=s["rows"])
        if c["op"] == "combine":
            if c["bwd"]:
                return mr.combine_bwd(s["grad_out"], s["rows"], s["pair_row"], s["topk_w"], s["ids"], s["used"],
                                      p=c["p"], rng=s["rng"], grad_rows=s["grad_rows"])
            return mr.combine(s["rows"], s["pair_row"], s["topk_w"], residual=s["residual"], p=c["p"], rng=s["rng"])
        if c["op"] == "act":
            kind = mr.MR_GELU if c["gelu"] else mr.MR_SILU
            if c["bwd"]:
                return mr.expert_act_bwd(s["grad_h"], s["gu"], s["used"], act=kind, p=c["p"], rng=s["rng"],
                                         grad_gu=s["grad_gu"], h=s["h"])
            return mr.expert_act(s["gu"], s["used"], act=kind, p=c["p"], rng=s["rng"], h=s["h"])
        if c["bwd"]:
            return mr.dropout_bwd(s["x"], c["p"], s["rng"])
        return mr.dropout(s["x"], c["p"], s["rng"], residual=s["residual"])
    if c["op"] == "dropout":
        return _plain_dropout(s)
    if c["op"] == "act":
        return _plain_act(s)
    if c["op"] == "permute":
        return _mine(s).sum(1).to(s["rows"].dtype) if c["bwd"] else _plain_permute(s)
    return _plain_combine_bwd(s) if c["bwd"] else _plain_combine(s)


def work(case):
    c = case
    size = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "dropout":
        n = c["T"] * c["H"]
        return {"bytes": n * size * (3 if c["residual"] else 2), "flops": 2.0 * n}
    if c["op"] == "act":
        n = c["used"] * c["I"]
        return {"bytes": n * size * (6 if c["bwd"] else 3), "flops": (16.0 if c["bwd"] else 7.0) * n}
    T, E, k, H = c["T"], c["E"], c["topk"], c["H"]
    pairs = T * k * (1 - c["dropped"])
    # padding of each expert that has a pair: half a block (experts taken as evenly loaded)
    pad = E * (1 - (1 - 1 / E) ** pairs) * (c["block"] - 1) / 2
    token, row = T * H * size, pairs * H * size
    if c["op"] == "permute":
        if c["bwd"]:
            return {"bytes": row + T * k * 4 + token, "flops": pairs * H}
        return {"bytes": token + T * k * 8 + (pairs + pad) * (H * size + 4), "flops": 0.0}
    if c["bwd"]:
        return {"bytes": token + 2 * row + pad * H * size + (pairs + pad) * 4 + T * k * 12, "flops": 3.0 * pairs * H}
    return {"bytes": row + T * k * 8 + token * (2 if c["residual"] else 1), "flops": 2.0 * pairs * H}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------


def _factors(s, rows, cols):
    """What dropout multiplies each element with, from the generator's definition on the host's unsigned words."""
    cut = int(s["case"]["p"] * 65536 + 0.5)
    if cut == 0:
        return torch.ones(rows, cols, dtype=torch.float64, device="cuda")
    seed, offset = (int(v) % (1 << 64) for v in s["rng"].tolist())
    u, mask = numpy.uint64, numpy.uint64(0xFFFFFFFF)
    blocks = -(-cols // 8)
    at = numpy.arange(rows * blocks, dtype=u)
    ctr = [at % u(blocks), at // u(blocks), numpy.full(len(at), offset % (1 << 32), u), numpy.full(len(at), offset >> 32, u)]
    key = [seed % (1 << 32), seed >> 32]
    for turn in range(10):
        left, right = u(0xD2511F53) * ctr[0], u(0xCD9E8D57) * ctr[2]
        ctr = [(right >> u(32)) ^ ctr[1] ^ u(key[0]), right & mask, (left >> u(32)) ^ ctr[3] ^ u(key[1]), left & mask]
        key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
    half = numpy.empty((len(at), 8), numpy.uint16)
    for i, word in enumerate(ctr):
        half[:, 2 * i] = word & u(0xFFFF)
        half[:, 2 * i + 1] = word >> u(16)
    kept = torch.from_numpy((half.reshape(rows, -1)[:, :cols] >= cut)).cuda()
    return kept.double() * (65536.0 / (65536.0 - cut))


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "dropout":
        y = s["x"].double() * _factors(s, c["T"], c["H"])
        return y + s["residual"].double() if c["residual"] else y
    if c["op"] == "act":
        n, I = c["used"], c["I"]
        g, u = s["gu"][:n, :I].double(), s["gu"][:n, I:].double()
        f = _factors(s, n, I)
        if c["gelu"]:
            phi = torch.special.ndtr(g)
            a, da = g * phi, phi + g * torch.exp(g.square() / -2) / math.sqrt(2 * math.pi)
        else:
            t = torch.tanh(g / 2)  # the sigmoid is (1 + t) / 2
            a, da = g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) / 4
        h = torch.zeros(c["rows"], I, dtype=torch.float64, device="cuda")
        h[:n] = f * a * u
        if not c["bwd"]:
            return h
        grad = torch.zeros(c["rows"], 2 * I, dtype=torch.float64, device="cuda")
        d = s["grad_h"][:n].double() * f
        grad[:n, :I], grad[:n, I:] = d * u * da, d * a
        return dict(grad_gu=grad, h=h)
    T, k, H = c["T"], c["topk"], c["H"]
    if c["op"] == "permute" and not c["bwd"]:
        rows = torch.zeros(len(s["ids"]), H, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = (s["pair_row"][:, j] >= 0).nonzero()[:, 0]
            rows[s["pair_row"][t, j].long()] = s["x"][t].double()
        return dict(rows=rows, pair_row=None)
    if c["op"] == "combine" and c["bwd"]:
        g = s["grad_out"].double() * _factors(s, T, H)
        grad_rows = torch.zeros(len(s["ids"]), H, dtype=torch.float64, device="cuda")
        grad_w = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = (s["pair_row"][:, j] >= 0).nonzero()[:, 0]
            r = s["pair_row"][t, j].long()
            grad_rows[r] = g[t] * s["topk_w"][t, j].double()[:, None]
            grad_w[t, j] = torch.einsum("th,th->t", g[t], s["rows"][r].double())
        return dict(grad_rows=grad_rows, grad_w=grad_w)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = (s["pair_row"][:, j] >= 0).nonzero()[:, 0]
        w = s["topk_w"][t, j].double() if c["op"] == "combine" else torch.ones(len(t), dtype=torch.float64, device="cuda")
        out[t] += s["rows"][s["pair_row"][t, j].long()].double() * w[:, None]
    if c["op"] == "combine":
        out *= _factors(s, T, H)
        if c["residual"]:
            out += s["residual"].double()
    return out
