"""The experts' products of a mixture-of-experts layer and the adapter projection, as they are measured.

Three operators: ``layer`` (router logits to the layer's output), ``experts`` (the same from a given choice of
experts) and ``adapter`` (a shared projection with a low-rank adapter per request). Every case is a dict of sizes;
the plain forms here are elementary torch operations in fp32, the framework's own calls run where ``own`` is true.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


def _layer(name, T, E, topk, H, I, **kw):
    c = dict(op="layer", T=T, E=E, topk=topk, H=H, I=I, sigmoid=False, renorm=True, scaling=1.0, shared=0,
             logits="bf16", zipf=0.0)
    c.update(kw)
    return dict(c, name=name) if name else c


def _experts(name, T, E, topk, H, I, **kw):
    c = dict(op="experts", T=T, E=E, topk=topk, H=H, I=I, dropped=0.0)
    c.update(kw)
    return dict(c, name=name) if name else c


def _adapter(name, T, K, N, rank, adapters, **kw):
    c = dict(op="adapter", T=T, K=K, N=N, rank=rank, adapters=adapters, segment=1, none=0.0, out="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through a toy-sized layer (the repository's 8 experts, top-2): nothing but latency
        _layer("layer_T1_E8_k2", 1, 8, 2, 512, 256, logits="fp32"),
        # single-token decode, 256 experts top-8: eight experts' weights stream once
        _layer("layer_T1_E256_k8", 1, 256, 8, 2048, 768),
        # a decode batch of 16 requests of the same layer: about 100 experts have one or two tokens each
        _layer("layer_T16_E256_k8", 16, 256, 8, 2048, 768),
        # a larger decode batch, 128 experts top-4, sigmoid scores: most experts are active with a few tokens
        _layer("layer_T64_E128_k4", 64, 128, 4, 2048, 1024, sigmoid=True, scaling=2.5),
        # the largest "few tokens": 384 routed experts and a shared one that every token takes, skewed load
        _layer("layer_T512_E384s1_k9", 512, 384, 9, 1024, 512, sigmoid=True, scaling=2.827, shared=1, zipf=1.1),
        # odd sizes, with slots that belong to another rank's experts (ids of -1) and tokens left with none
        _experts("experts_T37_E100_k5", 37, 100, 5, 1000, 344, dropped=0.3),
        # a prompt chunk over 64 experts top-4: 128 tokens an expert
        _experts("experts_T2048_E64_k4", 2048, 64, 4, 2048, 1024),
        # a long prompt over 8 large experts top-2: bound by the matrix products
        _experts("experts_T8192_E8_k2", 8192, 8, 2, 2048, 2048),
        # one token's router logits (256 experts, fp32), from a router with the request's adapter
        _adapter("adapter_T1_N256_r16", 1, 2048, 256, 16, 8, out="fp32"),
        # a decode batch, a request each with its adapter (a fifth without one) beside a square projection
        _adapter("adapter_T48_N4096_r16", 48, 4096, 4096, 16, 64, none=0.2),
        # odd sizes and a small rank, short prompts of several requests
        _adapter("adapter_T333_N1000_r8", 333, 1544, 1000, 8, 20, segment=29, none=0.1, out="fp32"),
        # prompts of 512 tokens of eight requests with wide adapters: bound by the matrix product
        _adapter("adapter_T4096_N4096_r64", 4096, 4096, 4096, 64, 16, segment=512),
    ]


def _logu(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], uniform in its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["layer", "experts", "adapter"])
        if op == "adapter":
            T = _logu(rng, 1, 4096)
            out = rng.choice(["bf16", "fp32"])
            c = _adapter(None, T, _logu(rng, 512, 4096, 8), _logu(rng, 64, 4096, 8), rng.choice([8, 16, 32, 64]),
                         _logu(rng, 2, 64), segment=_logu(rng, 1, 512), none=rng.choice([0.0, 0.1, 0.5]), out=out)
        else:
            E = _logu(rng, 8, 384)
            topk = min(E, rng.randint(1, 9))
            H, I = _logu(rng, 256, 2560, 8), _logu(rng, 128, 2048, 8)
            if op == "layer":
                T, shared = _logu(rng, 1, 512), 1 if topk > 1 and rng.random() < 0.3 else 0
                sig = rng.random() < 0.5
                c = _layer(None, T, E, topk, H, I, sigmoid=sig, scaling=rng.choice([1.0, 2.5]), shared=shared,
                           logits="bf16" if sig else rng.choice(["bf16", "fp32"]), zipf=rng.choice([0.0, 1.1]))
            else:
                T = _logu(rng, 1, 8192)
                c = _experts(None, T, E, topk, H, I, dropped=rng.choice([0.0, 0.0, 0.3]) if T >= 16 else 0.0)
        if _cost(c) <= most:
            return c


# ---- inputs ----------------------------------------------------------------------------------------------------


def _skew(E, s, gen):
    """Offsets that make expert loads fall off as rank^-s."""
    rank = torch.randperm(E, generator=gen, device="cuda") + 1
    return -s * torch.log(rank.double()).float()


def prepare(case, seed):
    c, gen = dict(case), torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def rand(*shape, sd=1.0, dtype=BF16):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype).mul_(sd)

    s = dict(case=c)
    if c["op"] == "adapter":
        T, K, N, r, n = c["T"], c["K"], c["N"], c["rank"], c["adapters"]
        s["x"] = rand(T, K)
        s["w"] = rand(N, K, sd=K ** -0.5)
        s["a"] = rand(n, r, K, sd=K ** -0.5)
        s["b"] = rand(n, N, r, sd=r ** -0.5)
        s["scale"] = 0.5 + torch.rand(n, generator=gen, device="cuda")
        requests = -(-T // c["segment"])
        pick = torch.randint(0, n, (requests,), generator=gen, device="cuda", dtype=torch.int32)
        if requests <= n:  # as many requests as adapters or fewer: each has its own
            pick = torch.randperm(n, generator=gen, device="cuda")[:requests].to(torch.int32)
        bare = torch.rand(requests, generator=gen, device="cuda") < c["none"]
        pick = torch.where(bare, torch.full_like(pick, -1), pick)
        s["adapter"] = pick.repeat_interleave(c["segment"])[:T].contiguous()
        return s
    T, E, k, H, I = c["T"], c["E"], c["topk"], c["H"], c["I"]
    s["x"] = rand(T, H)
    s["w13"] = rand(E + c.get("shared", 0), 2 * I, H, sd=H ** -0.5)
    s["w2"] = rand(E + c.get("shared", 0), H, I, sd=I ** -0.5)
    logits = torch.randn(T, E, generator=gen, device="cuda")
    if c["op"] == "layer":
        if c["zipf"]:
            logits = logits + _skew(E, c["zipf"], gen)
        s["logits"] = logits.to(BF16 if c["logits"] == "bf16" else F32)
    else:
        top = logits.topk(k, dim=1)
        idx = top.indices.to(torch.int32)
        if c["dropped"]:
            gone = torch.rand(T, k, generator=gen, device="cuda") < c["dropped"]
            gone[1 :: max(2, T // 8)] = True  # tokens whose experts all live elsewhere
            idx = torch.where(gone, torch.full_like(idx, -1), idx)
        s["topk_idx"] = idx.contiguous()
        s["topk_w"] = torch.softmax(top.values, dim=1).contiguous()
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------


def _plain_route(c, logits):
    """(ids, weights): top-k by score, ties to the lower index, then the shared experts."""
    E, k_r = c["E"], c["topk"] - c["shared"]
    x = logits.double()  # 64 bits: scores next to the selection's border decide whole numbers
    scores = torch.sigmoid(x) if c["sigmoid"] else torch.softmax(x, dim=1)
    idx = torch.sort(scores if c["sigmoid"] else x, dim=1, descending=True, stable=True).indices[:, :k_r]
    w = scores.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = (w * c["scaling"]).float()
    if c["shared"]:
        ids = torch.arange(E, E + c["shared"], device=idx.device).expand(len(idx), -1)
        idx, w = torch.cat([idx, ids], 1), torch.cat([w, torch.ones_like(ids, dtype=F32)], 1)
    return idx.to(torch.int32), w


def _plain_experts(x, idx, w, w13, w2):
    """Pairs gathered by expert into a padded batch, two batched products, and the weighted sum over a token's slots."""
    (T, k), E, H, I = idx.shape, w13.shape[0], x.shape[1], w2.shape[2]
    pair = ((idx >= 0) & (idx < E)).reshape(-1).nonzero()[:, 0]
    y = torch.zeros(T * k, H, device=x.device)
    if len(pair):
        used, slot = torch.unique(idx.reshape(-1)[pair].long(), return_inverse=True)
        count = torch.bincount(slot, minlength=len(used))
        order = torch.argsort(slot, stable=True)
        place = torch.empty_like(order)
        place[order] = torch.arange(len(pair), device=x.device) - (count.cumsum(0) - count)[slot[order]]
        rows = torch.zeros(len(used), int(count.max()), H, device=x.device)
        rows[slot, place] = x[pair // k].float()
        gu = torch.bmm(rows, w13[used].float().transpose(1, 2))
        g, u = gu[..., :I], gu[..., I:]
        h = g * torch.sigmoid(g) * u
        y[pair] = torch.bmm(h, w2[used].float().transpose(1, 2))[slot, place]
    return (y.view(T, k, H) * w[:, :, None]).sum(1).to(x.dtype)


def _plain_adapter(s):
    x, a, b = s["x"].float(), s["a"].float(), s["b"].float()
    n, r, K = a.shape
    low = (x @ a.reshape(n * r, K).t()).view(-1, n, r)
    mine = s["adapter"][:, None] == torch.arange(n, device=x.device)[None, :]
    low = torch.where(mine[:, :, None], low * s["scale"][None, :, None], torch.zeros_like(low))
    out = x @ s["w"].float().t() + low.reshape(-1, n * r) @ b.permute(0, 2, 1).reshape(n * r, -1)
    return out.to(F32 if s["case"]["out"] == "fp32" else BF16)


def run(s):
    c = s["case"]
    if own:
        import top_gating_expert_row_gb300 as mr

        if c["op"] == "adapter":
            return mr.adapter_proj(s["x"], s["w"], s["a"], s["b"], s["adapter"], s["scale"],
                                   out_dtype=F32 if c["out"] == "fp32" else BF16)
        if c["op"] == "experts":
            return mr.experts(s["x"], s["topk_idx"], s["topk_w"], s["w13"], s["w2"])
        return mr.layer(s["x"], s["logits"], c["topk"], s["w13"], s["w2"],
                        score_fn=mr.MR_SIGMOID if c["sigmoid"] else mr.MR_SOFTMAX, renorm=int(c["renorm"]),
                        scaling=c["scaling"], n_shared=c["shared"])
    if c["op"] == "adapter":
        return _plain_adapter(s)
    if c["op"] == "experts":
        return _plain_experts(s["x"], s["topk_idx"], s["topk_w"], s["w13"], s["w2"])
    idx, w = _plain_route(c, s["logits"])
    return dict(out=_plain_experts(s["x"], idx, w, s["w13"], s["w2"]), topk_idx=idx, topk_w=w)


def work(case):
    c = case
    if c["op"] == "adapter":
        T, K, N, r = c["T"], c["K"], c["N"], c["rank"]
        requests, n = -(-T // c["segment"]), c["adapters"]
        used = (requests if requests <= n else n * (1 - (1 - 1 / n) ** requests)) * (1 - c["none"])
        size = 4 if c["out"] == "fp32" else 2
        return {"bytes": T * K * 2 + N * K * 2 + used * r * (K + N) * 2 + T * 4 + T * N * size,
                "flops": 2.0 * T * N * K + 2.0 * T * (1 - c["none"]) * r * (K + N)}
    T, E, k, H, I = c["T"], c["E"], c["topk"], c["H"], c["I"]
    shared, kept = c.get("shared", 0), 1 - c.get("dropped", 0.0)
    # distinct experts that T tokens of k_r uniform choices reach (a skewed load reaches fewer: taken as uniform)
    used = E * (1 - (1 - (k - shared) * kept / E) ** T) + shared
    b = T * H * 2 * 2 + T * k * 8 + used * 3 * H * I * 2
    if c["op"] == "layer":
        b += T * E * (2 if c["logits"] == "bf16" else 4)
    return {"bytes": b, "flops": 6.0 * T * k * kept * H * I}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------


def _exact_choice(c, logits):
    """The selection one row after another on the host, in Python's own floats."""
    E, k_r = c["E"], c["topk"] - c["shared"]
    ids, ws = [], []
    for row in logits.double().cpu().tolist():
        top = max(row)
        s = [1 / (1 + math.exp(-v)) for v in row] if c["sigmoid"] else [math.exp(v - top) for v in row]
        total = 1.0 if c["sigmoid"] else math.fsum(s)
        best = sorted(range(E), key=lambda i: (-row[i], i))[:k_r]
        w = [s[i] / total for i in best]
        if c["renorm"]:
            z = math.fsum(w)
            w = [v / z for v in w]
        ids.append(best + list(range(E, E + c["shared"])))
        ws.append([v * c["scaling"] for v in w] + [1.0] * c["shared"])
    return torch.tensor(ids, device="cuda"), torch.tensor(ws, dtype=torch.float64, device="cuda")


def _exact_experts(x, idx, w, w13, w2):
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    I = w2.shape[2]
    for e in range(w13.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        up = w13[e].double() @ x[t].double().t()
        h = up[:I] / (1 + torch.exp(-up[:I])) * up[I:]
        out.index_add_(0, t, (w2[e].double() @ h).t() * w[t, j].double()[:, None])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "experts":
        return _exact_experts(s["x"], s["topk_idx"], s["topk_w"], s["w13"], s["w2"])
    if c["op"] == "layer":
        idx, w = _exact_choice(c, s["logits"])
        return dict(out=_exact_experts(s["x"], idx, w, s["w13"], s["w2"]), topk_idx=None, topk_w=w)
    x = s["x"].double()
    out = x @ s["w"].double().t()
    for i in range(c["adapters"]):
        t = (s["adapter"] == i).nonzero()[:, 0]
        low = x[t] @ s["a"][i].double().t()
        out[t] += s["scale"][i].double() * (low @ s["b"][i].double().t())
    return out
