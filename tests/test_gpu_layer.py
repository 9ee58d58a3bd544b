"""The experts' products, the whole layer and the adapter projection on the GPU against their definitions in
64 bits (tests/layer_reference.py has the bounds and their derivation)."""
import pytest
import torch

from layer_reference import adapter64, assert_within, experts64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def make_experts(T, E, k, H, I, seed=0, E_tot=None):
    g = _gen(seed)
    E_tot = E if E_tot is None else E_tot
    x = torch.randn(T, H, generator=g).to(BF16)
    w13 = (torch.randn(E_tot, 2 * I, H, generator=g) * H ** -0.5).to(BF16)
    w2 = (torch.randn(E_tot, H, I, generator=g) * I ** -0.5).to(BF16)
    top = torch.randn(T, E, generator=g).topk(k, dim=1)
    return x, top.indices.to(torch.int32), torch.softmax(top.values, 1), w13, w2


def shifted(t, by):
    """The same values at a base `by` elements past a 256-byte boundary."""
    room = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    v = room[by:].view(t.shape)
    v.copy_(t)
    return v


# T, E, topk, H, I: one token to a prompt, rows that are multiples of 8 and not, of 64 and not, more experts than
# pairs and fewer
EXPERT_SIZES = [
    (1, 8, 2, 64, 32), (1, 8, 2, 512, 256), (1, 256, 8, 256, 128), (2, 3, 3, 72, 40), (3, 16, 1, 64, 64),
    (5, 4, 4, 200, 104), (16, 32, 4, 256, 96), (17, 10, 2, 136, 72), (33, 5, 5, 128, 264), (64, 2, 1, 320, 128),
    (100, 7, 3, 192, 88), (130, 3, 2, 128, 128), (300, 2, 2, 256, 64), (513, 9, 4, 128, 64), (700, 1, 1, 64, 192),
    (1200, 4, 2, 128, 128), (2500, 3, 2, 64, 64),
    (1, 1, 1, 1, 1), (3, 4, 2, 7, 5), (9, 5, 3, 33, 17), (40, 6, 2, 66, 31), (4, 3, 2, 64, 37), (4, 3, 2, 37, 64),
]


@pytest.mark.parametrize("size", EXPERT_SIZES, ids=lambda s: "T%d_E%d_k%d_H%d_I%d" % s)
def test_experts(mr, size):
    x, idx, w, w13, w2 = make_experts(*size)
    want, bound = experts64(x, idx, w, w13, w2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mr.experts(x.cuda(), idx.cuda(), w.cuda(), w13.cuda(), w2.cuda(), status=status)
    assert_within(out, want, bound, "out")
    assert int(status.item()) == 0


@pytest.mark.parametrize("size", [(5, 4, 2, 128, 64), (20, 3, 2, 33, 17)])
def test_experts_gelu(mr, size):
    x, idx, w, w13, w2 = make_experts(*size, seed=4)
    want, bound = experts64(x, idx, w, w13, w2, act=1)
    assert_within(mr.experts(x.cuda(), idx.cuda(), w.cuda(), w13.cuda(), w2.cuda(), act=mr.MR_GELU), want, bound, "out")


@pytest.mark.parametrize("size", [(1, 8, 4, 64, 32), (37, 20, 5, 200, 88), (600, 6, 3, 128, 64), (11, 5, 3, 31, 9)])
def test_slots_without_an_expert(mr, size):
    """Ids outside [0, E) contribute nothing, tokens with none of theirs left get zeros, and the status says so."""
    T, E, k, H, I = size
    x, idx, w, w13, w2 = make_experts(*size, seed=1)
    gone = torch.rand(T, k, generator=_gen(2)) < 0.4
    gone[::3] = True
    other = torch.tensor([-1, E, E + 1000, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)
    idx = torch.where(gone, other[torch.randint(0, 5, (T, k), generator=_gen(3))], idx)
    w = torch.where(gone, torch.tensor(float("nan")), w)  # nothing of a skipped slot is used
    want, bound = experts64(x, idx, torch.nan_to_num(w), w13, w2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mr.experts(x.cuda(), idx.cuda(), w.cuda(), w13.cuda(), w2.cuda(), status=status)
    assert_within(out, want, bound, "out")
    assert not out[::3].any()
    assert int(status.item()) == mr.MR_ERANGE


def test_every_slot_without_an_expert(mr):
    x, idx, w, w13, w2 = make_experts(50, 8, 2, 128, 64)
    out = mr.experts(x.cuda(), torch.full_like(idx, -1).cuda(), w.cuda(), w13.cuda(), w2.cuda())
    assert not out.any()


@pytest.mark.parametrize("T,k", [(1, 4), (40, 3), (700, 2)])
def test_one_expert_in_every_slot(mr, T, k):
    """All pairs on one expert, the same one several times in a token."""
    x, _, w, w13, w2 = make_experts(T, 4, k, 128, 64)
    idx = torch.full((T, k), 2, dtype=torch.int32)
    want, bound = experts64(x, idx, w, w13, w2)
    assert_within(mr.experts(x.cuda(), idx.cuda(), w.cuda(), w13.cuda(), w2.cuda()), want, bound, "out")


def test_infinities_and_nan_stay_in_their_tokens(mr):
    T = 40
    x, idx, w, w13, w2 = make_experts(T, 6, 2, 128, 64)
    clean = mr.experts(x.cuda(), idx.cuda(), w.cuda(), w13.cuda(), w2.cuda())
    x[3, 5], x[17, 0], x[31, 127] = float("inf"), float("nan"), float("-inf")
    out = mr.experts(x.cuda(), idx.cuda(), w.cuda(), w13.cuda(), w2.cuda())
    rest = torch.ones(T, dtype=torch.bool)
    rest[[3, 17, 31]] = False
    assert torch.equal(out[rest.cuda()], clean[rest.cuda()])
    assert not torch.isfinite(out[17].float()).any()


def test_an_unused_experts_weights_are_not_read_into_the_sum(mr):
    x, idx, w, w13, w2 = make_experts(12, 6, 2, 128, 64)
    idx = torch.where(idx == 5, torch.zeros_like(idx), idx)
    want, bound = experts64(x, idx, w, w13, w2)
    w13[5], w2[5] = float("nan"), float("inf")
    assert_within(mr.experts(x.cuda(), idx.cuda(), w.cuda(), w13.cuda(), w2.cuda()), want, bound, "out")


@pytest.mark.parametrize("by", [1, 4, 8])
def test_unaligned_bases(mr, by):
    x, idx, w, w13, w2 = make_experts(6, 4, 2, 64, 32)
    want, bound = experts64(x, idx, w, w13, w2)
    a = [shifted(t.cuda(), by) for t in (x, idx, w, w13, w2)]
    assert_within(mr.experts(*a), want, bound, "out")


@pytest.mark.parametrize("T,E,k,H,I", [(1, 64, 8, 256, 128), (48, 16, 4, 200, 72), (1500, 8, 2, 128, 64)])
def test_same_bits_every_time(mr, T, E, k, H, I):
    a = [t.cuda() for t in make_experts(T, E, k, H, I)]
    first = mr.experts(*a)
    for _ in range(5):
        assert torch.equal(mr.experts(*a), first)


def test_nothing_past_the_output(mr):
    for T, E, k, H, I in [(1, 8, 2, 64, 32), (37, 6, 2, 200, 72), (5, 3, 2, 33, 17), (600, 4, 2, 136, 64)]:
        x, idx, w, w13, w2 = [t.cuda() for t in make_experts(T, E, k, H, I)]
        p = mr.mr_expert_params(T, H, I, E, k, mr.MR_BF16, mr.MR_SILU)
        nb = mr.moe_experts_workspace_bytes(p)
        room = torch.full((T + 4, H), 7.0, dtype=BF16, device="cuda")
        ws = torch.full((nb + 4096,), 0xA5, dtype=torch.uint8, device="cuda")  # any contents
        mr.moe_experts_fwd(p, x, idx, w, w13, w2, room, ws, nb)
        assert (room[T:] == 7.0).all() and (ws[nb:] == 0xA5).all()
        assert torch.equal(room[:T], mr.experts(x, idx, w, w13, w2))


LAYERS = [
    # T, E, topk, H, I, options
    (1, 8, 2, 512, 256, dict(renorm=1)), (1, 256, 8, 256, 64, dict(renorm=1)), (4, 256, 8, 128, 64, {}),
    (8, 128, 4, 192, 64, dict(renorm=1)), (16, 256, 8, 128, 64, dict(renorm=1)), (16, 1024, 4, 64, 32, {}),
    (12, 20, 10, 128, 64, {}), (16, 64, 9, 128, 64, dict(score_fn=1, renorm=1, n_shared=1, scaling=2.5)),
    (17, 64, 4, 128, 64, {}), (64, 32, 4, 256, 64, dict(score_fn=1, renorm=1, scaling=2.5)),
    (65, 96, 9, 64, 64, dict(score_fn=1, n_group=8, topk_group=4, n_shared=1, renorm=1)),
    (300, 16, 3, 128, 64, dict(n_shared=1, shared_weight=0.5)), (513, 8, 2, 64, 64, dict(renorm=1)),
    (16, 1024, 1008, 64, 32, dict(n_shared=1000, shared_weight=0.25)),
    (3, 4, 2, 33, 17, dict(renorm=1)), (2, 2304, 36, 64, 32, {}), (6, 37, 3, 128, 64, {}),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "T%d_E%d_k%d_H%d_I%d" % c[:5])
def test_layer(mr, orc, case, dtype):
    """The routing is moe_router_fwd's, bit for bit, and the output its experts'."""
    T, E, k, H, I, kw = case
    x, _, _, w13, w2 = make_experts(T, E, 1, H, I, E_tot=E + kw.get("n_shared", 0))
    logits = torch.randn(T, E, generator=_gen(7)).to(dtype)
    got = mr.layer(x.cuda(), logits.cuda(), k, w13.cuda(), w2.cuda(), **kw)
    routed = mr.route(logits.cuda(), k, dense=False, **kw)
    assert torch.equal(got["topk_idx"], routed["topk_idx"]) and torch.equal(got["topk_w"], routed["topk_w"])
    ref = orc.router_fwd(logits.float().numpy(), k, kw.get("score_fn", 0), kw.get("renorm", 0), kw.get("n_group", 0),
                         kw.get("topk_group", 0), kw.get("n_shared", 0), kw.get("scaling", 1.0),
                         kw.get("shared_weight", 1.0), None)
    idx = torch.from_numpy(ref["topk_idx"])
    want, bound = experts64(x, idx, got["topk_w"].cpu(), w13, w2)
    assert torch.equal(got["topk_idx"].cpu(), idx.to(torch.int32))
    assert_within(got["out"], want, bound, "out")


def test_layer_with_bias_and_without_compact_outputs(mr):
    T, E, k, H, I = 9, 64, 6, 128, 64
    x, _, _, w13, w2 = [t.cuda() for t in make_experts(T, E, k, H, I)]
    logits = torch.randn(T, E, generator=_gen(1)).cuda()
    bias = (torch.rand(E, generator=_gen(2)) - 0.5).cuda()
    got = mr.layer(x, logits, k, w13, w2, score_fn=mr.MR_SIGMOID, bias=bias)
    p = mr.params_for(logits, k, score_fn=mr.MR_SIGMOID, bias=bias)
    nb = mr.moe_layer_workspace_bytes(p, H, I)
    out, ws = torch.empty_like(x), torch.empty(nb, dtype=torch.uint8, device="cuda")
    mr.moe_layer_fwd(p, H, I, mr.MR_SILU, x, logits, w13, w2, out, None, None, ws)
    assert torch.equal(out, got["out"])
    assert torch.equal(out, mr.experts(x, got["topk_idx"], got["topk_w"], w13, w2))


ADAPTERS = [
    # T, K, N, rank, adapters, out
    (1, 64, 8, 8, 1, F32), (1, 512, 256, 16, 8, F32), (1, 128, 64, 64, 3, BF16), (7, 200, 136, 8, 5, F32),
    (16, 256, 128, 32, 40, BF16), (48, 256, 512, 16, 64, BF16), (33, 72, 40, 24, 3, F32), (65, 128, 130, 16, 100, F32),
    (128, 320, 96, 128, 4, BF16), (200, 136, 264, 40, 7, F32), (600, 128, 256, 16, 3, BF16), (1100, 64, 128, 64, 900, F32),
    (300, 264, 200, 48, 2, F32), (5, 64, 64, 136, 2, F32),
    # few units: the sum over K shared by clusters of 2, 4 and 8 CTAs
    (8, 2048, 128, 16, 4, F32), (20, 1032, 256, 8, 3, BF16), (64, 4096, 2048, 16, 9, BF16), (40, 1544, 1000, 24, 40, F32),
    (3, 4096, 64, 8, 2, F32), (4, 2056, 72, 40, 3, BF16),
    (1, 1, 1, 1, 1, F32), (5, 33, 17, 3, 4, F32), (9, 64, 31, 8, 2, BF16), (9, 64, 32, 5, 2, F32), (4, 30, 32, 8, 2, BF16),
]


def make_adapters(T, K, N, r, n, seed=0):
    g = _gen(seed)
    x = torch.randn(T, K, generator=g).to(BF16)
    w = (torch.randn(N, K, generator=g) * K ** -0.5).to(BF16)
    a = (torch.randn(n, r, K, generator=g) * K ** -0.5).to(BF16)
    b = (torch.randn(n, N, r, generator=g) * r ** -0.5).to(BF16)
    ad = torch.randint(-1, n, (T,), generator=g, dtype=torch.int32)
    return x, w, a, b, ad, 0.5 + torch.rand(n, generator=g)


@pytest.mark.parametrize("case", ADAPTERS, ids=lambda c: "T%d_K%d_N%d_r%d_n%d_%s" % (*c[:5], "fp32" if c[5] == F32 else "bf16"))
def test_adapter_proj(mr, case):
    *size, out = case
    v = make_adapters(*size)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mr.adapter_proj(*[t.cuda() for t in v], out_dtype=out, status=status)
    assert got.dtype == out
    assert_within(got, *adapter64(*v, out == BF16), "out")
    assert int(status.item()) == 0


@pytest.mark.parametrize("T,K,r,n,segment", [
    (20000, 64, 8, 7, 300), (20000, 64, 64, 5, 300), (20000, 72, 40, 3, 5000), (40000, 64, 128, 4, 700),
    (40000, 128, 16, 40, 1), (40000, 64, 24, 3, 40000),
])
def test_adapter_wide_tiles(mr, T, K, r, n, segment):
    """Prompts: tiles of 128 and 256 tokens that name one adapter, several, or none."""
    N = 128
    x, w, a, b, _, sc = make_adapters(T, K, N, r, n)
    pick = torch.randint(-1, n, (-(-T // segment),), generator=_gen(8), dtype=torch.int32)
    pick[0] = n - 1
    ad = pick.repeat_interleave(segment)[:T].contiguous()
    got = mr.adapter_proj(*[t.cuda() for t in (x, w, a, b, ad, sc)])
    assert_within(got, *adapter64(x, w, a, b, ad, sc, True), "out")
    if segment < T:  # the next request's adapter is corrupt: the others' tokens stay as they were
        bad = int(ad[-1])
        b[bad] = float("inf")
        other = mr.adapter_proj(*[t.cuda() for t in (x, w, a, b, ad, sc)])
        rest = (ad != bad).cuda() if bad >= 0 else torch.ones(T, dtype=torch.bool, device="cuda")
        assert torch.equal(other[rest], got[rest])


@pytest.mark.parametrize("T,K,N", [(1, 64, 64), (20, 128, 264), (300, 256, 128), (4, 33, 9)])
def test_projection_without_adapters(mr, T, K, N):
    x, w, a, b, ad, sc = make_adapters(T, K, N, 8, 4)
    want, bound = adapter64(x, w, None, None, None, None, False)
    assert_within(mr.adapter_proj(x.cuda(), w.cuda(), out_dtype=F32), want, bound, "alone")
    none = torch.full_like(ad, -1)
    got = mr.adapter_proj(x.cuda(), w.cuda(), a.cuda(), b.cuda(), none.cuda(), sc.cuda(), out_dtype=F32)
    assert_within(got, want, bound, "every token without one")


def test_adapter_ids_out_of_range(mr):
    x, w, a, b, ad, sc = make_adapters(30, 128, 64, 16, 4)
    ad[::4] = torch.tensor([4, 2 ** 31 - 1, -2 ** 31, 100], dtype=torch.int32).repeat(2)[: len(ad[::4])]
    want, bound = adapter64(x, w, a, b, ad, sc, False)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mr.adapter_proj(*[t.cuda() for t in (x, w, a, b, ad, sc)], out_dtype=F32, status=status)
    assert_within(got, want, bound, "out")
    assert int(status.item()) == mr.MR_ERANGE


def test_adapters_of_other_requests_do_not_reach_a_token(mr):
    """NaN and infinities in one adapter (and its scale) stay in the tokens that name it."""
    x, w, a, b, ad, sc = make_adapters(40, 128, 72, 16, 5)
    ad[:5] = torch.arange(5, dtype=torch.int32)
    clean = mr.adapter_proj(*[t.cuda() for t in (x, w, a, b, ad, sc)], out_dtype=F32)
    a[1], b[2], sc[3] = float("nan"), float("inf"), float("nan")
    x[39, 0], ad[39] = float("inf"), -1
    got = mr.adapter_proj(*[t.cuda() for t in (x, w, a, b, ad, sc)], out_dtype=F32)
    rest = ((ad == 0) | (ad == 4) | (ad < 0)) & (torch.arange(40) < 39)
    assert torch.equal(got[rest.cuda()], clean[rest.cuda()])
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[2]).any() and torch.isnan(got[3]).all()


def test_adapter_without_scale_and_unaligned(mr):
    x, w, a, b, ad, _ = make_adapters(12, 64, 40, 8, 3)
    want, bound = adapter64(x, w, a, b, ad, None, True)
    assert_within(mr.adapter_proj(*[t.cuda() for t in (x, w, a, b, ad)]), want, bound, "out")
    for by in (1, 4):
        moved = [shifted(t.cuda(), by) for t in (x, w, a, b, ad)]
        assert_within(mr.adapter_proj(*moved), want, bound, "unaligned")


def test_adapter_nothing_past_the_output(mr):
    for T, K, N, r, n, dt in [(1, 64, 40, 8, 2, F32), (37, 200, 72, 16, 5, BF16), (300, 64, 130, 64, 2, F32)]:
        x, w, a, b, ad, sc = [t.cuda() for t in make_adapters(T, K, N, r, n)]
        p = mr.mr_adapter_params(T, K, N, n, r, mr.MR_BF16, mr.MR_F32 if dt == F32 else mr.MR_BF16)
        nb = mr.moe_adapter_proj_workspace_bytes(p)
        room = torch.full((T + 4, N), 7.0, dtype=dt, device="cuda")
        ws = torch.full((nb + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        mr.moe_adapter_proj_fwd(p, x, w, a, b, ad, sc, room, ws, nb)
        assert (room[T:] == 7.0).all() and (ws[nb:] == 0xA5).all()
        assert torch.equal(room[:T], mr.adapter_proj(x, w, a, b, ad, sc, out_dtype=dt))


# ---- as they are used: the projection that makes the logits, then the layer ------------------------------------


def decode_step(mr, x, wg, a, b, ad, sc, w13, w2, k):
    logits = mr.adapter_proj(x, wg, a, b, ad, sc, out_dtype=F32)
    return logits, mr.layer(x, logits, k, w13, w2, renorm=1)


def step_inputs(T, E, k, H, I, seed=0):
    x, _, _, w13, w2 = make_experts(T, E, k, H, I, seed)
    _, wg, a, b, ad, sc = make_adapters(T, H, E, 8, 4, seed + 1)
    return [t.cuda() for t in (x, wg, a, b, ad, sc, w13, w2)]


@pytest.mark.parametrize("overlap", [True, False])
@pytest.mark.parametrize("T", [1, 16, 100, 600])
def test_projection_and_layer_together(mr, T, overlap):
    E, k, H, I = 32, 4, 256, 64
    v = step_inputs(T, E, k, H, I)
    mr.moe_router_set_launch_overlap(overlap)
    try:
        for _ in range(3):
            logits, got = decode_step(mr, *v, k)
    finally:
        mr.moe_router_set_launch_overlap(True)
    x, wg, a, b, ad, sc, w13, w2 = [t.cpu() for t in v]
    assert_within(logits, *adapter64(x, wg, a, b, ad, sc, False), "logits")
    routed = mr.route(logits, k, dense=False, renorm=1)
    assert torch.equal(routed["topk_idx"], got["topk_idx"]) and torch.equal(routed["topk_w"], got["topk_w"])
    want, bound = experts64(x, got["topk_idx"].cpu(), got["topk_w"].cpu(), w13, w2)
    assert_within(got["out"], want, bound, "out")


@pytest.mark.parametrize("T", [1, 24, 600])
def test_captured_and_replayed_on_new_inputs(mr, T):
    E, k, H, I = 16, 2, 128, 64
    v = step_inputs(T, E, k, H, I)
    other = step_inputs(T, E, k, H, I, seed=50)
    want = [decode_step(mr, *u, k) for u in (v, other)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode_step(mr, *v, k)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits, got = decode_step(mr, *v, k)
    for u, (wl, wg) in ((None, want[0]), (other, want[1])):
        if u is not None:
            for dst, src in zip(v, u):
                dst.copy_(src)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(logits, wl) and torch.equal(got["out"], wg["out"])
        assert torch.equal(got["topk_idx"], wg["topk_idx"])


@pytest.mark.parametrize("T,E,k,H,I", [(1, 24, 3, 192, 72), (29, 24, 3, 192, 72), (900, 6, 3, 192, 72)])
def test_a_shapes_first_call_is_captured(mr, T, E, k, H, I):
    v = step_inputs(T, E, k, H, I, seed=9)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits, got = decode_step(mr, *v, k)
    graph.replay()
    torch.cuda.synchronize()
    wl, wg = decode_step(mr, *v, k)
    assert torch.equal(logits, wl) and torch.equal(got["out"], wg["out"])


def test_two_streams_at_once(mr):
    """Calls on two streams, each with its own workspace, beside one another."""
    E, k, H, I = 64, 4, 256, 128
    sizes = (1, 40, 300)
    ins = {T: step_inputs(T, E, k, H, I, seed=T) for T in sizes}
    want = {T: decode_step(mr, *ins[T], k)[1]["out"] for T in sizes}
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for r in range(6):
        for s, st in enumerate(streams):
            T = sizes[(r + s) % 3]
            x, wg, a, b, ad, sc, w13, w2 = ins[T]
            logits = mr.adapter_proj(x, wg, a, b, ad, sc, out_dtype=F32, stream=st)
            outs.append((T, mr.layer(x, logits, k, w13, w2, renorm=1, stream=st)["out"]))
    torch.cuda.synchronize()
    for T, o in outs:
        assert torch.equal(o, want[T])


def test_no_tokens(mr):
    x, idx, w, w13, w2 = [t.cuda() for t in make_experts(4, 4, 2, 64, 32)]
    assert mr.experts(x[:0], idx[:0], w[:0], w13, w2).shape == (0, 64)
    assert mr.layer(x[:0], torch.zeros(0, 4, device="cuda"), 2, w13, w2)["out"].shape == (0, 64)
    y = [t.cuda() for t in make_adapters(4, 64, 16, 8, 2)]
    assert mr.adapter_proj(y[0][:0], y[1], y[2], y[3], y[4][:0], y[5]).shape == (0, 16)


def test_binding_refuses(mr):
    x, idx, w, w13, w2 = [t.cuda() for t in make_experts(4, 4, 2, 64, 32)]
    for bad in ((x.float(), idx, w, w13, w2), (x, idx.long(), w, w13, w2), (x, idx, w.half(), w13, w2),
                (x, idx, w, w13.float(), w2)):
        with pytest.raises(TypeError):
            mr.experts(*bad)
    for bad in ((x[:3], idx, w, w13, w2), (x, idx, w[:, :1], w13, w2), (x, idx, w, w13[:, :62], w2),
                (x, idx, w, w13, w2[:3]), (x, idx, w, w13.cpu(), w2), (x.t().contiguous().t(), idx, w, w13, w2)):
        with pytest.raises(ValueError):
            mr.experts(*bad)
    with pytest.raises(ValueError):
        mr.layer(x, torch.zeros(4, 5, device="cuda"), 2, w13, w2)
    with pytest.raises(mr.MoERouterError):
        mr.layer(x, torch.zeros(4, 4, device="cuda"), 5, w13, w2)
    y = [t.cuda() for t in make_adapters(4, 64, 16, 8, 2)]
    with pytest.raises(ValueError):
        mr.adapter_proj(y[0], y[1], y[2])
    with pytest.raises(TypeError):
        mr.adapter_proj(*y, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        mr.adapter_proj(y[0], y[1], y[2], y[3], y[4][:3], y[5])


def test_bounded_waits_give_up_and_report_it(mr):
    """With the copies left out every wait of the tensor-core kernels runs out: the call's status says so (the
    library's word for a call without one), and the next normal call is right."""
    x, idx, w, w13, w2 = [t.cuda() for t in make_experts(40, 8, 4, 128, 64)]
    big = [t.cuda() for t in make_experts(3000, 2, 2, 128, 64)]
    want = [mr.experts(*v) for v in ((x, idx, w, w13, w2), big)]
    projections = [[t.cuda() for t in make_adapters(T, K, N, 16, 3)] for T, K, N in ((20, 1024, 128), (300, 128, 256))]
    wide = [t.cuda() for t in make_adapters(40000, 64, 128, 64, 2)]
    projections.append(wide)
    right = [mr.adapter_proj(*v) for v in projections]
    assert mr.device_status(clear=True) == 0
    mr.moe_router_set_wait_test(4, 1)
    try:
        for call in [lambda s: mr.experts(x, idx, w, w13, w2, status=s), lambda s: mr.experts(*big, status=s)] + [
                lambda s, v=v: mr.adapter_proj(*v, status=s) for v in projections]:
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            call(status)
            assert int(status.item()) == mr.MR_ETIMEOUT
            assert mr.device_status() == 0
        mr.experts(x, idx, w, w13, w2)
        assert mr.device_status(clear=True) == mr.MR_ETIMEOUT
    finally:
        mr.moe_router_set_wait_test(0, 0)
    assert torch.equal(mr.experts(x, idx, w, w13, w2), want[0]) and torch.equal(mr.experts(*big), want[1])
    for v, r in zip(projections, right):
        assert torch.equal(mr.adapter_proj(*v), r)
    assert mr.device_status() == 0


def test_two_graphs_beside_one_another(mr):
    """Two captured steps, each with the workspaces of its own capture, replayed on two streams at once."""
    E, k, H, I = 64, 4, 256, 128
    graphs, wants = [], []
    side = torch.cuda.Stream()
    for T in (40, 300):
        v = step_inputs(T, E, k, H, I, seed=T)
        with torch.cuda.stream(side):
            want = decode_step(mr, *v, k)[1]["out"].clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = decode_step(mr, *v, k)[1]["out"]
        graphs.append((g, got, v))
        wants.append(want)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, _, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_, got, _), want in zip(graphs, wants):
        assert torch.equal(got, want)


def test_a_workspace_of_any_contents_is_reused(mr):
    """One workspace for calls of other sizes, one after the other on one stream, eagerly and without a wait."""
    sizes = [(1, 8, 2, 64, 32), (40, 16, 4, 128, 64), (700, 4, 2, 128, 64), (9, 5, 3, 33, 17), (3000, 2, 2, 64, 64)]
    ins = [[t.cuda() for t in make_experts(*s, seed=i)] for i, s in enumerate(sizes)]
    want = [mr.experts(*v) for v in ins]
    ps = [mr.mr_expert_params(T, H, I, E, k, mr.MR_BF16, mr.MR_SILU) for T, E, k, H, I in sizes]
    nb = max(mr.moe_experts_workspace_bytes(p) for p in ps)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(v[0]) for v in ins]
    for _ in range(4):
        for p, (x, idx, w, w13, w2), o in zip(ps, ins, outs):
            mr.moe_experts_fwd(p, x, idx, w, w13, w2, o, ws, nb)
    torch.cuda.synchronize()
    for o, r in zip(outs, want):
        assert torch.equal(o, r)
