"""Refusals of the experts', the layer's and the adapter projection's entry points, on the host without a GPU:
every call here fails its checks (or has nothing to do) before any CUDA call."""
import ctypes

import pytest

FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from top_gating_expert_row_gb300 import build

    build.build()
    import top_gating_expert_row_gb300 as m

    return m


def experts(lib, ptr=None, wsb=1 << 40, **kw):
    f = dict(T=4, H=64, I=32, E=8, topk=2, dtype=1, act=0)
    f.update(kw)
    a = dict(x=FAKE, idx=FAKE, w=FAKE, w13=FAKE, w2=FAKE, out=FAKE, ws=FAKE, status=None)
    a.update(ptr or {})
    p = lib.mr_expert_params(**f)
    return lib._lib.moe_experts_fwd(ctypes.byref(p), a["x"], a["idx"], a["w"], a["w13"], a["w2"], a["out"], a["ws"],
                                    wsb, a["status"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(I=0), 1), (dict(E=0), 1), (dict(topk=0), 1), (dict(dtype=7), 1),
    (dict(act=2), 1), (dict(act=-1), 1), (dict(T=1 << 30, topk=2), 1), (dict(dtype=0), 2), (dict(E=4097), 2),
    (dict(H=(1 << 20) + 1), 2), (dict(I=(1 << 20) + 1), 2),
])
def test_experts_sizes(lib, kw, code):
    assert experts(lib, **kw) == code


@pytest.mark.parametrize("name", ["x", "idx", "w", "w13", "w2", "out", "ws"])
def test_experts_null_and_misaligned(lib, name):
    assert experts(lib, {name: None}) == 1
    assert experts(lib, {name: FAKE + 1}) == 1


def test_experts_workspace_and_empty(lib):
    need = lib.moe_experts_workspace_bytes(lib.mr_expert_params(4, 64, 32, 8, 2, 1, 0))
    assert need > 0
    assert experts(lib, wsb=need - 1) == 1 and experts(lib, dict(ws=FAKE + 128), wsb=need) == 1
    assert experts(lib, dict(status=FAKE + 2)) == 1
    assert experts(lib, T=0) == 0
    assert lib._lib.moe_experts_fwd(None, *[FAKE] * 7, 1 << 40, None, None) == 1
    for bad in ((0, 64, 32, 8, 2, 1, 0), (4, 64, 32, 8, 2, 0, 0), (4, 0, 32, 8, 2, 1, 0)):
        assert lib.moe_experts_workspace_bytes(lib.mr_expert_params(*bad)) == 0


def layer(lib, ptr=None, wsb=1 << 40, H=64, I=32, act=0, **kw):
    f = dict(T=4, E=8, topk=2)
    f.update(kw)
    cp = lib.RouterParams(**f).c()
    a = dict(x=FAKE, logits=FAKE, w13=FAKE, w2=FAKE, out=FAKE, idx=None, w=None, ws=FAKE, status=None)
    a.update(ptr or {})
    return lib._lib.moe_layer_fwd(ctypes.byref(cp), H, I, act, a["x"], a["logits"], a["w13"], a["w2"], a["out"],
                                  a["idx"], a["w"], a["ws"], wsb, a["status"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(H=0), 1), (dict(I=0), 1), (dict(act=5), 1), (dict(T=-1), 1), (dict(topk=9), 1), (dict(n_shared=2), 1),
    (dict(n_group=2, topk_group=1, topk=2), 2), (dict(E=5000), 2), (dict(E=4096, topk=3, n_shared=1), 2),
    (dict(n_shared=2147483000, topk=2147483002), 1), (dict(H=1 << 21), 2),
])
def test_layer_sizes(lib, kw, code):
    assert layer(lib, **kw) == code


@pytest.mark.parametrize("name", ["x", "logits", "w13", "w2", "out", "ws"])
def test_layer_null_and_misaligned(lib, name):
    assert layer(lib, {name: None}) == 1
    assert layer(lib, {name: FAKE + 1}) == 1


def test_layer_workspace_and_empty(lib):
    p = lib.RouterParams(4, 8, 2)
    need = lib.moe_layer_workspace_bytes(p, 64, 32)
    assert need > lib.moe_experts_workspace_bytes(lib.mr_expert_params(4, 64, 32, 8, 2, 1, 0))
    assert layer(lib, wsb=need - 1) == 1
    assert layer(lib, dict(idx=FAKE + 2)) == 1 and layer(lib, dict(w=FAKE + 2)) == 1
    assert layer(lib, T=0) == 0
    assert lib._lib.moe_layer_fwd(None, 64, 32, 0, *[FAKE] * 8, 1 << 40, None, None) == 1
    assert lib.moe_layer_workspace_bytes(lib.RouterParams(4, 5000, 2), 64, 32) == 0
    assert lib.moe_layer_workspace_bytes(lib.RouterParams(4, 8, 2), 0, 32) == 0


def adapter(lib, ptr=None, wsb=1 << 40, **kw):
    f = dict(T=4, K=64, N=32, n_adapters=3, rank=8, dtype=1, out_dtype=0)
    f.update(kw)
    a = dict(x=FAKE, w=FAKE, a=FAKE, b=FAKE, ad=FAKE, scale=None, out=FAKE, ws=FAKE, status=None)
    a.update(ptr or {})
    p = lib.mr_adapter_params(**f)
    return lib._lib.moe_adapter_proj_fwd(ctypes.byref(p), a["x"], a["w"], a["a"], a["b"], a["ad"], a["scale"],
                                         a["out"], a["ws"], wsb, a["status"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(n_adapters=-1), 1), (dict(rank=0), 1), (dict(dtype=3), 1),
    (dict(out_dtype=3), 1), (dict(dtype=0), 2), (dict(K=1 << 21), 2), (dict(N=1 << 21), 2), (dict(rank=1 << 21), 2),
])
def test_adapter_sizes(lib, kw, code):
    assert adapter(lib, **kw) == code


@pytest.mark.parametrize("name", ["x", "w", "a", "b", "ad", "out", "ws"])
def test_adapter_null_and_misaligned(lib, name):
    assert adapter(lib, {name: None}) == 1
    assert adapter(lib, {name: FAKE + 1}) == 1


def test_adapter_workspace_and_empty(lib):
    need = lib.moe_adapter_proj_workspace_bytes(lib.mr_adapter_params(4, 64, 32, 3, 8, 1, 0))
    assert need >= 4 * 8 * 4
    assert adapter(lib, wsb=need - 1) == 1 and adapter(lib, dict(scale=FAKE + 2)) == 1
    assert adapter(lib, dict(out=FAKE + 2)) == 1  # fp32 output
    assert adapter(lib, T=0) == 0
    assert lib._lib.moe_adapter_proj_fwd(None, *[FAKE] * 8, 1 << 40, None, None) == 1
    assert lib.moe_adapter_proj_workspace_bytes(lib.mr_adapter_params(4, 64, 32, -1, 8, 1, 0)) == 0
