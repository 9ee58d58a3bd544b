"""Python binding of libmoerouter.so, the GB300 MoE routing library.

Argument marshalling only: every function here passes device pointers, sizes
and the current CUDA stream to the C entry point of the same name (declared in
include/moe_router.h) and turns a non-zero status into an exception. All
arithmetic runs in the library's CUDA kernels; PyTorch supplies device memory
and streams. There is no fallback: without the compiled library, importing
this package raises.

The ``route`` / ``sort`` / ... helpers at the bottom only allocate the output
tensors and call the entry points.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoerouter.so")

MR_OK, MR_EINVAL, MR_EUNSUPPORTED, MR_ECUDA, MR_ERANGE, MR_ETIMEOUT = 0, 1, 2, 3, 4, 5
MR_SOFTMAX, MR_SIGMOID = 0, 1
MR_F32, MR_BF16 = 0, 1
MR_SILU, MR_GELU = 0, 1
MR_MAX_FUSED_TOKENS = 16
MR_MAX_FUSED_EXPERTS = 1024
MR_MAX_FUSED_TOKENS_SMALL_E = 64
MR_MAX_FUSED_EXPERTS_SMALL = 256



class mr_router_params(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("score_fn", ctypes.c_int32), ("in_dtype", ctypes.c_int32), ("renorm", ctypes.c_int32),
                ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("scaling", ctypes.c_float), ("shared_weight", ctypes.c_float),
                ("bias", ctypes.c_void_p)]


class mr_expert_params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "I", "E", "topk", "dtype", "act")]


class mr_adapter_params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "K", "N", "n_adapters", "rank", "dtype", "out_dtype")]


_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_PP = ctypes.POINTER(mr_router_params)
_PE = ctypes.POINTER(mr_expert_params)
_PA = ctypes.POINTER(mr_adapter_params)
_SIGS = {
    "moe_router_fwd": ([_PP, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "moe_router_bwd": ([_PP, _P, _P, _P, _P, _P], _I),
    "moe_aux_scores_fwd": ([_I, _I, _I, _I, _I, _P, _P, _P, _P], _I),
    "moe_aux_scores_bwd": ([_I, _I, _I, _P, _P, _P, _P], _I),
    "moe_sort_capacity": ([_I, _I, _I, _I], _SZ),
    "moe_sort_workspace_bytes": ([_I, _I, _I, _I], _SZ),
    "moe_sort": ([_P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P, _P], _I),
    "moe_sort_noalloc": ([_P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P], _I),
    "moe_sort_noalloc_scratch_bytes": ([], _SZ),
    "moe_router_set_wait_test": ([ctypes.c_uint, _I], _I),
    "moe_router_set_launch_overlap": ([_I], _I),
    "moe_router_fused_workspace_bytes": ([_PP, _I], _SZ),
    "moe_router_fused_fwd_sort": ([_PP, _P, _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P], _I),
    "moe_experts_workspace_bytes": ([_PE], _SZ),
    "moe_experts_fwd": ([_PE, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P], _I),
    "moe_layer_workspace_bytes": ([_PP, _I, _I, _I], _SZ),
    "moe_layer_fwd": ([_PP, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P], _I),
    "moe_adapter_proj_workspace_bytes": ([_PA], _SZ),
    "moe_adapter_proj_fwd": ([_PA, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P], _I),
    "moe_router_strerror": ([_I], ctypes.c_char_p),
    "moe_router_set_topk_path": ([_I, _I], _I),
    "moe_router_expf": ([_P, _P, _I, _P], _I),
    "moe_router_exp_value": ([_P, _P, _I, _P], _I),
    "moe_router_noop": ([_P], _I),
    "moe_router_device_status": ([_P, _I, _P], _I),
    "moe_router_bwd_dtype": ([_PP, _I, _P, _P, _P, _P, _P], _I),
    "moe_tokens_per_expert": ([_I, _I, _P, _P, _P], _I),
    "moe_aux_loss_workspace_bytes": ([_I, _I], _SZ),
    "moe_aux_loss_fwd": ([_I, _I, _I, ctypes.c_float, ctypes.c_longlong, _P, _P, _P, _P, _SZ, _P], _I),
    "moe_aux_loss_bwd": ([_I, _I, _I, ctypes.c_float, ctypes.c_longlong, _P, _P, _P, _P], _I),
}


class _Lib:
    """The loaded library; loading happens on first use so that the build
    script inside this package can run before the library exists."""

    _cdll = None

    def __getattr__(self, name):
        if _Lib._cdll is None:
            _Lib._cdll = _load()
        fn = getattr(_Lib._cdll, name)
        setattr(self, name, fn)  # found at once from now on
        return fn


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m top_gating_expert_row_gb300.build` "
            "(nvcc, sm_103a). There is no CPU or PyTorch fallback.")
    cdll = ctypes.CDLL(LIB_PATH)
    for name, (args, res) in _SIGS.items():
        f = getattr(cdll, name)
        f.argtypes = args
        f.restype = res
    return cdll


_lib = _Lib()


class MoERouterError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {strerror(code)}")
        self.code = code


def moe_router_strerror(code: int) -> str:
    return _lib.moe_router_strerror(code).decode()


strerror = moe_router_strerror


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE routing library must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ok(rc: int, where: str) -> int:
    if rc != MR_OK:
        raise MoERouterError(rc, where)
    return rc


@dataclass
class RouterParams:
    T: int
    E: int
    topk: int
    score_fn: int = MR_SOFTMAX
    in_dtype: int = MR_F32
    renorm: int = 0
    n_group: int = 0
    topk_group: int = 0
    n_shared: int = 0
    scaling: float = 1.0
    shared_weight: float = 1.0
    bias: Optional[torch.Tensor] = None

    def c(self) -> mr_router_params:
        return mr_router_params(self.T, self.E, self.topk, self.score_fn, self.in_dtype, self.renorm,
                                self.n_group, self.topk_group, self.n_shared, self.scaling,
                                self.shared_weight, _ptr(self.bias))


def _params(p) -> mr_router_params:
    return p.c() if isinstance(p, RouterParams) else p


# ------------------------------------------------------------------- entry points (same names as the C ABI)


def moe_router_fwd(p, logits, probs=None, routing_map=None, intermediate=None, topk_idx=None,
                   topk_w=None, status=None, stream=None) -> int:
    cp = _params(p)
    return _ok(_lib.moe_router_fwd(ctypes.byref(cp), _ptr(logits), _ptr(probs), _ptr(routing_map),
                                   _ptr(intermediate), _ptr(topk_idx), _ptr(topk_w), _ptr(status),
                                   _stream(stream)),
               "moe_router_fwd")


def moe_router_bwd_dtype(p, grad_dtype, grad_probs, intermediate, routing_map, grad_logits, stream=None) -> int:
    cp = _params(p)
    return _ok(_lib.moe_router_bwd_dtype(ctypes.byref(cp), grad_dtype, _ptr(grad_probs), _ptr(intermediate),
                                         _ptr(routing_map), _ptr(grad_logits), _stream(stream)),
               "moe_router_bwd_dtype")


def moe_router_bwd(p, grad_probs, intermediate, routing_map, grad_logits, stream=None) -> int:
    cp = _params(p)
    return _ok(_lib.moe_router_bwd(ctypes.byref(cp), _ptr(grad_probs), _ptr(intermediate),
                                   _ptr(routing_map), _ptr(grad_logits), _stream(stream)), "moe_router_bwd")


def moe_aux_scores_fwd(T, E, topk, score_fn, in_dtype, logits, scores=None, routing_map=None,
                       stream=None) -> int:
    return _ok(_lib.moe_aux_scores_fwd(T, E, topk, score_fn, in_dtype, _ptr(logits), _ptr(scores),
                                       _ptr(routing_map), _stream(stream)), "moe_aux_scores_fwd")


def moe_aux_scores_bwd(T, E, score_fn, grad_scores, scores, grad_logits, stream=None) -> int:
    return _ok(_lib.moe_aux_scores_bwd(T, E, score_fn, _ptr(grad_scores), _ptr(scores), _ptr(grad_logits),
                                       _stream(stream)), "moe_aux_scores_bwd")


def moe_sort_capacity(T, topk, E_tot, block_m) -> int:
    return int(_lib.moe_sort_capacity(T, topk, E_tot, block_m))


def moe_sort_workspace_bytes(T, topk, E_tot, block_m) -> int:
    return int(_lib.moe_sort_workspace_bytes(T, topk, E_tot, block_m))


def moe_sort(topk_idx, topk_w, T, topk, E_tot, block_m, sorted_token_ids, sorted_weights, expert_ids,
             num_tokens_post_pad, workspace, ws_bytes=None, status=None, stream=None) -> int:
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return _ok(_lib.moe_sort(_ptr(topk_idx), _ptr(topk_w), T, topk, E_tot, block_m, _ptr(sorted_token_ids),
                             _ptr(sorted_weights), _ptr(expert_ids), _ptr(num_tokens_post_pad),
                             _ptr(workspace), ws_bytes, _ptr(status), _stream(stream)), "moe_sort")


def moe_sort_noalloc(topk_idx, topk_w, T, topk, E_tot, block_m, sorted_token_ids, sorted_weights, expert_ids,
                     num_tokens_post_pad, status=None, stream=None) -> int:
    """moe_sort without a workspace: for callers that cannot allocate device
    memory. Its scratch is a fixed device array inside the library (see
    include/moe_router.h); calls that overlap on the GPU race on it."""
    return _ok(_lib.moe_sort_noalloc(_ptr(topk_idx), _ptr(topk_w), T, topk, E_tot, block_m,
                                     _ptr(sorted_token_ids), _ptr(sorted_weights), _ptr(expert_ids),
                                     _ptr(num_tokens_post_pad), _ptr(status), _stream(stream)),
               "moe_sort_noalloc")


def moe_sort_noalloc_scratch_bytes() -> int:
    """Bytes of moe_sort_noalloc's fixed scratch array, as the loaded library has it."""
    return int(_lib.moe_sort_noalloc_scratch_bytes())


def moe_router_fused_workspace_bytes(p, block_m) -> int:
    cp = _params(p)
    return int(_lib.moe_router_fused_workspace_bytes(ctypes.byref(cp), block_m))


def moe_router_fused_fwd_sort(p, logits, block_m, topk_idx, topk_w, sorted_token_ids, sorted_weights,
                              expert_ids, num_tokens_post_pad, workspace=None, ws_bytes=None, status=None,
                              stream=None) -> int:
    cp = _params(p)
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return _ok(_lib.moe_router_fused_fwd_sort(ctypes.byref(cp), _ptr(logits), block_m, _ptr(topk_idx),
                                              _ptr(topk_w), _ptr(sorted_token_ids), _ptr(sorted_weights),
                                              _ptr(expert_ids), _ptr(num_tokens_post_pad), _ptr(workspace),
                                              ws_bytes, _ptr(status), _stream(stream)), "moe_router_fused_fwd_sort")


def moe_router_set_topk_path(select_threshold: int = 8, force_path: int = 0) -> int:
    return _ok(_lib.moe_router_set_topk_path(select_threshold, force_path), "moe_router_set_topk_path")


def moe_router_set_launch_overlap(enable: bool = True) -> int:
    """Programmatic dependent launch of the library's kernels (on by default)."""
    return _ok(_lib.moe_router_set_launch_overlap(1 if enable else 0), "moe_router_set_launch_overlap")


def moe_router_set_wait_test(tries: int = 0, drop_copies: int = 0) -> int:
    """Test hook of the bounded waits (0, 0 restores the defaults)."""
    return _ok(_lib.moe_router_set_wait_test(tries, drop_copies), "moe_router_set_wait_test")


def moe_router_expf(x, y, stream=None) -> int:
    return _ok(_lib.moe_router_expf(_ptr(x), _ptr(y), x.numel(), _stream(stream)), "moe_router_expf")


def moe_router_exp_value(x, y, stream=None) -> int:
    return _ok(_lib.moe_router_exp_value(_ptr(x), _ptr(y), x.numel(), _stream(stream)), "moe_router_exp_value")


def moe_router_noop(stream=None) -> int:
    return _ok(_lib.moe_router_noop(_stream(stream)), "moe_router_noop")


def moe_router_device_status(out, clear: bool = False, stream=None) -> int:
    return _ok(_lib.moe_router_device_status(_ptr(out), 1 if clear else 0, _stream(stream)),
               "moe_router_device_status")


def device_status(clear: bool = False) -> int:
    """The library's device status word on the current device (0 or MR_ETIMEOUT)."""
    out = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe_router_device_status(out, clear)
    return int(out.item())


def moe_tokens_per_expert(T, E, routing_map, tokens_per_expert, stream=None) -> int:
    return _ok(_lib.moe_tokens_per_expert(T, E, _ptr(routing_map), _ptr(tokens_per_expert), _stream(stream)),
               "moe_tokens_per_expert")


def moe_aux_loss_workspace_bytes(T: int, E: int) -> int:
    return int(_lib.moe_aux_loss_workspace_bytes(T, E))


def moe_aux_loss_fwd(T, E, topk, coeff, total_num_tokens, probs, tokens_per_expert, loss, workspace,
                     ws_bytes=None, stream=None) -> int:
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return _ok(_lib.moe_aux_loss_fwd(T, E, topk, coeff, total_num_tokens, _ptr(probs), _ptr(tokens_per_expert),
                                     _ptr(loss), _ptr(workspace), ws_bytes, _stream(stream)), "moe_aux_loss_fwd")


def moe_aux_loss_bwd(T, E, topk, coeff, total_num_tokens, tokens_per_expert, grad_loss, grad_probs,
                     stream=None) -> int:
    return _ok(_lib.moe_aux_loss_bwd(T, E, topk, coeff, total_num_tokens, _ptr(tokens_per_expert),
                                     _ptr(grad_loss), _ptr(grad_probs), _stream(stream)), "moe_aux_loss_bwd")


def moe_experts_workspace_bytes(p: mr_expert_params) -> int:
    return int(_lib.moe_experts_workspace_bytes(ctypes.byref(p)))


def moe_experts_fwd(p: mr_expert_params, x, topk_idx, topk_w, w13, w2, out, workspace, ws_bytes=None, status=None,
                    stream=None) -> int:
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return _ok(_lib.moe_experts_fwd(ctypes.byref(p), _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(w13), _ptr(w2),
                                    _ptr(out), _ptr(workspace), ws_bytes, _ptr(status), _stream(stream)),
               "moe_experts_fwd")


def moe_layer_workspace_bytes(p, H: int, I: int, act: int = MR_SILU) -> int:
    cp = _params(p)
    return int(_lib.moe_layer_workspace_bytes(ctypes.byref(cp), H, I, act))


def moe_layer_fwd(p, H, I, act, x, logits, w13, w2, out, topk_idx=None, topk_w=None, workspace=None, ws_bytes=None,
                  status=None, stream=None) -> int:
    cp = _params(p)
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return _ok(_lib.moe_layer_fwd(ctypes.byref(cp), H, I, act, _ptr(x), _ptr(logits), _ptr(w13), _ptr(w2), _ptr(out),
                                  _ptr(topk_idx), _ptr(topk_w), _ptr(workspace), ws_bytes, _ptr(status),
                                  _stream(stream)), "moe_layer_fwd")


def moe_adapter_proj_workspace_bytes(p: mr_adapter_params) -> int:
    return int(_lib.moe_adapter_proj_workspace_bytes(ctypes.byref(p)))


def moe_adapter_proj_fwd(p: mr_adapter_params, x, w, a, b, adapter, scale, out, workspace, ws_bytes=None, status=None,
                         stream=None) -> int:
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return _ok(_lib.moe_adapter_proj_fwd(ctypes.byref(p), _ptr(x), _ptr(w), _ptr(a), _ptr(b), _ptr(adapter),
                                         _ptr(scale), _ptr(out), _ptr(workspace), ws_bytes, _ptr(status),
                                         _stream(stream)), "moe_adapter_proj_fwd")


# ------------------------------------------------------------------- allocating helpers

PATH_AUTO, PATH_ARGMAX, PATH_SELECT = 0, 1, 2


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MR_F32
    if t.dtype == torch.bfloat16:
        return MR_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def params_for(logits: torch.Tensor, topk: int, **kw) -> RouterParams:
    T, E = logits.shape
    return RouterParams(T=T, E=E, topk=topk, in_dtype=_dtype_code(logits), **kw)


def route(logits: torch.Tensor, topk: int, dense: bool = True, compact: bool = True, stream=None,
          status: Optional[torch.Tensor] = None, **kw) -> dict:
    """moe_router_fwd with freshly allocated outputs (probs in the logits dtype)."""
    p = params_for(logits, topk, **kw)
    T, E = logits.shape
    dev = logits.device
    out = {}
    if dense:
        out["probs"] = torch.empty(T, E, dtype=logits.dtype, device=dev)
        out["routing_map"] = torch.empty(T, E, dtype=torch.uint8, device=dev)
        out["intermediate"] = torch.empty(T, E, dtype=torch.float32, device=dev)
    if compact:
        out["topk_idx"] = torch.empty(T, topk, dtype=torch.int32, device=dev)
        out["topk_w"] = torch.empty(T, topk, dtype=torch.float32, device=dev)
    moe_router_fwd(p, logits, out.get("probs"), out.get("routing_map"), out.get("intermediate"),
                   out.get("topk_idx"), out.get("topk_w"), status, stream)
    return out


def route_bwd(p: RouterParams, grad_probs, intermediate, routing_map, stream=None) -> torch.Tensor:
    """grad_logits in grad_probs' dtype (fp32, or bf16 for bf16 logits)."""
    if grad_probs.dtype == torch.bfloat16:
        dx = torch.empty(intermediate.shape, dtype=torch.bfloat16, device=intermediate.device)
        moe_router_bwd_dtype(p, MR_BF16, grad_probs, intermediate, routing_map, dx, stream)
        return dx
    dx = torch.empty_like(intermediate)
    moe_router_bwd(p, grad_probs, intermediate, routing_map, dx, stream)
    return dx


def aux_scores(logits: torch.Tensor, topk: int, score_fn: int = MR_SOFTMAX, stream=None) -> dict:
    T, E = logits.shape
    scores = torch.empty(T, E, dtype=torch.float32, device=logits.device)
    rmap = torch.empty(T, E, dtype=torch.uint8, device=logits.device)
    moe_aux_scores_fwd(T, E, topk, score_fn, _dtype_code(logits), logits, scores, rmap, stream)
    return dict(scores=scores, routing_map=rmap)


def aux_scores_bwd(grad, scores, score_fn: int = MR_SOFTMAX, stream=None) -> torch.Tensor:
    T, E = scores.shape
    dx = torch.empty_like(scores)
    moe_aux_scores_bwd(T, E, score_fn, grad, scores, dx, stream)
    return dx


def sort_buffers(T: int, topk: int, E_tot: int, block_m: int, device) -> dict:
    cap = moe_sort_capacity(T, topk, E_tot, block_m)
    return dict(sorted_token_ids=torch.empty(cap, dtype=torch.int32, device=device),
                sorted_weights=torch.empty(cap, dtype=torch.float32, device=device),
                expert_ids=torch.empty(max(1, -(-cap // block_m)), dtype=torch.int32, device=device),
                num_tokens_post_pad=torch.empty(1, dtype=torch.int32, device=device))


def sort(topk_idx: torch.Tensor, topk_w: Optional[torch.Tensor], E_tot: int, block_m: int,
         status: Optional[torch.Tensor] = None, stream=None) -> dict:
    T, k = topk_idx.shape
    out = sort_buffers(T, k, E_tot, block_m, topk_idx.device)
    ws = torch.empty(max(1, moe_sort_workspace_bytes(T, k, E_tot, block_m)), dtype=torch.uint8,
                     device=topk_idx.device)
    moe_sort(topk_idx, topk_w, T, k, E_tot, block_m, out["sorted_token_ids"], out["sorted_weights"],
             out["expert_ids"], out["num_tokens_post_pad"], ws, None, status, stream)
    return out


def fused_route_sort(logits: torch.Tensor, topk: int, block_m: int, compact: bool = True, stream=None,
                     status: Optional[torch.Tensor] = None, **kw) -> dict:
    p = params_for(logits, topk, **kw)
    T, E = logits.shape
    E_tot = E + p.n_shared
    out = sort_buffers(T, topk, E_tot, block_m, logits.device)
    if compact:
        out["topk_idx"] = torch.empty(T, topk, dtype=torch.int32, device=logits.device)
        out["topk_w"] = torch.empty(T, topk, dtype=torch.float32, device=logits.device)
    nb = moe_router_fused_workspace_bytes(p, block_m)
    ws = torch.empty(max(1, nb), dtype=torch.uint8, device=logits.device) if nb else None
    moe_router_fused_fwd_sort(p, logits, block_m, out.get("topk_idx"), out.get("topk_w"),
                              out["sorted_token_ids"], out["sorted_weights"], out["expert_ids"],
                              out["num_tokens_post_pad"], ws, nb, status, stream)
    return out


def header_symbols() -> list[str]:
    """Function names declared in include/moe_router.h."""
    import re

    hdr = os.path.join(os.path.dirname(_HERE), "include", "moe_router.h")
    with open(hdr) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\*?(moe_\w+)\s*\(", text, re.M)))


def tokens_per_expert(routing_map: torch.Tensor, stream=None) -> torch.Tensor:
    """Per-expert count of routed rows of a uint8 [T, E] routing map (int32 [E])."""
    T, E = routing_map.shape
    out = torch.empty(E, dtype=torch.int32, device=routing_map.device)
    moe_tokens_per_expert(T, E, routing_map, out, stream)
    return out


def aux_loss(probs: torch.Tensor, tokens_per_expert: torch.Tensor, topk: int, coeff: float,
             total_num_tokens: int = None, stream=None) -> torch.Tensor:
    """The aux-loss scalar (one fp32 on the device) of fp32 probs [T, E]."""
    T, E = probs.shape
    N = T if total_num_tokens is None else total_num_tokens
    loss = torch.empty(1, dtype=torch.float32, device=probs.device)
    ws = torch.empty(max(1, moe_aux_loss_workspace_bytes(T, E)), dtype=torch.uint8, device=probs.device)
    moe_aux_loss_fwd(T, E, topk, coeff, N, probs, tokens_per_expert, loss, ws, stream=stream)
    return loss


def aux_loss_bwd(grad_loss: torch.Tensor, tokens_per_expert: torch.Tensor, T: int, topk: int, coeff: float,
                 total_num_tokens: int = None, stream=None) -> torch.Tensor:
    """d loss / d probs (fp32 [T, E])."""
    E = tokens_per_expert.numel()
    N = T if total_num_tokens is None else total_num_tokens
    g = torch.empty(T, E, dtype=torch.float32, device=tokens_per_expert.device)
    moe_aux_loss_bwd(T, E, topk, coeff, N, tokens_per_expert, grad_loss, g, stream)
    return g


# ------------------------------------------------------------------- the layer behind the router
# Serving operators: they have no backward pass, so inputs that ask for a gradient are refused instead of giving
# results that are cut off from them (under torch.no_grad(), as in serving, they are taken).


def _forward_only(*tensors) -> None:
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError("this operator has no backward pass: call it under torch.no_grad(), or detach its inputs")


def _check(what: str, t: torch.Tensor, shape, dtype, device) -> None:
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, x on {device}")
    raise ValueError(f"{what} must be contiguous")


def _check_status(status, device) -> Optional[int]:
    if status is None:
        return None
    if status.numel() < 1:
        raise ValueError("status must hold an int32")
    _check("status", status, status.shape, torch.int32, device)
    return status.data_ptr()


class _Launch:
    """The device of x made current, and on it `stream` (default: that device's current stream), on which the
    call's tensors are allocated, so that a workspace is not reused before the call's kernels are done. Entering
    gives the stream's handle."""

    __slots__ = ("index", "device", "stream")

    def __init__(self, device, stream):
        self.index, self.device, self.stream = device.index, None, None
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            if stream.device != device:
                raise ValueError(f"stream is on {stream.device}, x on {device}")
            self.stream = torch.cuda.stream(stream)
        else:
            self.device = torch.cuda.device(device)

    def __enter__(self):
        if self.device is not None:
            self.device.__enter__()
        if self.stream is not None:
            self.stream.__enter__()
        return torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        if self.stream is not None:
            self.stream.__exit__(*exc)
        if self.device is not None:
            self.device.__exit__(*exc)


class _Here:
    """_Launch where the device is current already and the stream its current one."""

    __slots__ = ("raw",)

    def __init__(self, index):
        self.raw = torch._C._cuda_getCurrentRawStream(index)

    def __enter__(self):
        return self.raw

    def __exit__(self, *exc):
        pass


def _launch(device, stream):
    if device.type != "cuda":
        raise ValueError(f"x must be on a CUDA device, got {device}")
    if stream is None and torch._C._cuda_getDevice() == device.index:
        return _Here(device.index)
    return _Launch(device, stream)


# The options of a call and the workspace it needs depend on its sizes alone: kept, so that a decode step does not
# build them again (and nothing else is).


@functools.lru_cache(maxsize=1024)
def _experts_plan(T, H, I, E, topk, act):
    p = mr_expert_params(T, H, I, E, topk, MR_BF16, act)
    return ctypes.byref(p), moe_experts_workspace_bytes(p)


@functools.lru_cache(maxsize=1024)
def _layer_plan(H, I, act, *options):
    cp = mr_router_params(*options, None)
    return ctypes.byref(cp), moe_layer_workspace_bytes(cp, H, I, act)


@functools.lru_cache(maxsize=1024)
def _adapter_plan(T, K, N, n, rank, out_f32):
    p = mr_adapter_params(T, K, N, n, rank, MR_BF16, MR_F32 if out_f32 else MR_BF16)
    return ctypes.byref(p), moe_adapter_proj_workspace_bytes(p)


def _weights_shape(x, w13, w2):
    if x.dim() != 2 or w13.dim() != 3 or w2.dim() != 3:
        raise ValueError("x is [T, H], w13 [E, 2*I, H], w2 [E, H, I]")
    E, H, I = w2.shape
    device = x.device
    _check("x", x, (x.shape[0], H), torch.bfloat16, device)
    _check("w13", w13, (E, 2 * I, H), torch.bfloat16, device)
    _check("w2", w2, (E, H, I), torch.bfloat16, device)
    return E, H, I


def experts(x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
            act: int = MR_SILU, status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_experts_fwd with a freshly allocated output and workspace: out [T, H] (bf16) of x [T, H] (bf16) through
    the experts topk_idx [T, topk] (int32; ids outside [0, E) are skipped) with weights topk_w (fp32).
    w13 [E, 2*I, H] holds each expert's gate rows, then its up rows; w2 is [E, H, I]. No backward pass."""
    _forward_only(x, topk_w, w13, w2)
    E, H, I = _weights_shape(x, w13, w2)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx is [T, topk]")
    T, k, dev = x.shape[0], topk_idx.shape[1], x.device
    _check("topk_idx", topk_idx, (T, k), torch.int32, dev)
    _check("topk_w", topk_w, (T, k), torch.float32, dev)
    st = _check_status(status, dev)
    p, nb = _experts_plan(T, H, I, E, k, act)
    with _launch(dev, stream) as raw:
        out = torch.empty_like(x)
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        _ok(_lib.moe_experts_fwd(p, x.data_ptr(), topk_idx.data_ptr(), topk_w.data_ptr(), w13.data_ptr(),
                                 w2.data_ptr(), out.data_ptr(), ws.data_ptr(), nb, st, raw), "moe_experts_fwd")
    return out


def layer(x: torch.Tensor, logits: torch.Tensor, topk: int, w13: torch.Tensor, w2: torch.Tensor, act: int = MR_SILU,
          status: Optional[torch.Tensor] = None, stream=None, score_fn: int = MR_SOFTMAX, renorm: int = 0,
          n_group: int = 0, topk_group: int = 0, n_shared: int = 0, scaling: float = 1.0, shared_weight: float = 1.0,
          bias: Optional[torch.Tensor] = None) -> dict:
    """moe_layer_fwd with freshly allocated outputs: the layer's out [T, H] and the routing it took (topk_idx,
    topk_w) from x [T, H] (bf16) and router logits [T, E] (fp32 or bf16). Routing options as for route(); w13 / w2
    as for experts(), with the shared experts last. No backward pass."""
    _forward_only(x, logits, w13, w2, bias)
    E_tot, H, I = _weights_shape(x, w13, w2)
    T, E, dev = x.shape[0], E_tot - n_shared, x.device
    dtype = _dtype_code(logits)
    _check("logits", logits, (T, E), logits.dtype, dev)
    st = _check_status(status, dev)
    options = (T, E, topk, score_fn, dtype, int(renorm), n_group, topk_group, n_shared, scaling, shared_weight)
    if bias is None:
        p, nb = _layer_plan(H, I, act, *options)
    else:
        _check("bias", bias, (E,), torch.float32, dev)
        cp = mr_router_params(*options, bias.data_ptr())
        p, nb = ctypes.byref(cp), moe_layer_workspace_bytes(cp, H, I, act)
    with _launch(dev, stream) as raw:
        out = torch.empty_like(x)
        idx = torch.empty(T, max(topk, 0), dtype=torch.int32, device=dev)
        w = torch.empty(T, max(topk, 0), dtype=torch.float32, device=dev)
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        _ok(_lib.moe_layer_fwd(p, H, I, act, x.data_ptr(), logits.data_ptr(), w13.data_ptr(), w2.data_ptr(),
                               out.data_ptr(), idx.data_ptr(), w.data_ptr(), ws.data_ptr(), nb, st, raw),
            "moe_layer_fwd")
    return dict(out=out, topk_idx=idx, topk_w=w)


def adapter_proj(x: torch.Tensor, w: torch.Tensor, a: Optional[torch.Tensor] = None,
                 b: Optional[torch.Tensor] = None, adapter: Optional[torch.Tensor] = None,
                 scale: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                 status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_adapter_proj_fwd with a freshly allocated output: x [T, K] through the shared w [N, K], plus for each
    token its adapter's scale[i] * b[i] (a[i] x), i = adapter[t] (int32 [T]; negative: none), a [n, rank, K],
    b [n, N, rank]; out [T, N] in out_dtype (bf16 or fp32). Without a, b, adapter: the projection alone. No backward
    pass."""
    _forward_only(x, w, a, b, scale)
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x is [T, K], w [N, K]")
    (T, K), N, dev = x.shape, w.shape[0], x.device
    _check("x", x, (T, K), torch.bfloat16, dev)
    _check("w", w, (N, K), torch.bfloat16, dev)
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    st = _check_status(status, dev)
    n = rank = 0
    pa = pb = pi = ps = None
    if a is not None or b is not None or adapter is not None or scale is not None:
        if a is None or b is None or adapter is None:
            raise ValueError("a, b and adapter come together")
        if a.dim() != 3:
            raise ValueError("a is [n, rank, K], b [n, N, rank]")
        n, rank = a.shape[:2]
        _check("a", a, (n, rank, K), torch.bfloat16, dev)
        _check("b", b, (n, N, rank), torch.bfloat16, dev)
        _check("adapter", adapter, (T,), torch.int32, dev)
        pa, pb, pi = a.data_ptr(), b.data_ptr(), adapter.data_ptr()
        if scale is not None:
            _check("scale", scale, (n,), torch.float32, dev)
            ps = scale.data_ptr()
    p, nb = _adapter_plan(T, K, N, n, rank, out_dtype == torch.float32)
    with _launch(dev, stream) as raw:
        out = torch.empty(T, N, dtype=out_dtype, device=dev)
        ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
        _ok(_lib.moe_adapter_proj_fwd(p, x.data_ptr(), w.data_ptr(), pa, pb, pi, ps, out.data_ptr(),
                                      ws.data_ptr() if nb else None, nb, st, raw), "moe_adapter_proj_fwd")
    return out
