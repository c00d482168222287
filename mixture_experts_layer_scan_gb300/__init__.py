"""Python binding of the GB300 fused MoE layer library (ctypes over include/moe_api.h).

Argument marshalling only: every step of the layer runs in the CUDA kernels of
libmoe_gb300.so.  PyTorch supplies device memory and streams.  The names
mirror the C entry points; each raises MoeError on a nonzero return code.
If the shared library is missing this module fails at import, loudly: there is
no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gb300.so")

MOE_F32, MOE_BF16, MOE_E4M3, MOE_INT4, MOE_E4M3_B128 = 0, 1, 2, 3, 4
MOE_OK, MOE_ERR_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE = 0, -1, -2, -3
MOE_ERR_CUDA, MOE_ERR_DEVICE_TIMEOUT, MOE_ERR_DEVICE_INDEX, MOE_ERR_ALIGNMENT = -4, -5, -6, -7
ORIENT_AUTO, ORIENT_SWAP_AB, ORIENT_TOKEN_MAJOR = 0, 1, 2
STAGES = ("route", "align", "gather", "gemm1", "act", "gemm2", "combine")
NUM_STAGES = len(STAGES)
# phase stamps of the single-launch kernel (moe_options.trace), in the order of moe_trace_event
TRACE_EVENTS = ("start", "router", "barrier0", "topk", "barrier1", "tables", "gathered", "g1_issued", "g2_ready",
                "issued", "mma_done", "g1_done", "epi_done", "comb_first", "comb_done", "end")
TRACE_WORDS = len(TRACE_EVENTS)

# every entry point include/moe_api.h declares
EXPORTS = ("moe_strerror", "moe_workspace_size", "moe_plan_info", "moe_align_capacity", "moe_route",
           "moe_topk_from_logits", "moe_align", "moe_forward", "moe_forward_noalloc", "moe_get_status",
           "moe_version", "moe_inv_rope_fp8_quant", "moe_forward_routed", "moe_cache_create", "moe_cache_destroy",
           "moe_cache_workspace_size", "moe_forward_cached", "moe_cache_stats", "moe_cache_lru_plan",
           "moe_cache_set_copy_mode", "moe_copy_from_host", "moe_forward_host", "moe_topk_grouped",
           "moe_route_grouped", "moe_quant_block", "moe_silu_quant_block", "moe_gemm_block", "moe_permute",
           "moe_unpermute", "moe_permute_backward", "moe_unpermute_backward", "moe_prenorm", "moe_norm_workspace_size",
           "moe_prenorm_backward", "moe_postnorm", "moe_postnorm_backward", "moe_lora_workspace_size", "moe_lora")
NOALLOC_MAX_WORKSPACE = 32 << 20


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {strerror(code)} ({code})")


class moe_options(ctypes.Structure):
    _fields_ = [("orientation", ctypes.c_int), ("split_k", ctypes.c_int), ("inject_timeout", ctypes.c_int),
                ("act_split", ctypes.c_int), ("trace", ctypes.c_void_p), ("single_launch", ctypes.c_int),
                ("stage_begin", ctypes.c_void_p * NUM_STAGES),
                ("stage_end", ctypes.c_void_p * NUM_STAGES), ("cta_pair", ctypes.c_int)]


class moe_plan(ctypes.Structure):
    _fields_ = [("orientation", ctypes.c_int), ("block", ctypes.c_int), ("splits_gemm1", ctypes.c_int),
                ("splits_gemm2", ctypes.c_int), ("act_split", ctypes.c_int), ("kernel_launches", ctypes.c_int),
                ("single_launch", ctypes.c_int), ("workspace_bytes", ctypes.c_size_t), ("cta_pair", ctypes.c_int)]


class moe_route_rule(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int), ("n_group", ctypes.c_int), ("topk_group", ctypes.c_int),
                ("group_sum", ctypes.c_int), ("renorm", ctypes.c_int), ("scale", ctypes.c_float)]


SCORES = {"softmax": 0, "sigmoid": 1}
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3


class moe_postnorm_rule(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("scale", ctypes.c_float), ("res_scale", ctypes.c_float),
                ("gate", ctypes.c_int), ("gate_sigmoid", ctypes.c_int), ("gate_dtype", ctypes.c_int),
                ("w_dtype", ctypes.c_int)]


class moe_cache_stats_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_ulonglong) for n in ("calls", "hits", "misses", "evictions", "bytes_h2d", "passes")]


CACHE_COPY_OVERLAP, CACHE_COPY_SERIAL, CACHE_COPY_KERNEL = 0, 1, 2


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() (nvcc, sm_103a)")
    lib = ctypes.CDLL(LIB_PATH)
    P, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.moe_strerror.restype = ctypes.c_char_p
    lib.moe_strerror.argtypes = [i]
    lib.moe_version.restype = i
    lib.moe_version.argtypes = []
    lib.moe_workspace_size.restype = i
    lib.moe_workspace_size.argtypes = [i, i, i, i, i, i, i, P, ctypes.POINTER(sz)]
    lib.moe_plan_info.restype = i
    lib.moe_plan_info.argtypes = [i, i, i, i, i, i, i, P, ctypes.POINTER(moe_plan)]
    lib.moe_align_capacity.restype = i
    lib.moe_align_capacity.argtypes = [i, i, i, i, ctypes.POINTER(sz), ctypes.POINTER(sz)]
    lib.moe_route.restype = i
    lib.moe_route.argtypes = [P, P, i, i, i, i, i, i, P, P, P, P]
    lib.moe_topk_from_logits.restype = i
    lib.moe_topk_from_logits.argtypes = [P, i, i, i, i, P, P, P]
    lib.moe_align.restype = i
    lib.moe_align.argtypes = [P, i, i, i, i, P, P, P, P, P]
    lib.moe_forward.restype = i
    lib.moe_forward.argtypes = [P, P, P, P, i, i, i, i, i, i, i, i, P, P, P, P, sz, P, P]
    lib.moe_forward_noalloc.restype = i
    lib.moe_forward_noalloc.argtypes = [P, P, P, P, i, i, i, i, i, i, i, i, P, P, P, P, P]
    lib.moe_forward_host.restype = i
    lib.moe_forward_host.argtypes = [P, P, P, P, P, i, i, i, i, i, i, i, i, P, P, P, P, sz, P, P]
    lib.moe_get_status.restype = i
    lib.moe_get_status.argtypes = [P]
    lib.moe_forward_routed.restype = i
    lib.moe_forward_routed.argtypes = [P, P, P, P, P, i, i, i, i, i, i, i, P, P, P, P, sz, P, P]
    lib.moe_cache_create.restype = i
    lib.moe_cache_create.argtypes = [P, P, P, P, i, i, i, i, i, i, i, ctypes.POINTER(P)]
    lib.moe_cache_destroy.restype = i
    lib.moe_cache_destroy.argtypes = [P]
    lib.moe_cache_set_copy_mode.restype = i
    lib.moe_cache_set_copy_mode.argtypes = [P, i]
    lib.moe_copy_from_host.restype = i
    lib.moe_copy_from_host.argtypes = [P, P, sz, P]
    lib.moe_cache_workspace_size.restype = i
    lib.moe_cache_workspace_size.argtypes = [P, i, i, P, ctypes.POINTER(sz)]
    lib.moe_forward_cached.restype = i
    lib.moe_forward_cached.argtypes = [P, P, P, i, i, i, P, P, sz, P, P]
    lib.moe_cache_stats.restype = i
    lib.moe_cache_stats.argtypes = [P, ctypes.POINTER(moe_cache_stats_t)]
    lib.moe_cache_lru_plan.restype = i
    lib.moe_cache_lru_plan.argtypes = [i, i, i, i, P, P, P, ctypes.POINTER(ctypes.c_ulonglong),
                                       ctypes.POINTER(ctypes.c_ulonglong)]
    lib.moe_inv_rope_fp8_quant.restype = i
    lib.moe_inv_rope_fp8_quant.argtypes = [P, i, i, i, i, P, P, i, P, P, P]
    lib.moe_topk_grouped.restype = i
    lib.moe_topk_grouped.argtypes = [P, P, i, i, i, ctypes.POINTER(moe_route_rule), P, P, P]
    lib.moe_route_grouped.restype = i
    lib.moe_route_grouped.argtypes = [P, P, P, i, i, i, i, ctypes.POINTER(moe_route_rule), i, P, P, P, P]
    lib.moe_quant_block.restype = i
    lib.moe_quant_block.argtypes = [P, i, i, i, P, P, P]
    lib.moe_silu_quant_block.restype = i
    lib.moe_silu_quant_block.argtypes = [P, i, i, i, P, P, P]
    lib.moe_gemm_block.restype = i
    lib.moe_gemm_block.argtypes = [P, P, P, P, i, i, i, i, P, P]
    f, rule = ctypes.c_float, ctypes.POINTER(moe_postnorm_rule)
    for name, args in (("moe_permute", [P, P, i, i, i, i, i, i, P, P, P, P, P, P, P]),
                       ("moe_unpermute", [P, i, P, P, i, i, i, i, P, P]),
                       ("moe_permute_backward", [P, i, P, i, i, i, i, P, P]),
                       ("moe_unpermute_backward", [P, P, i, P, P, P, P, i, i, i, i, P, P, P]),
                       ("moe_prenorm", [P, P, i, i, f, i, i, P, P]),
                       ("moe_norm_workspace_size", [i, i, ctypes.POINTER(sz)]),
                       ("moe_prenorm_backward", [P, P, P, i, i, f, i, i, P, P, P, sz, P]),
                       ("moe_postnorm", [P, P, P, P, P, i, i, i, rule, P, P, P]),
                       ("moe_postnorm_backward", [P] * 7 + [i, i, i, rule] + [P] * 6 + [sz, P]),
                       ("moe_lora_workspace_size", [i, i, i, i, i, ctypes.POINTER(sz)]),
                       ("moe_lora", [P] * 6 + [i] * 6 + [P, P, sz, P])):
        getattr(lib, name).restype = i
        getattr(lib, name).argtypes = args
    return lib


_lib = _load()


def lib():
    return _lib


def strerror(code: int) -> str:
    return _lib.moe_strerror(int(code)).decode()


def version() -> int:
    return int(_lib.moe_version())


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise MoeError(rc, where)


_DTYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float8_e4m3fn: MOE_E4M3, torch.uint8: MOE_E4M3}


def _dt(t: torch.Tensor) -> int:
    return _DTYPES[t.dtype]


def _p(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _empty(shape, dtype: torch.dtype, device, stream, zero: bool = False) -> torch.Tensor:
    """A new tensor for a call on `stream`.

    Beside the current stream its memory is that stream's own, and goes back only after the current stream's
    work too: torch would else hand it to the current stream's next tensor while the call still runs."""
    make = torch.zeros if zero else torch.empty
    if stream is not None and torch.device(device).type == "cuda":
        handle, current = _stream(stream), torch.cuda.current_stream(device)
        if handle != current.cuda_stream:
            side = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
            with torch.cuda.stream(side):
                t = make(shape, dtype=dtype, device=device)
            t.record_stream(current)
            return t
    return make(shape, dtype=dtype, device=device)


def _out(t: Optional[torch.Tensor], shape, dtype, device, stream) -> torch.Tensor:
    """The caller's output tensor, checked, or a new one."""
    if t is None:
        return _empty(shape, dtype, device, stream)
    if t.shape != shape or (t.dtype != dtype and not (dtype == torch.float8_e4m3fn and t.dtype == torch.uint8)):
        raise ValueError(f"an output must be {dtype} {tuple(shape)}")
    return t


def _stream(stream) -> int:
    if stream is None:
        # (the raw handle: building a Stream object costs 3 us of a call's 10 on the host)
        if torch.cuda.is_initialized():
            return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _opts(options) -> Optional[ctypes.POINTER(moe_options)]:
    if options is None:
        return None
    if isinstance(options, moe_options):
        return ctypes.byref(options)
    o = moe_options()
    o.orientation = int(options.get("orientation", 0))
    o.split_k = int(options.get("split_k", 0))
    o.inject_timeout = int(options.get("inject_timeout", 0))
    o.act_split = int(options.get("act_split", 0))
    o.single_launch = int(options.get("single_launch", 0))
    o.cta_pair = int(options.get("cta_pair", 0))
    if options.get("trace") is not None:
        o.trace = ctypes.c_void_p(options["trace"].data_ptr())
    for name, ev in (options.get("stage_begin") or {}).items():
        o.stage_begin[STAGES.index(name)] = ctypes.c_void_p(ev.cuda_event)
    for name, ev in (options.get("stage_end") or {}).items():
        o.stage_end[STAGES.index(name)] = ctypes.c_void_p(ev.cuda_event)
    return ctypes.byref(o)


def moe_workspace_size(T: int, H: int, I: int, E: int, topk: int, act_dtype: int, w_dtype: int, options=None) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.moe_workspace_size(T, H, I, E, topk, act_dtype, w_dtype, _opts(options), ctypes.byref(n)),
           "moe_workspace_size")
    return int(n.value)


def moe_plan_info(T: int, H: int, I: int, E: int, topk: int, act_dtype: int, w_dtype: int, options=None) -> dict:
    info = moe_plan()
    _check(_lib.moe_plan_info(T, H, I, E, topk, act_dtype, w_dtype, _opts(options), ctypes.byref(info)),
           "moe_plan_info")
    return {name: getattr(info, name) for name, _ in moe_plan._fields_}


def moe_align_capacity(T: int, topk: int, E: int, block: int):
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(_lib.moe_align_capacity(T, topk, E, block, ctypes.byref(a), ctypes.byref(b)), "moe_align_capacity")
    return int(a.value), int(b.value)


def moe_route(hidden: torch.Tensor, router_w: torch.Tensor, topk: int, renorm: bool, logits=None, topk_w=None,
              topk_ids=None, stream=None):
    """Router logits [T,E] fp32, top-k weights [T,k] fp32 and ids [T,k] int32."""
    T, H = hidden.shape
    E = router_w.shape[0]
    dev = hidden.device
    logits = _empty((T, E), torch.float32, dev, stream) if logits is None else logits
    topk_w = _empty((T, topk), torch.float32, dev, stream) if topk_w is None else topk_w
    topk_ids = _empty((T, topk), torch.int32, dev, stream) if topk_ids is None else topk_ids
    _check(_lib.moe_route(_p(hidden), _p(router_w), T, H, E, topk, int(bool(renorm)), _dt(hidden), _p(logits),
                          _p(topk_w), _p(topk_ids), _stream(stream)), "moe_route")
    return logits, topk_w, topk_ids


def moe_topk_from_logits(logits: torch.Tensor, topk: int, renorm: bool, topk_w=None, topk_ids=None, stream=None):
    T, E = logits.shape
    dev = logits.device
    topk_w = _empty((T, topk), torch.float32, dev, stream) if topk_w is None else topk_w
    topk_ids = _empty((T, topk), torch.int32, dev, stream) if topk_ids is None else topk_ids
    _check(_lib.moe_topk_from_logits(_p(logits), T, E, topk, int(bool(renorm)), _p(topk_w), _p(topk_ids),
                                     _stream(stream)), "moe_topk_from_logits")
    return topk_w, topk_ids


def _route_rule(score: str, n_group: int, topk_group: Optional[int], group_sum: int, renorm: bool,
                scale: float) -> moe_route_rule:
    if score not in SCORES:
        raise ValueError(f"score {score!r}: {', '.join(SCORES)}")
    return moe_route_rule(SCORES[score], int(n_group), int(n_group if topk_group is None else topk_group),
                          int(group_sum), int(bool(renorm)), float(scale))


def moe_topk_grouped(logits: torch.Tensor, topk: int, bias=None, score: str = "sigmoid", n_group: int = 1,
                     topk_group: Optional[int] = None, group_sum: int = 2, renorm: bool = True, scale: float = 1.0,
                     topk_w=None, topk_ids=None, stream=None):
    """Routing by expert groups from fp32 logits [T,E]: (weights fp32 [T,topk], ids int32 [T,topk]).

    score: "sigmoid" or "softmax"; bias: fp32 [E] added for the choice only; the topk_group best of
    n_group groups are kept (topk_group None: all), a group scored by the sum of its group_sum largest."""
    T, E = logits.shape
    if logits.dtype != torch.float32 or (bias is not None and (bias.dtype != torch.float32 or bias.shape != (E,))):
        raise ValueError("logits must be float32 [T, E] and bias float32 [E]")
    dev = logits.device
    topk_w = _out(topk_w, (T, topk), torch.float32, dev, stream)
    topk_ids = _out(topk_ids, (T, topk), torch.int32, dev, stream)
    rule = _route_rule(score, n_group, topk_group, group_sum, renorm, scale)
    _check(_lib.moe_topk_grouped(_p(logits), _p(bias), T, E, topk, ctypes.byref(rule), _p(topk_w), _p(topk_ids),
                                 _stream(stream)), "moe_topk_grouped")
    return topk_w, topk_ids


def moe_route_grouped(hidden: torch.Tensor, router_w: torch.Tensor, topk: int, bias=None, score: str = "sigmoid",
                      n_group: int = 1, topk_group: Optional[int] = None, group_sum: int = 2, renorm: bool = True,
                      scale: float = 1.0, logits=None, topk_w=None, topk_ids=None, stream=None):
    """moe_topk_grouped on the router logits hidden . router_w^T: (logits [T,E], weights, ids)."""
    T, H = hidden.shape
    E = router_w.shape[0]
    if router_w.shape != (E, H) or router_w.dtype != hidden.dtype or (
            bias is not None and (bias.dtype != torch.float32 or bias.shape != (E,))):
        raise ValueError("router_w must be [E, H] of hidden's type and bias float32 [E]")
    dev = hidden.device
    logits = _out(logits, (T, E), torch.float32, dev, stream)
    topk_w = _out(topk_w, (T, topk), torch.float32, dev, stream)
    topk_ids = _out(topk_ids, (T, topk), torch.int32, dev, stream)
    rule = _route_rule(score, n_group, topk_group, group_sum, renorm, scale)
    _check(_lib.moe_route_grouped(_p(hidden), _p(router_w), _p(bias), T, H, E, topk, ctypes.byref(rule), _dt(hidden),
                                  _p(logits), _p(topk_w), _p(topk_ids), _stream(stream)), "moe_route_grouped")
    return logits, topk_w, topk_ids


def moe_quant_block(x: torch.Tensor, q=None, scale=None, stream=None):
    """e4m3 codes [T,K] (float8_e4m3fn) and float32 scales [T,ceil(K/128)] of x [T,K] by blocks of 128 columns."""
    T, K = x.shape
    q = _out(q, (T, K), torch.float8_e4m3fn, x.device, stream)
    scale = _out(scale, (T, (K + 127) // 128), torch.float32, x.device, stream)
    _check(_lib.moe_quant_block(_p(x), T, K, _dt(x), _p(q), _p(scale), _stream(stream)), "moe_quant_block")
    return q, scale


def moe_silu_quant_block(gate_up: torch.Tensor, q=None, scale=None, stream=None):
    """moe_quant_block of SiLU(g) * u for rows [g | u] of gate_up [T, 2I]: codes [T,I], scales [T,ceil(I/128)]."""
    T, two_i = gate_up.shape
    if two_i % 2:
        raise ValueError("gate_up must be [T, 2 I]")
    I = two_i // 2
    dev = gate_up.device
    q = _out(q, (T, I), torch.float8_e4m3fn, dev, stream)
    scale = _out(scale, (T, (I + 127) // 128), torch.float32, dev, stream)
    _check(_lib.moe_silu_quant_block(_p(gate_up), T, I, _dt(gate_up), _p(q), _p(scale), _stream(stream)),
           "moe_silu_quant_block")
    return q, scale


def moe_gemm_block(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                   out_dtype: torch.dtype = torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """a [T,K] . w [N,K]^T of block-scaled e4m3 operands -> out [T,N] (bfloat16 or float32).

    a_scale float32 [T,ceil(K/128)] (moe_quant_block), w_scale float32 [ceil(N/128),ceil(K/128)]."""
    T, K = a.shape
    N, Kw = w.shape
    kb = (K + 127) // 128
    if Kw != K or a_scale.shape != (T, kb) or w_scale.shape != ((N + 127) // 128, kb):
        raise ValueError("inconsistent shapes")
    if _dt(a) != MOE_E4M3 or _dt(w) != MOE_E4M3 or a_scale.dtype != torch.float32 or w_scale.dtype != torch.float32:
        raise ValueError("a and w must be e4m3 codes with float32 scales")
    if out is None:
        out = _empty((T, N), out_dtype, a.device, stream)
    elif out.shape != (T, N):
        raise ValueError("out must be [T, N]")
    _check(_lib.moe_gemm_block(_p(a), _p(a_scale), _p(w), _p(w_scale), T, N, K, _dt(out), _p(out), _stream(stream)),
           "moe_gemm_block")
    return out


def moe_align(topk_ids: torch.Tensor, E: int, block: int, stream=None, with_counts: bool = True):
    """(sorted_ids, expert_ids, num_post_pad[1], expert_counts) as full-capacity int32 device tensors."""
    T, k = topk_ids.shape
    cap, bcap = moe_align_capacity(T, k, E, block)
    dev = topk_ids.device
    sorted_ids = _empty(max(cap, 1), torch.int32, dev, stream)
    expert_ids = _empty(max(bcap, 1), torch.int32, dev, stream)
    npp = _empty(4, torch.int32, dev, stream, zero=T == 0)  # (an empty batch launches nothing)
    counts = _empty(E, torch.int32, dev, stream, zero=T == 0) if with_counts else None
    _check(_lib.moe_align(_p(topk_ids), T, k, E, block, _p(sorted_ids), _p(expert_ids), _p(npp), _p(counts),
                          _stream(stream)), "moe_align")
    return sorted_ids, expert_ids, npp[:1], counts


def _begin(stream, x: torch.Tensor, *others) -> int:
    """The handle of a call's stream.  Its arrays have to lie on the current CUDA device (the library reads their
    addresses as that device's)."""
    d = x.get_device()
    if d < 0 or d != torch._C._cuda_getDevice():
        raise ValueError("tensors must be on the current CUDA device")
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError("tensors must be on the current CUDA device")
    return torch._C._cuda_getCurrentRawStream(d) if stream is None else _stream(stream)


def _out_like(t: Optional[torch.Tensor], x: torch.Tensor, stream) -> torch.Tensor:
    """The caller's output of x's shape and type, checked, or a new one."""
    if t is None and stream is None:
        return torch.empty_like(x)  # (cheaper on the host than a new shape)
    return _out(t, x.shape, x.dtype, x.device, stream)


_ACTS = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


def _act(t: torch.Tensor, what: str) -> int:
    if t.dtype not in _ACTS:
        raise ValueError(f"{what} must be float32 or bfloat16")
    return _ACTS[t.dtype]


def _like(t: Optional[torch.Tensor], shape, dtype, what: str) -> None:
    """An optional argument's shape and type."""
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError(f"{what} must be {dtype} {tuple(shape)}")


class PermutedRows:
    """Rows in expert order (moe_permute): rows [cap,H]; row_of int32 [T,k], the row of each pair (-1: none); and
    moe_align's maps: sorted_ids [cap], expert_ids [cap/block], num_post_pad [1], expert_counts [E].  The maps are views
    of one tensor."""
    __slots__ = ("rows", "_maps", "_at", "_shape")

    def __init__(self, rows: torch.Tensor, maps: torch.Tensor, at, shape):
        self.rows, self._maps, self._at, self._shape = rows, maps, at, shape

    def _view(self, i: int) -> torch.Tensor:  # (as_strided: a third of the host time of a slice and a view)
        begin, end = self._at[i]
        return torch.as_strided(self._maps, (end - begin,), (1,), begin)

    row_of = property(lambda self: torch.as_strided(self._maps, self._shape, (self._shape[1], 1)))
    sorted_ids = property(lambda self: self._view(1))
    expert_ids = property(lambda self: self._view(2))
    num_post_pad = property(lambda self: self._view(3))
    expert_counts = property(lambda self: self._view(4))


def moe_permute(x: torch.Tensor, topk_ids: torch.Tensor, E: int, block: int = 1, rows=None, stream=None) -> PermutedRows:
    """Rows of x [T,H] (float32 or bfloat16) in expert order, each expert's run padded with zero rows to a multiple of
    block; rows behind the last run are left as they were (rows=: a buffer of [cap,H], moe_align_capacity's cap)."""
    T, H = x.shape
    dt = _act(x, "x")
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T or topk_ids.dtype != torch.int32:
        raise ValueError("topk_ids must be int32 [T, k]")
    handle = _begin(stream, x, topk_ids, rows)
    k = topk_ids.shape[1]
    n = T * k
    if min(E, block, k) < 1:
        raise MoeError(MOE_ERR_ARG, "moe_permute")
    cap = n + min(E, n) * (block - 1)  # (moe_align_capacity)
    rows = _out(rows, (cap, H), x.dtype, x.device, stream)
    # (one allocation for the maps, each at a multiple of 16 bytes)
    at, end = [], 0
    for size in (n, cap, cap // block, 1, E):
        at.append((end, end + size))
        end += (size + 3) & -4
    maps = _empty(end, torch.int32, x.device, stream, zero=T == 0)  # (an empty batch launches nothing)
    p = maps.data_ptr()
    _check(_lib.moe_permute(_p(x), _p(topk_ids), T, H, E, k, block, dt, _p(rows), p, p + 4 * at[1][0], p + 4 * at[2][0],
                            p + 4 * at[3][0], p + 4 * at[4][0], handle), "moe_permute")
    return PermutedRows(rows, maps, at, (T, k))


def _row_map(row_of: torch.Tensor, rows: torch.Tensor, topk_w=None):
    if row_of.dim() != 2 or row_of.dtype != torch.int32 or rows.dim() != 2:
        raise ValueError("row_of must be int32 [T, k] and rows [n, H]")
    _like(topk_w, row_of.shape, torch.float32, "topk_w")
    return row_of.shape[0], row_of.shape[1], rows.shape[0], rows.shape[1]


def moe_unpermute(rows: torch.Tensor, row_of: torch.Tensor, topk_w: Optional[torch.Tensor] = None, out=None,
                  stream=None) -> torch.Tensor:
    """out [T,H] = sum over j of topk_w[t,j] * rows[row_of[t,j]] (topk_w float32 [T,k]; None: weights of 1)."""
    T, k, n, H = _row_map(row_of, rows, topk_w)
    dt = _act(rows, "rows")
    handle = _begin(stream, rows, row_of, topk_w, out)
    out = _out(out, (T, H), rows.dtype, rows.device, stream)
    _check(_lib.moe_unpermute(_p(rows), n, _p(row_of), _p(topk_w), T, H, k, dt, _p(out), handle), "moe_unpermute")
    return out


def moe_permute_backward(d_rows: torch.Tensor, row_of: torch.Tensor, d_x=None, stream=None) -> torch.Tensor:
    """Gradient of moe_permute in x: d_x [T,H] = sum over j of d_rows[row_of[t,j]]."""
    T, k, n, H = _row_map(row_of, d_rows)
    dt = _act(d_rows, "d_rows")
    handle = _begin(stream, d_rows, row_of, d_x)
    d_x = _out(d_x, (T, H), d_rows.dtype, d_rows.device, stream)
    _check(_lib.moe_permute_backward(_p(d_rows), n, _p(row_of), T, H, k, dt, _p(d_x), handle), "moe_permute_backward")
    return d_x


def moe_unpermute_backward(d_out: torch.Tensor, rows: torch.Tensor, row_of: torch.Tensor,
                           topk_w: Optional[torch.Tensor] = None, sorted_ids=None, num_post_pad=None, d_rows=None,
                           d_w=None, stream=None):
    """Gradients of moe_unpermute: (d_rows [n,H], d_w float32 [T,k]).

    With the permutation's sorted_ids and num_post_pad its padding rows become zero; rows of d_rows that no pair
    names are else left as they were."""
    T, k, n, H = _row_map(row_of, rows, topk_w)
    dt = _act(rows, "rows")
    if d_out.shape != (T, H) or d_out.dtype != rows.dtype:
        raise ValueError("d_out must be [T, H] of rows' type")
    if (sorted_ids is None) != (num_post_pad is None):
        raise ValueError("sorted_ids and num_post_pad go together")
    _like(sorted_ids, (n,), torch.int32, "sorted_ids")
    _like(num_post_pad, (1,), torch.int32, "num_post_pad")
    handle = _begin(stream, d_out, rows, row_of, topk_w, sorted_ids, num_post_pad, d_rows, d_w)
    d_rows = _out_like(d_rows, rows, stream)
    d_w = _out(d_w, (T, k), torch.float32, rows.device, stream)
    _check(_lib.moe_unpermute_backward(_p(d_out), _p(rows), n, _p(row_of), _p(topk_w), _p(sorted_ids), _p(num_post_pad),
                                       T, H, k, dt, _p(d_rows), _p(d_w), handle), "moe_unpermute_backward")
    return d_rows, d_w


def moe_prenorm(x: torch.Tensor, w: torch.Tensor, eps: float = 1e-6, h=None, stream=None) -> torch.Tensor:
    """RMS norm of the rows of x [T,H] times w [H] (float32 or bfloat16, either with either)."""
    T, H = x.shape
    dt, wdt = _act(x, "x"), _act(w, "w")
    if w.shape != (H,):
        raise ValueError("w must be [H]")
    handle = _begin(stream, x, w, h)
    h = _out_like(h, x, stream)
    _check(_lib.moe_prenorm(_p(x), _p(w), T, H, eps, dt, wdt, _p(h), handle), "moe_prenorm")
    return h


def moe_norm_workspace_size(T: int, H: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.moe_norm_workspace_size(T, H, ctypes.byref(n)), "moe_norm_workspace_size")
    return int(n.value)


def moe_prenorm_backward(d_h: torch.Tensor, x: torch.Tensor, w: torch.Tensor, eps: float = 1e-6, d_x=None, d_w=None,
                         workspace=None, stream=None):
    """Gradients of moe_prenorm: (d_x [T,H], d_w float32 [H])."""
    T, H = x.shape
    dt, wdt = _act(x, "x"), _act(w, "w")
    if w.shape != (H,) or d_h.shape != (T, H) or d_h.dtype != x.dtype:
        raise ValueError("w must be [H] and d_h [T, H] of x's type")
    handle = _begin(stream, x, d_h, w, d_x, d_w, workspace)
    d_x = _out_like(d_x, x, stream)
    d_w = _out(d_w, (H,), torch.float32, x.device, stream)
    if workspace is None:
        workspace = _empty(moe_norm_workspace_size(T, H), torch.uint8, x.device, stream)
    _check(_lib.moe_prenorm_backward(_p(d_h), _p(x), _p(w), T, H, eps, dt, wdt, _p(d_x), _p(d_w), _p(workspace),
                                     workspace.numel(), handle), "moe_prenorm_backward")
    return d_x, d_w


_POSTNORM_RULES: dict = {}  # (the library reads them only)


def _postnorm(x, y, post_w, gate, sigmoid, scale, res_scale, next_w, eps):
    """Checked sizes and the rule of a postnorm, by reference: (T, H, type, kind of gate, rule)."""
    T, H = x.shape
    dt = _act(x, "x")
    if y.shape != (T, H) or y.dtype != x.dtype:
        raise ValueError("y must be [T, H] of x's type")
    w = post_w if post_w is not None else next_w
    wdt = dt if w is None else _act(w, "weights")
    for v in (post_w, next_w):
        if v is not None and (v.shape != (H,) or v.dtype != w.dtype):
            raise ValueError("post_w and next_w must be [H] of one type")
    kind, gdt = GATE_NONE, dt
    if gate is not None:
        kind = {(H,): GATE_CHANNEL, (T, H): GATE_FULL, (T, 1): GATE_TOKEN}.get(tuple(gate.shape))
        if kind is None:
            raise ValueError("gate must be [H], [T, 1] or [T, H]")
        gdt = _act(gate, "gate")
    # (numbers, not objects that hold one and may change)
    key = (float(eps), float(scale), float(res_scale), kind, bool(sigmoid), gdt, wdt)
    rule = _POSTNORM_RULES.get(key)
    if rule is None:
        if len(_POSTNORM_RULES) >= 256:  # (scales that change from call to call)
            _POSTNORM_RULES.clear()
        rule = _POSTNORM_RULES[key] = ctypes.byref(moe_postnorm_rule(*key))
    return T, H, dt, kind, rule


def moe_postnorm(x: torch.Tensor, y: torch.Tensor, post_w=None, gate=None, sigmoid: bool = False, scale: float = 1.0,
                 res_scale: float = 1.0, next_w=None, eps: float = 1e-6, out=None, h=None, stream=None):
    """(out, h): out = res_scale * x + scale * gate * norm(y) * post_w and h = norm(out) * next_w.

    x: the residual [T,H]; y: the block's output; post_w [H] (None: y without a norm); gate [H], [T,1] or [T,H] (None:
    1), through a sigmoid if asked; next_w [H]: the next block's norm (None: h is None).  out may be x or y."""
    T, H, dt, _, rule = _postnorm(x, y, post_w, gate, sigmoid, scale, res_scale, next_w, eps)
    handle = _begin(stream, x, y, post_w, gate, next_w, out, h)
    out = _out_like(out, x, stream)
    if next_w is not None:
        h = _out_like(h, x, stream)
    elif h is not None:
        raise ValueError("h needs next_w")
    _check(_lib.moe_postnorm(_p(x), _p(y), _p(post_w), _p(gate), _p(next_w), T, H, dt, rule, _p(out),
                             _p(h), handle), "moe_postnorm")
    return out, h


class PostnormGrads(NamedTuple):
    """Gradients of moe_postnorm (None for what the call has not): weights and a broadcast gate in float32."""
    d_x: torch.Tensor
    d_y: torch.Tensor
    d_post_w: Optional[torch.Tensor]
    d_gate: Optional[torch.Tensor]
    d_next_w: Optional[torch.Tensor]


def moe_postnorm_backward(d_out: Optional[torch.Tensor], d_h: Optional[torch.Tensor], x: torch.Tensor, y: torch.Tensor,
                          post_w=None, gate=None, sigmoid: bool = False, scale: float = 1.0, res_scale: float = 1.0,
                          next_w=None, eps: float = 1e-6, d_x=None, d_y=None, workspace=None,
                          stream=None) -> PostnormGrads:
    """Gradients of moe_postnorm from those of out and h (None: zero)."""
    T, H, dt, kind, rule = _postnorm(x, y, post_w, gate, sigmoid, scale, res_scale, next_w, eps)
    _like(d_out, (T, H), x.dtype, "d_out")
    _like(d_h, (T, H), x.dtype, "d_h")
    if d_h is not None and next_w is None:
        raise ValueError("d_h needs next_w")
    handle = _begin(stream, x, y, post_w, gate, next_w, d_out, d_h, d_x, d_y, workspace)
    dev = x.device
    d_x = _out_like(d_x, x, stream)
    d_y = _out_like(d_y, x, stream)
    d_post_w = None if post_w is None else _empty((H,), torch.float32, dev, stream)
    d_next_w = None if next_w is None else _empty((H,), torch.float32, dev, stream)
    d_gate = None
    if gate is not None:
        d_gate = _empty(gate.shape, gate.dtype if kind == GATE_FULL else torch.float32, dev, stream)
    if workspace is None:
        workspace = _empty(moe_norm_workspace_size(T, H), torch.uint8, dev, stream)
    _check(_lib.moe_postnorm_backward(_p(d_out), _p(d_h), _p(x), _p(y), _p(post_w), _p(gate), _p(next_w), T, H, dt,
                                      rule, _p(d_x), _p(d_y), _p(d_post_w), _p(d_gate), _p(d_next_w),
                                      _p(workspace), workspace.numel(), handle), "moe_postnorm_backward")
    return PostnormGrads(d_x, d_y, d_post_w, d_gate, d_next_w)


def moe_lora_workspace_size(T: int, K: int, N: int, rank: int, L: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.moe_lora_workspace_size(T, K, N, rank, L, ctypes.byref(n)), "moe_lora_workspace_size")
    return int(n.value)


def moe_lora(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, ids: torch.Tensor, scale=None, base=None,
             out_dtype: torch.dtype = torch.bfloat16, out=None, workspace=None, stream=None) -> torch.Tensor:
    """out[t] = base[t] + scale[l] * b[l] . (a[l] . x[t]) with l = ids[t] (-1: base alone).

    x bfloat16 [T,K]; a bfloat16 [L,r,K]; b bfloat16 [L,N,r]; ids int32 [T]; scale float32 [L] (None: 1); base [T,N]
    (None: 0), whose type out then has, and which may be out itself."""
    T, K = x.shape
    L, r, Ka = a.shape
    N = b.shape[1]
    if Ka != K or b.shape != (L, N, r) or ids.shape != (T,) or (scale is not None and scale.shape != (L,)):
        raise ValueError("inconsistent shapes")
    if x.dtype != torch.bfloat16 or a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16 or ids.dtype != torch.int32 or (
            scale is not None and scale.dtype != torch.float32):
        raise ValueError("x, a and b must be bfloat16, ids int32 and scale float32")
    if base is not None:
        if base.shape != (T, N) or base.dtype not in _ACTS:
            raise ValueError("base must be float32 or bfloat16 [T, N]")
        out_dtype = base.dtype
    elif out is not None:
        out_dtype = out.dtype
    handle = _begin(stream, x, a, b, ids, scale, base, out, workspace)
    out = _out(out, (T, N), out_dtype, x.device, stream) if base is None else _out_like(out, base, stream)
    dt = _act(out, "out")
    if workspace is None:
        workspace = _empty(moe_lora_workspace_size(T, K, N, r, L), torch.uint8, x.device, stream)
    _check(_lib.moe_lora(_p(x), _p(a), _p(b), _p(ids), _p(scale), _p(base), T, K, N, r, L, dt, _p(out), _p(workspace),
                         workspace.numel(), handle), "moe_lora")
    return out


_W_FORMATS = {"int4": MOE_INT4, "e4m3_block": MOE_E4M3_B128}
# no format beside the tensors' type, and names of that type
_OWN_FORMATS = (None, "", "f32", "fp32", "float32", "bf16", "bfloat16", "e4m3", "fp8", "float8_e4m3fn")


def _w_dtype(w13: torch.Tensor, w_format: Optional[str]) -> int:
    if w_format in _OWN_FORMATS:
        return _dt(w13)
    if w_format not in _W_FORMATS:
        raise ValueError(f"w_format {w_format!r}: {', '.join(_W_FORMATS)}, or the weights' own type (None)")
    return _W_FORMATS[w_format]


def _check_block_scales(w_format, E, H, I, w13, w2, w13_scale, w2_scale) -> None:
    if w_format != "e4m3_block":
        return
    if _dt(w13) != MOE_E4M3 or _dt(w2) != MOE_E4M3 or w13.shape != (E, 2 * I, H) or w2.shape != (E, H, I):
        raise ValueError("block-scaled weights must be e4m3 codes w13 [E, 2 I, H] and w2 [E, H, I]")
    for s, shape in ((w13_scale, (E, 2 * I // 128, H // 128)), (w2_scale, (E, H // 128, I // 128))):
        if s is None or s.dtype != torch.float32 or s.shape != shape:
            raise ValueError(f"block scales must be float32 {shape}")


def moe_forward(hidden: torch.Tensor, router_w: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, topk: int,
                renorm: bool, w13_scale=None, w2_scale=None, out=None, workspace=None, options=None, stream=None,
                w_format=None):
    """One fused MoE layer forward; returns out [T,H] in the activation dtype.

    w_format="int4": w13 [E,2I,H/2] and w2 [E,H,I/2] are packed INT4 codes (uint8) with bf16 group
    scales, group-major per expert: w13_scale [E,H/128,2I] and w2_scale [E,I/128,H].
    w_format="e4m3_block": w13 and w2 are e4m3 codes with one float32 scale per 128 x 128 block:
    w13_scale [E,2I/128,H/128] and w2_scale [E,H/128,I/128]."""
    T, H = hidden.shape
    E, twoI, H2 = w13.shape
    I = twoI // 2
    div = 2 if w_format == "int4" else 1
    if H2 * div != H or w2.shape != (E, H, I // div) or router_w.shape != (E, H):
        raise ValueError("inconsistent shapes")
    _check_block_scales(w_format, E, H, I, w13, w2, w13_scale, w2_scale)
    act, wdt = _dt(hidden), _w_dtype(w13, w_format)
    opts = _opts(options)
    need = moe_workspace_size(T, H, I, E, topk, act, wdt, options)
    if workspace is None:
        workspace = _empty(need, torch.uint8, hidden.device, stream)
    out = _empty(hidden.shape, hidden.dtype, hidden.device, stream) if out is None else out
    _check(_lib.moe_forward(_p(hidden), _p(router_w), _p(w13), _p(w2), T, H, I, E, topk, int(bool(renorm)), act, wdt,
                            _p(w13_scale), _p(w2_scale), _p(out), _p(workspace), workspace.numel(), opts,
                            _stream(stream)), "moe_forward")
    return out


def moe_forward_host(hidden_host: torch.Tensor, router_w: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, topk: int,
                     renorm: bool, w13_scale=None, w2_scale=None, hidden_dev=None, out_host=None, workspace=None,
                     options=None, stream=None, w_format=None):
    """The layer from pinned host memory to pinned host memory (moe_forward_host): a copy kernel
    brings hidden_host into the device staging buffer hidden_dev, and the layer stores its output
    straight into out_host, all on `stream`.  Returns out_host, complete once the stream's work is.
    hidden_host and out_host must be page-locked (Tensor.pin_memory())."""
    T, H = hidden_host.shape
    E, twoI, H2 = w13.shape
    I = twoI // 2
    div = 2 if w_format == "int4" else 1
    if H2 * div != H or w2.shape != (E, H, I // div) or router_w.shape != (E, H):
        raise ValueError("inconsistent shapes")
    _check_block_scales(w_format, E, H, I, w13, w2, w13_scale, w2_scale)
    dev = router_w.device
    act, wdt = _dt(hidden_host), _w_dtype(w13, w_format)
    need = moe_workspace_size(T, H, I, E, topk, act, wdt, options)
    if workspace is None:
        workspace = _empty(need, torch.uint8, dev, stream)
    hidden_dev = _empty(hidden_host.shape, hidden_host.dtype, dev, stream) if hidden_dev is None else hidden_dev
    out_host = torch.empty(hidden_host.shape, dtype=hidden_host.dtype).pin_memory() if out_host is None else out_host
    _check(_lib.moe_forward_host(_p(hidden_host), _p(hidden_dev), _p(router_w), _p(w13), _p(w2), T, H, I, E, topk,
                                 int(bool(renorm)), act, wdt, _p(w13_scale), _p(w2_scale), _p(out_host),
                                 _p(workspace), workspace.numel(), _opts(options), _stream(stream)),
           "moe_forward_host")
    return out_host


def moe_forward_noalloc(hidden: torch.Tensor, router_w: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, topk: int,
                        renorm: bool, w13_scale=None, w2_scale=None, out=None, options=None, stream=None,
                        w_format=None):
    """moe_forward without a workspace argument, for callers that cannot allocate device memory.

    The library keeps the workspace in its own fixed device array (NOALLOC_MAX_WORKSPACE bytes per
    device); larger shapes raise MoeError(MOE_ERR_WORKSPACE).  Pass `out` to allocate nothing here either.
    w_format="int4" takes packed INT4 weights as moe_forward does.
    """
    T, H = hidden.shape
    E, twoI, H2 = w13.shape
    I = twoI // 2
    div = 2 if w_format == "int4" else 1
    if H2 * div != H or w2.shape != (E, H, I // div) or router_w.shape != (E, H):
        raise ValueError("inconsistent shapes")
    _check_block_scales(w_format, E, H, I, w13, w2, w13_scale, w2_scale)
    wdt = _w_dtype(w13, w_format)
    out = _empty(hidden.shape, hidden.dtype, hidden.device, stream) if out is None else out
    _check(_lib.moe_forward_noalloc(_p(hidden), _p(router_w), _p(w13), _p(w2), T, H, I, E, topk, int(bool(renorm)),
                                    _dt(hidden), wdt, _p(w13_scale), _p(w2_scale), _p(out), _opts(options),
                                    _stream(stream)), "moe_forward_noalloc")
    return out


def moe_get_status(stream=None) -> int:
    return int(_lib.moe_get_status(_stream(stream)))


def moe_inv_rope_fp8_quant(x: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor, rot_dim: int,
                           q_out=None, scale_out=None, stream=None):
    """Inverse rotary embedding + per-head e4m3 quantisation of x [T, heads, head_dim] (bf16):
    (codes uint8 [T, heads, head_dim], scales float32 [T, heads])."""
    T, heads, D = x.shape
    assert x.dtype == torch.bfloat16 and x.is_contiguous()
    dev = x.device
    q_out = _empty((T, heads, D), torch.uint8, dev, stream) if q_out is None else q_out
    scale_out = _empty((T, heads), torch.float32, dev, stream) if scale_out is None else scale_out
    _check(_lib.moe_inv_rope_fp8_quant(_p(x), T, heads, D, int(rot_dim), _p(positions), _p(cos_sin),
                                       cos_sin.shape[0], _p(q_out), _p(scale_out), _stream(stream)),
           "moe_inv_rope_fp8_quant")
    return q_out, scale_out


_ROUTED_OPTIONS = moe_options(single_launch=2)  # (the library reads it only)


def moe_forward_routed(hidden: torch.Tensor, topk_w: torch.Tensor, topk_ids: torch.Tensor, w13: torch.Tensor,
                       w2: torch.Tensor, w13_scale=None, w2_scale=None, out=None, workspace=None, options=None,
                       stream=None, w_format=None):
    """Steps 3-7 of the layer on a given routing (topk_w fp32 [T,k], topk_ids int32 [T,k]; buffers of more than T
    rows and a flat topk_w serve too).

    w_format="e4m3_block": e4m3 weights with a scale per 128 x 128 block, as in moe_forward."""
    T, H = hidden.shape
    E, twoI, _ = w13.shape
    I = twoI // 2
    k = topk_ids.shape[1]
    # (any shape with the values of the first T tokens in front: buffers of a larger batch, a flat topk_w)
    if topk_ids.dtype != torch.int32 or topk_w.dtype != torch.float32 or min(topk_ids.numel(), topk_w.numel()) < T * k:
        raise ValueError("topk_w must be float32 and topk_ids int32, both with T x k values in front")
    _check_block_scales(w_format, E, H, I, w13, w2, w13_scale, w2_scale)
    act, wdt = _dt(hidden), _w_dtype(w13, w_format)
    if options is None:
        opts = _ROUTED_OPTIONS
    else:
        opts = moe_options.from_buffer_copy(options) if isinstance(options, moe_options) else _opts(options)._obj
        opts.single_launch = 2
    if workspace is None:  # (a caller's own is checked by the library)
        workspace = _empty(moe_workspace_size(T, H, I, E, k, act, wdt, opts), torch.uint8, hidden.device, stream)
    out = _empty(hidden.shape, hidden.dtype, hidden.device, stream) if out is None else out
    _check(_lib.moe_forward_routed(_p(hidden), _p(topk_w), _p(topk_ids), _p(w13), _p(w2), T, H, I, E, k, act, wdt,
                                   _p(w13_scale), _p(w2_scale), _p(out), _p(workspace), workspace.numel(),
                                   ctypes.byref(opts), _stream(stream)), "moe_forward_routed")
    return out


class ExpertCache:
    """Host-resident expert weights with a pool of `n_slots` device slots (moe_cache_* in the C ABI).

    w13 [E,2I,H] and w2 [E,H,I] are CPU tensors (pinned ones avoid a registration); the cache keeps
    references to them for its lifetime.
    """

    def __init__(self, w13: torch.Tensor, w2: torch.Tensor, n_slots: int, max_tokens: int, topk: int, w13_scale=None,
                 w2_scale=None):
        if w13.is_cuda or w2.is_cuda:
            raise ValueError("expert weights must be host tensors")
        E, twoI, H = w13.shape
        self.E, self.H, self.I, self.topk, self.n_slots = E, H, twoI // 2, topk, n_slots
        self._keep = (w13.contiguous(), w2.contiguous(),
                      None if w13_scale is None else w13_scale.float().contiguous(),
                      None if w2_scale is None else w2_scale.float().contiguous())
        h = ctypes.c_void_p(0)
        _check(_lib.moe_cache_create(_p(self._keep[0]), _p(self._keep[1]), _p(self._keep[2]), _p(self._keep[3]), E, H,
                                     self.I, _dt(w13), n_slots, max_tokens, topk, ctypes.byref(h)), "moe_cache_create")
        self._h = h

    def set_copy_mode(self, mode: int) -> None:
        """CACHE_COPY_OVERLAP (default), CACHE_COPY_SERIAL or CACHE_COPY_KERNEL."""
        _check(_lib.moe_cache_set_copy_mode(self._h, int(mode)), "moe_cache_set_copy_mode")

    def close(self):
        if self._h is not None and self._h.value:
            _lib.moe_cache_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace_size(self, T: int, act_dtype: int = MOE_BF16, options=None) -> int:
        n = ctypes.c_size_t(0)
        _check(_lib.moe_cache_workspace_size(self._h, T, act_dtype, _opts(options), ctypes.byref(n)),
               "moe_cache_workspace_size")
        return int(n.value)

    def forward(self, hidden: torch.Tensor, router_w: torch.Tensor, renorm: bool, out=None, workspace=None,
                options=None, stream=None) -> torch.Tensor:
        T = hidden.shape[0]
        if workspace is None:
            workspace = _empty(self.workspace_size(T, _dt(hidden), options), torch.uint8, hidden.device, stream)
        out = _empty(hidden.shape, hidden.dtype, hidden.device, stream) if out is None else out
        _check(_lib.moe_forward_cached(self._h, _p(hidden), _p(router_w), T, int(bool(renorm)), _dt(hidden), _p(out),
                                       _p(workspace), workspace.numel(), _opts(options), _stream(stream)),
               "moe_forward_cached")
        return out

    def stats(self) -> dict:
        st = moe_cache_stats_t()
        _check(_lib.moe_cache_stats(self._h, ctypes.byref(st)), "moe_cache_stats")
        return {n: int(getattr(st, n)) for n, _ in moe_cache_stats_t._fields_}


def moe_copy_from_host(src: torch.Tensor, dst: torch.Tensor, stream=None) -> torch.Tensor:
    """The expert cache's copy kernel: src (pinned host tensor) -> dst (device tensor, same bytes)."""
    n = src.numel() * src.element_size()
    if src.is_cuda or not dst.is_cuda or dst.numel() * dst.element_size() != n:
        raise ValueError("src must be a host tensor and dst a device tensor of the same size")
    _check(_lib.moe_copy_from_host(_p(src), _p(dst), n, _stream(stream)), "moe_copy_from_host")
    return dst


def moe_cache_lru_plan(E: int, n_slots: int, ids):
    """The cache's slot policy on a sequence of calls (ids int32 [n_calls, pairs]), host only:
    (slot_ids [n_calls, pairs], loaded_expert [n_calls, n_slots], hits, misses)."""
    import numpy as np

    ids = np.ascontiguousarray(np.asarray(ids, dtype=np.int32))
    n_calls, pairs = ids.shape
    slot_ids = np.empty_like(ids)
    loaded = np.empty((n_calls, n_slots), dtype=np.int32)
    hits, misses = ctypes.c_ulonglong(0), ctypes.c_ulonglong(0)
    _check(_lib.moe_cache_lru_plan(E, n_slots, n_calls, pairs, ids.ctypes.data_as(ctypes.c_void_p),
                                   slot_ids.ctypes.data_as(ctypes.c_void_p), loaded.ctypes.data_as(ctypes.c_void_p),
                                   ctypes.byref(hits), ctypes.byref(misses)), "moe_cache_lru_plan")
    return slot_ids, loaded, int(hits.value), int(misses.value)
