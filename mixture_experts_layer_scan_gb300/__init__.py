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
from typing import Optional

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
           "moe_route_grouped", "moe_quant_block", "moe_silu_quant_block", "moe_gemm_block")
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
