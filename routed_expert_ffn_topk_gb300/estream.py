"""Python binding of libestream (the C ABI in include/estream.h).

Argument marshalling only: torch tensors become device/host pointers, the
current torch CUDA stream becomes the ``cuda_stream`` argument, and status
codes become exceptions. Every step of the MoE layer runs in the library's
CUDA kernels; there is no other implementation behind these names, and the
module refuses to load when the library has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libestream.so")

OK, ERR_INVALID_ARG, ERR_CAPACITY, ERR_NOT_BOUND, ERR_CUDA, ERR_PAGER, ERR_TIMEOUT, \
    ERR_DEVICE, ERR_UNSUPPORTED = range(9)
F32, BF16, Q4 = 0, 1, 2
SCHED_AFTER_ROUTING, SCHED_PREFETCH = 0, 1
FFN_AUTO, FFN_SINGLE, FFN_PAIR = 0, 1, 2
PAIR_MIN_ROWS = 160
DECODE_MAX_T = 32
FP4_E4M3X16, FP4_E8M0X32 = 0, 1
_MX4_ELEM = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
KV_BF16, KV_F16, KV_E4M3 = 0, 1, 2
_KV_ELEM = {torch.bfloat16: KV_BF16, torch.float16: KV_F16, torch.float8_e4m3fn: KV_E4M3}
SAMPLE_MAX_V = 393216
STATE_NAMES = {0: "Available", 1: "Filling", 2: "Ready", 3: "InUse"}


class EStreamError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class ArenaDesc(ctypes.Structure):
    _fields_ = [
        ("L", ctypes.c_int), ("E", ctypes.c_int), ("H", ctypes.c_int), ("F", ctypes.c_int),
        ("G", ctypes.c_int), ("B", ctypes.c_int), ("Q", ctypes.c_int),
        ("wdtype", ctypes.c_int),
        ("arena_dev", ctypes.c_void_p), ("arena_bytes", ctypes.c_size_t),
        ("host_pool", ctypes.POINTER(ctypes.c_void_p)),
        ("perm", ctypes.POINTER(ctypes.c_int32)),
        ("n_shared", ctypes.c_int), ("F_shared", ctypes.c_int),
        ("shared_dev", ctypes.POINTER(ctypes.c_void_p)),
        ("T_max", ctypes.c_int), ("k_max", ctypes.c_int),
        ("deterministic", ctypes.c_int), ("schedule", ctypes.c_int),
        ("ffn_form", ctypes.c_int),
    ]


class Stats(ctypes.Structure):
    _fields_ = [
        ("calls", ctypes.c_int), ("launches", ctypes.c_int),
        ("ms_route", ctypes.c_double), ("ms_ffn", ctypes.c_double),
        ("ms_shared", ctypes.c_double),
        ("ms_combine", ctypes.c_double), ("ms_total", ctypes.c_double),
        ("n_ffn", ctypes.c_int),
        ("h2d_bytes", ctypes.c_double),
        ("groups_loaded", ctypes.c_int), ("groups_skipped", ctypes.c_int),
        ("groups_hit", ctypes.c_int),
        ("ms_io_busy", ctypes.c_double),
        ("hidden_fraction", ctypes.c_double), ("bubble_rate", ctypes.c_double),
    ]


class KvCache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("elem", ctypes.c_int), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
        ("heads", ctypes.c_int), ("dim", ctypes.c_int),
        ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
        ("k_page", ctypes.c_longlong), ("k_token", ctypes.c_longlong), ("k_head", ctypes.c_longlong),
        ("v_page", ctypes.c_longlong), ("v_token", ctypes.c_longlong), ("v_head", ctypes.c_longlong),
    ]


_lib = None
_fast = None  # the compiled part of the binding, once the library is loaded

# name -> (restype, argtypes)
_P, _I, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_L, _F = ctypes.c_longlong, ctypes.c_float
SIGNATURES = {
    "estream_status_string": (ctypes.c_char_p, [_I]),
    "estream_version": (_I, []),
    "estream_route_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "estream_route_build": (_I, [_P, _I, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "estream_workspace_error": (_I, [_P, _P]),
    "estream_route_build_noalloc": (_I, [_P, _I, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P]),
    "estream_route_noalloc_error": (_I, [_P]),
    "estream_poison_workspace": (_I, [_P, _P]),
    "estream_route_build_from_x": (_I, [_P, _I, _I, _P, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P,
                                        _P, _SZ, _P]),
    "estream_route_build_from_x_fused": (_I, [_I, _I, _I, _I]),
    "estream_moe_layer_prefill_from_x": (_I, [_P, _I, _P, _P, _I, _I, _I, _P, _P, _P, _P]),
    "estream_router_workspace_bytes": (_SZ, [_I, _I, _I]),
    "estream_router_logits": (_I, [_P, _I, _I, _P, _I, _P, _P, _SZ, _P]),
    "estream_arena_bytes": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "estream_pool_bytes": (_SZ, [_I, _I, _I, _I]),
    "estream_shared_bytes": (_SZ, [_I, _I, _I, _I]),
    "estream_pack_shared": (_I, [ctypes.POINTER(ArenaDesc), _P, _P, _P, _P]),
    "estream_bind_arena": (_I, [ctypes.POINTER(_P), ctypes.POINTER(ArenaDesc)]),
    "estream_pack_experts": (_I, [ctypes.POINTER(ArenaDesc), _I, _P, _P, _P, _P]),
    "estream_arena_preload": (_I, [_P, _I, _P]),
    "estream_arena_invalidate": (_I, [_P]),
    "estream_moe_layer_prefill": (_I, [_P, _I, _P, _P, _I, _I, _I, _P, _P]),
    "estream_moe_layer_prefill_residual": (_I, [_P, _I, _P, _P, _I, _I, _I, _P, _P, _P]),
    "estream_moe_layer_decode": (_I, [_P, _I, _P, _P, _I, _I, _I, _P, _P, _P]),
    "estream_moe_layer_decode_from_x": (_I, [_P, _I, _P, _P, _I, _I, _I, _P, _P, _P, _P]),
    "estream_mx4_code_bytes": (_SZ, [_L, _I]),
    "estream_mx4_scale_bytes": (_SZ, [_L, _I, _I]),
    "estream_mx4_weight_scale_bytes": (_SZ, [_I, _I, _I]),
    "estream_mx4_quantize": (_I, [_P, _I, _L, _I, _I, _I, _P, _I, _I, _F, _P, _P, _P]),
    "estream_mx4_dequantize": (_I, [_P, _P, _I, _F, _I, _I, _P, _I, _L, _P]),
    "estream_mx4_weight_scales": (_I, [_P, _I, _I, _I, _I, _P, _P]),
    "estream_mx4_product": (_I, [_P, _P, _I, _P, _P, _I, _I, _I, _I, _F, _P, _P, _I, _L, _P]),
    "estream_mx4_error": (_I, [_P]),
    "estream_kv_append": (_I, [_P, _I, _I, _P, _L, _L, _P, _L, _L, _P, _P, _P, _I, _I, _L, _P, _L, _L, _I, _P, _L, _L,
                              _P, _I, _I, _P]),
    "estream_kv_attend_workspace_bytes": (_SZ, [_P, _I, _I, _I, _I]),
    "estream_kv_attend": (_I, [_P, _I, _I, _I, _P, _L, _L, _P, _I, _L, _P, _F, _I, _P, _L, _L, _P, _P, _SZ, _P]),
    "estream_sample_tokens": (_I, [_P, _I, _L, _I, _I, _P, _F, _P, _I, _P, _F, _P, _F, _P, _P, _P, _P]),
    "estream_set_timing": (_I, [_P, _I]),
    "estream_reset_stats": (_I, [_P]),
    "estream_last_stats": (_I, [_P, ctypes.POINTER(Stats)]),
    "estream_get_device_error": (_I, [_P]),
    "estream_residency_trace": (_I, [_P, _P, _I, ctypes.POINTER(_I)]),
    "estream_inject_pager_fault": (_I, [_P, _I, _I]),
    "estream_inject_route_timeout": (_I, [_P]),
    "estream_inject_expert_timeout": (_I, [_P]),
    "estream_inject_late_arrival": (_I, [_P, _I]),
    "estream_pipeline_trace": (_I, [_P, _P, _I, ctypes.POINTER(_I), ctypes.POINTER(ctypes.c_double)]),
    "estream_maxplus_pipeline": (ctypes.c_double, [_P, _P, _I, _I, _I, ctypes.c_double, _P]),
    "estream_bank_bound": (_I, [_I, ctypes.c_double, ctypes.c_double, ctypes.c_double, _I]),
    "estream_autoconfig": (_I, [_I, _P, _P, _P, _P, ctypes.c_double, _I, ctypes.c_double, _P,
                                ctypes.c_double, _I, ctypes.POINTER(_I), ctypes.POINTER(_I),
                                ctypes.POINTER(ctypes.c_double)]),
    "estream_unbind": (None, [_P]),
    "estream_cast_f32_bf16": (_I, [_P, _P, _SZ, _P]),
}


def lib():
    """Load libestream.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libestream.so not found at {LIB_PATH}; build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
        _load_fast(L)
    return _lib


def _load_fast(L) -> None:
    """The compiled part of the binding, where it was built for this interpreter and this
    library: the calls of a generation step are shorter than an interpreted check of
    their arguments. Else all calls take the interpreted way."""
    global _fast
    _fast = None
    try:
        from . import _binding
        if _binding.version != L.estream_version():
            return
        address = lambda name: ctypes.cast(getattr(L, name), ctypes.c_void_p).value
        _binding.setup(address("estream_kv_append"), address("estream_kv_attend"), address("estream_kv_attend_workspace_bytes"),
                       address("estream_sample_tokens"), torch.Tensor, torch.bfloat16, torch.float16, torch.float32, torch.int32,
                       torch.uint8, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
    except (ImportError, AttributeError):
        return
    _fast = _binding


def status_string(status: int) -> str:
    return lib().estream_status_string(status).decode()


def _check(status: int, where: str) -> None:
    if status != OK:
        raise EStreamError(status, where)


def _dptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream=None, device=None):
    """The cuda_stream argument: `stream` (a torch.cuda.Stream or a raw
    handle), else the current stream of `device`. A torch stream of another
    device than `device` is refused."""
    if stream is None:
        if isinstance(device, torch.device) and device.index is not None:
            return torch._C._cuda_getCurrentRawStream(device.index)  # current_stream without its object
        stream = torch.cuda.current_stream(device)
    if hasattr(stream, "cuda_stream"):
        if device is not None and stream.device != torch.device(device):
            raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
        return stream.cuda_stream
    return stream


def _current(stream, device: torch.device):
    """`stream` as the current one: what is allocated meanwhile belongs to it, so that its
    memory is not another stream's still, and not reused before the stream is done."""
    handle = _stream(stream, device)
    if not hasattr(stream, "cuda_stream"):
        # the legacy default stream's two handles are no external streams to torch, which would make a new one
        stream = torch.cuda.default_stream(device) if handle in (0, 1) else torch.cuda.ExternalStream(handle, device)
    return torch.cuda.stream(stream)


_SAME_DEVICE = contextlib.nullcontext()


def _allocating(stream, device: torch.device):
    """Where a call that launches on `stream` allocates what it returns or works in."""
    return _SAME_DEVICE if stream is None or device.type != "cuda" else _current(stream, device)


def _on(t: torch.Tensor):
    """Makes the tensors' device current for the duration of one library call
    (the library launches on the current device, with these pointers); costs
    nothing where it is already."""
    d = t.get_device()
    return _SAME_DEVICE if d == torch.cuda.current_device() else torch.cuda.device(d)


def version() -> int:
    return lib().estream_version()


# ---------------------------------------------------------------------------
# routing + route map
# ---------------------------------------------------------------------------

def route_workspace_bytes(T: int, E: int, k: int, P: int) -> int:
    return lib().estream_route_workspace_bytes(T, E, k, P)


def _need(t: torch.Tensor, numel: int, dtype, name: str, device) -> None:
    """A buffer the library writes or reads through a plain pointer."""
    if t.dtype != dtype or t.numel() < numel or t.device != device:
        raise ValueError(f"{name} must be {dtype} with at least {numel} elements on {device}")


def _check_route_args(logits: torch.Tensor, k: int, phi, P: int, o: dict) -> None:
    if logits.dim() != 2 or logits.dtype != torch.float32 or not logits.is_cuda:
        raise ValueError("logits must be a [T, E] fp32 CUDA tensor")
    T, E = logits.shape
    R = T * k
    dev = logits.device
    if phi is not None:
        _need(phi, E, torch.int32, "phi", dev)
    _need(o["topk_ids"], R, torch.int32, "topk_ids", dev)
    _need(o["alpha"], R, torch.float32, "alpha", dev)
    _need(o["offsets"], P + 2, torch.int32, "offsets", dev)
    _need(o["rec_tok"], R, torch.int32, "rec_tok", dev)
    _need(o["rec_route"], R, torch.int32, "rec_route", dev)


def _route_outputs(o: dict, R: int, P: int, stream, dev) -> None:
    """What a route build writes and the caller did not give."""
    with _allocating(stream, dev):
        o.setdefault("topk_ids", torch.empty(max(R, 1), dtype=torch.int32, device=dev))
        o.setdefault("alpha", torch.empty(max(R, 1), dtype=torch.float32, device=dev))
        o.setdefault("offsets", torch.empty(P + 2, dtype=torch.int32, device=dev))
        o.setdefault("rec_tok", torch.empty(max(R, 1), dtype=torch.int32, device=dev))
        o.setdefault("rec_route", torch.empty(max(R, 1), dtype=torch.int32, device=dev))


def route_build(logits: torch.Tensor, k: int, renorm: bool, phi: torch.Tensor | None = None,
                P: int | None = None, out: dict | None = None, workspace: torch.Tensor | None = None,
                stream=None) -> dict:
    """estream_route_build on device tensors. Returns a dict with topk_ids,
    alpha, offsets, rec_tok, rec_route (allocated when not given in ``out``)."""
    T, E = logits.shape
    P = E if P is None else P
    dev = logits.device
    R = T * k
    o = dict(out or {})
    _route_outputs(o, R, P, stream, dev)
    _check_route_args(logits, k, phi, P, o)
    nbytes = route_workspace_bytes(T, E, k, P)
    if workspace is None:
        with _allocating(stream, dev):
            workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    if workspace.device != dev:
        raise ValueError(f"workspace must be on {dev}")
    with _on(logits):
        st = lib().estream_route_build(
            _dptr(logits), T, E, k, int(bool(renorm)), _dptr(phi), P, _dptr(o["topk_ids"]),
            _dptr(o["alpha"]), _dptr(o["offsets"]), _dptr(o["rec_tok"]), _dptr(o["rec_route"]),
            _dptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream, dev))
    _check(st, "estream_route_build")
    o["workspace"] = workspace
    return o


def router_workspace_bytes(T: int, H: int, E: int) -> int:
    return lib().estream_router_workspace_bytes(T, H, E)


def router_logits(X: torch.Tensor, W_r: torch.Tensor, logits: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """estream_router_logits: logits [T, E] fp32 = X [T, H] bf16 @ W_r [E, H] bf16 ^T."""
    if (X.dim() != 2 or W_r.dim() != 2 or X.dtype != torch.bfloat16 or W_r.dtype != torch.bfloat16
            or W_r.shape[1] != X.shape[1]):
        raise ValueError("X must be [T, H] and W_r [E, H], both bf16")
    if not X.is_cuda or W_r.device != X.device:
        raise ValueError("X and W_r must be on one CUDA device")
    T, H = X.shape
    E = W_r.shape[0]
    with _allocating(stream, X.device):
        if logits is None:
            logits = torch.empty(T, E, dtype=torch.float32, device=X.device)
        if workspace is None:
            workspace = torch.empty(max(router_workspace_bytes(T, H, E), 256), dtype=torch.uint8,
                                    device=X.device)
    if tuple(logits.shape) != (T, E) or logits.dtype != torch.float32 or logits.device != X.device:
        raise ValueError(f"logits must be [{T}, {E}] fp32 on X's device")
    if workspace.device != X.device:
        raise ValueError("workspace must be on X's device")
    with _on(X):
        st = lib().estream_router_logits(_dptr(X), T, H, _dptr(W_r), E, _dptr(logits),
                                         _dptr(workspace), workspace.numel() * workspace.element_size(),
                                         _stream(stream, X.device))
    _check(st, "estream_router_logits")
    return logits


def route_build_from_x(X: torch.Tensor, W_r: torch.Tensor, k: int, renorm: bool,
                       phi: torch.Tensor | None = None, P: int | None = None, out: dict | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> dict:
    """estream_route_build_from_x: router logits X W_r^T and the route map in
    one call. Returns route_build's dict plus "logits" [T, E] fp32."""
    if (X.dim() != 2 or W_r.dim() != 2 or X.dtype != torch.bfloat16 or W_r.dtype != torch.bfloat16
            or W_r.shape[1] != X.shape[1]):
        raise ValueError("X must be [T, H] and W_r [E, H], both bf16")
    if not X.is_cuda or W_r.device != X.device:
        raise ValueError("X and W_r must be on one CUDA device")
    T, H = X.shape
    E = W_r.shape[0]
    P = E if P is None else P
    dev = X.device
    R = T * k
    o = dict(out or {})
    with _allocating(stream, dev):
        o.setdefault("logits", torch.empty(T, E, dtype=torch.float32, device=dev))
    _route_outputs(o, R, P, stream, dev)
    if tuple(o["logits"].shape) != (T, E) or o["logits"].dtype != torch.float32 \
            or o["logits"].device != dev:
        raise ValueError(f"logits must be [{T}, {E}] fp32 on X's device")
    _check_route_args(o["logits"], k, phi, P, o)
    nbytes = route_workspace_bytes(T, E, k, P)
    if workspace is None:
        with _allocating(stream, dev):
            workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    if workspace.device != dev:
        raise ValueError(f"workspace must be on {dev}")
    with _on(X):
        st = lib().estream_route_build_from_x(
            _dptr(X), T, H, _dptr(W_r), E, k, int(bool(renorm)), _dptr(phi), P, _dptr(o["logits"]),
            _dptr(o["topk_ids"]), _dptr(o["alpha"]), _dptr(o["offsets"]), _dptr(o["rec_tok"]),
            _dptr(o["rec_route"]), _dptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(stream, dev))
    _check(st, "estream_route_build_from_x")
    o["workspace"] = workspace
    return o


def route_build_from_x_fused(T: int, H: int, E: int, P: int | None = None) -> bool:
    """Whether route_build_from_x runs these sizes as one fused launch on
    the current device."""
    return bool(lib().estream_route_build_from_x_fused(T, H, E, E if P is None else P))


def route_build_noalloc(logits: torch.Tensor, k: int, renorm: bool, phi: torch.Tensor | None = None,
                        P: int | None = None, out: dict | None = None, stream=None) -> dict:
    """estream_route_build_noalloc: the same outputs as route_build, with the
    library's static device scratch instead of a caller workspace."""
    T, E = logits.shape
    P = E if P is None else P
    dev = logits.device
    R = T * k
    o = dict(out or {})
    _route_outputs(o, R, P, stream, dev)
    _check_route_args(logits, k, phi, P, o)
    with _on(logits):
        st = lib().estream_route_build_noalloc(
            _dptr(logits), T, E, k, int(bool(renorm)), _dptr(phi), P, _dptr(o["topk_ids"]),
            _dptr(o["alpha"]), _dptr(o["offsets"]), _dptr(o["rec_tok"]), _dptr(o["rec_route"]),
            _stream(stream, dev))
    _check(st, "estream_route_build_noalloc")
    return o


def route_noalloc_error(device=None, stream=None) -> int:
    """estream_route_noalloc_error on `device` (default: the current one):
    the status the latest allocation-free route build there recorded."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        return lib().estream_route_noalloc_error(_stream(stream, device))


def workspace_error(workspace: torch.Tensor, stream=None) -> int:
    with _on(workspace):
        return lib().estream_workspace_error(_dptr(workspace), _stream(stream, workspace.device))


def cast_f32_bf16(src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    if (src.dtype != torch.float32 or dst.dtype != torch.bfloat16 or src.numel() != dst.numel()
            or not src.is_cuda or dst.device != src.device):
        raise ValueError("src must be fp32 and dst bf16 of the same size, on one CUDA device")
    with _on(src):
        _check(lib().estream_cast_f32_bf16(_dptr(src), _dptr(dst), src.numel(),
                                           _stream(stream, src.device)), "estream_cast_f32_bf16")


# ---------------------------------------------------------------------------
# arena / layer
# ---------------------------------------------------------------------------

def arena_bytes(E, H, F, G, B, wdtype) -> int:
    return lib().estream_arena_bytes(E, H, F, G, B, wdtype)


def pool_bytes(E, H, F, wdtype) -> int:
    return lib().estream_pool_bytes(E, H, F, wdtype)


def shared_bytes(n_shared, H, F_shared, wdtype) -> int:
    return lib().estream_shared_bytes(n_shared, H, F_shared, wdtype)


def pack_shared(desc: ArenaDesc, sg: torch.Tensor, su: torch.Tensor, sd: torch.Tensor,
                out: torch.Tensor) -> None:
    for t in (sg, su, sd, out):
        assert t.device.type == "cpu" and t.is_contiguous()
    _check(lib().estream_pack_shared(ctypes.byref(desc), sg.data_ptr(), su.data_ptr(),
                                     sd.data_ptr(), out.data_ptr()), "estream_pack_shared")


def make_desc(L, E, H, F, G, B, wdtype, arena: torch.Tensor, pools, perm=None, n_shared=0,
              F_shared=0, shared=None, T_max=1, k_max=1, deterministic=False,
              schedule=SCHED_AFTER_ROUTING, Q=1, ffn_form=FFN_AUTO):
    """Fill an ArenaDesc; returns (desc, keepalive) -- keep both alive while bound."""
    d = ArenaDesc()
    d.L, d.E, d.H, d.F, d.G, d.B, d.Q = L, E, H, F, G, B, Q
    d.wdtype = wdtype
    d.arena_dev = arena.data_ptr() if arena is not None else None
    d.arena_bytes = arena.numel() * arena.element_size() if arena is not None else 0
    pool_arr = (ctypes.c_void_p * L)(*[p.data_ptr() if p is not None else None for p in pools])
    d.host_pool = ctypes.cast(pool_arr, ctypes.POINTER(ctypes.c_void_p))
    keep = [pool_arr]
    if perm is not None:
        perm_arr = (ctypes.c_int32 * (L * E))(*[int(v) for v in torch.as_tensor(perm).reshape(-1).tolist()])
        d.perm = ctypes.cast(perm_arr, ctypes.POINTER(ctypes.c_int32))
        keep.append(perm_arr)
    d.n_shared, d.F_shared = n_shared, F_shared
    if n_shared and shared is not None:
        sh_arr = (ctypes.c_void_p * L)(*[s.data_ptr() for s in shared])
        d.shared_dev = ctypes.cast(sh_arr, ctypes.POINTER(ctypes.c_void_p))
        keep.append(sh_arr)
    d.T_max, d.k_max = T_max, k_max
    d.deterministic = int(bool(deterministic))
    d.schedule = schedule
    d.ffn_form = ffn_form
    return d, keep


def pack_experts(desc: ArenaDesc, layer: int, wg: torch.Tensor, wu: torch.Tensor, wd: torch.Tensor,
                 pool_out: torch.Tensor) -> None:
    for t in (wg, wu, wd, pool_out):
        assert t.device.type == "cpu" and t.is_contiguous()
    _check(lib().estream_pack_experts(ctypes.byref(desc), layer, wg.data_ptr(), wu.data_ptr(),
                                      wd.data_ptr(), pool_out.data_ptr()), "estream_pack_experts")


def bind_arena(desc: ArenaDesc) -> int:
    ctx = ctypes.c_void_p()
    _check(lib().estream_bind_arena(ctypes.byref(ctx), ctypes.byref(desc)), "estream_bind_arena")
    return ctx.value


def arena_preload(ctx, layer: int, stream=None) -> None:
    _check(lib().estream_arena_preload(ctx, layer, _stream(stream)), "estream_arena_preload")


def arena_invalidate(ctx) -> None:
    _check(lib().estream_arena_invalidate(ctx), "estream_arena_invalidate")


def _check_layer_args(X: torch.Tensor, logits: torch.Tensor | None, Y: torch.Tensor,
                      A: torch.Tensor | None = None) -> None:
    """Shapes and types the layer call reads and writes through plain
    pointers: X [T, H] (bf16 or fp32), logits [T, E] fp32 (when given), Y
    [T, H] fp32 and the residual A like X, all on one CUDA device."""
    if X.dim() != 2 or Y.dim() != 2 or (logits is not None and logits.dim() != 2):
        raise ValueError("X, logits and Y must be 2-d")
    shape, dtype, dev = X.shape, X.dtype, X.device
    T, H = shape
    if (logits is not None and logits.shape[0] != T) or Y.shape != shape:
        raise ValueError(f"logits must be [T, E] and Y [T, H] with T={T}, H={H}")
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("X must be bf16 or fp32")
    if (logits is not None and logits.dtype != torch.float32) or Y.dtype != torch.float32:
        raise ValueError("logits and Y must be fp32")
    if A is not None and A is not X and (A.shape != shape or A.dtype != dtype or A.device != dev):
        raise ValueError("the residual must have X's shape and type, on its device")
    if dev.type != "cuda" or Y.device != dev or (logits is not None and logits.device != dev):
        raise ValueError("X, logits, Y (and the residual) must be on one CUDA device")


def moe_layer_prefill(ctx, layer: int, X: torch.Tensor, logits: torch.Tensor, k: int,
                      renorm: bool, Y: torch.Tensor, stream=None) -> None:
    _check_layer_args(X, logits, Y)
    T = X.shape[0]
    with _on(X):
        _check(lib().estream_moe_layer_prefill(ctx, layer, _dptr(X), _dptr(logits), T, k,
                                               int(bool(renorm)), _dptr(Y), _stream(stream, X.device)),
               "estream_moe_layer_prefill")


def moe_layer_prefill_residual(ctx, layer: int, X: torch.Tensor, logits: torch.Tensor, k: int,
                               renorm: bool, A: torch.Tensor, Y: torch.Tensor, stream=None) -> None:
    """Y = A + the layer's MoE output (Y written, not read)."""
    _check_layer_args(X, logits, Y, A)
    T = X.shape[0]
    with _on(X):
        _check(lib().estream_moe_layer_prefill_residual(ctx, layer, _dptr(X), _dptr(logits), T, k,
                                                        int(bool(renorm)), _dptr(A), _dptr(Y),
                                                        _stream(stream, X.device)),
               "estream_moe_layer_prefill_residual")


def moe_layer_prefill_from_x(ctx, layer: int, X: torch.Tensor, W_r: torch.Tensor, k: int,
                             renorm: bool, Y: torch.Tensor, A: torch.Tensor | None = None,
                             logits_out: torch.Tensor | None = None, stream=None) -> None:
    """Routing from the layer input (router logits, top-k and route map in
    one launch), then the experts: Y += MoE(X), or Y = A + MoE(X)."""
    if W_r.dim() != 2 or W_r.dtype != torch.bfloat16 or W_r.shape[1] != X.shape[1] \
            or W_r.device != X.device:
        raise ValueError("W_r must be [E, H] bf16 on X's device")
    T = X.shape[0]
    E = W_r.shape[0]
    if logits_out is not None and tuple(logits_out.shape) != (T, E):
        raise ValueError(f"logits_out must be [{T}, {E}]")
    _check_layer_args(X, logits_out, Y, A)
    with _on(X):
        _check(lib().estream_moe_layer_prefill_from_x(ctx, layer, _dptr(X), _dptr(W_r), T, k,
                                                      int(bool(renorm)), _dptr(A), _dptr(Y),
                                                      _dptr(logits_out), _stream(stream, X.device)),
               "estream_moe_layer_prefill_from_x")


def moe_layer_decode(ctx, layer: int, X: torch.Tensor, logits: torch.Tensor, k: int, renorm: bool,
                     Y: torch.Tensor, A: torch.Tensor | None = None, stream=None) -> None:
    """The layer for at most DECODE_MAX_T tokens, in one launch: Y += MoE(X), or
    Y = A + MoE(X). The layer must be resident in the arena."""
    _check_layer_args(X, logits, Y, A)
    T = X.shape[0]
    with _on(X):
        _check(lib().estream_moe_layer_decode(ctx, layer, _dptr(X), _dptr(logits), T, k,
                                              int(bool(renorm)), _dptr(A), _dptr(Y),
                                              _stream(stream, X.device)), "estream_moe_layer_decode")


def moe_layer_decode_from_x(ctx, layer: int, X: torch.Tensor, W_r: torch.Tensor, k: int, renorm: bool,
                            Y: torch.Tensor, A: torch.Tensor | None = None,
                            logits_out: torch.Tensor | None = None, stream=None) -> None:
    """moe_layer_decode with the router logits X W_r^T formed in the same launch."""
    if W_r.dim() != 2 or W_r.dtype != torch.bfloat16 or W_r.shape[1] != X.shape[1] \
            or W_r.device != X.device:
        raise ValueError("W_r must be [E, H] bf16 on X's device")
    T = X.shape[0]
    if logits_out is not None and tuple(logits_out.shape) != (T, W_r.shape[0]):
        raise ValueError(f"logits_out must be [{T}, {W_r.shape[0]}]")
    _check_layer_args(X, logits_out, Y, A)
    with _on(X):
        _check(lib().estream_moe_layer_decode_from_x(ctx, layer, _dptr(X), _dptr(W_r), T, k,
                                                     int(bool(renorm)), _dptr(A), _dptr(Y),
                                                     _dptr(logits_out), _stream(stream, X.device)),
               "estream_moe_layer_decode_from_x")


# ---------------------------------------------------------------------------
# microscaled 4-bit floating point
# ---------------------------------------------------------------------------

def mx4_padded(K: int) -> int:
    """Values a quantised row of K is padded to."""
    return -(-K // 32) * 32


def mx4_block(fmt: int) -> int:
    """Values that share a scale."""
    if fmt not in (FP4_E4M3X16, FP4_E8M0X32):
        raise ValueError(f"unknown 4-bit format {fmt}")
    return 16 if fmt == FP4_E4M3X16 else 32


def mx4_tensor_scale(amax: float, fmt: int) -> float:
    """A tensor scale for data whose largest magnitude is amax: for E4M3 block
    scales the power of two that puts the largest of them in (224, 448] (exact
    to divide by, and every value exact in bf16), 1 for E8M0 ones."""
    if mx4_block(fmt) == 32 or not amax > 0.0 or math.isinf(amax):
        return 1.0
    return 2.0 ** max(-100, min(100, math.ceil(math.log2(amax / (6.0 * 448.0)))))


class Mx4:
    """Quantised rows: codes [R, Kp/2] and scales [R, Kp/block] (uint8, contiguous,
    on one CUDA device), the width K, the format and the tensor scale."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, K: int, fmt: int, scale: float = 1.0):
        Kp, b = mx4_padded(K), mx4_block(fmt)
        if K < 1 or codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or codes.dim() != 2:
            raise ValueError("codes and scales must be 2-d uint8 tensors of K >= 1 values a row")
        R = codes.shape[0]
        if tuple(codes.shape) != (R, Kp // 2) or tuple(scales.shape) != (R, Kp // b):
            raise ValueError(f"codes must be [R, {Kp // 2}] and scales [R, {Kp // b}] for K = {K}")
        if not codes.is_cuda or scales.device != codes.device:
            raise ValueError("codes and scales must be on one CUDA device")
        if not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes and scales must be contiguous")
        self.K, self.fmt, self.scale, self.device = K, fmt, float(scale), codes.device
        self._codes, self._scales, self._buf, self._R = codes, scales, None, R

    @classmethod
    def _empty(cls, R, K, Kp, b, fmt, scale, device):
        """Uninitialised rows, of sizes already checked: one allocation, the codes and
        then the scales, which become tensors when they are asked for (an operation
        of PyTorch costs the host as long as a launch)."""
        q = cls.__new__(cls)
        q._buf = torch.empty(R * (Kp // 2 + Kp // b), dtype=torch.uint8, device=device)
        q._codes = q._scales = None
        q.K, q.fmt, q.scale, q.device, q._R = K, fmt, float(scale), device, R
        return q

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            row = mx4_padded(self.K) // 2
            self._codes = self._buf[:self._R * row].view(self._R, row)
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            Kp = mx4_padded(self.K)
            self._scales = self._buf[self._R * (Kp // 2):].view(self._R, Kp // mx4_block(self.fmt))
        return self._scales

    def _ptrs(self):
        """Addresses of the codes and the scales."""
        if self._buf is None:
            return self._codes.data_ptr(), self._scales.data_ptr()
        p = self._buf.data_ptr()
        return p, p + self._R * (mx4_padded(self.K) // 2)

    @property
    def shape(self):
        return self._R, self.K


class Mx4Weights:
    """Weights [P, N, K] of mx4_product: quantised codes [P, N, Kp/2] and the scale
    tiles made by mx4_weights."""

    def __init__(self, codes, tiles, K, fmt, scale):
        self.codes, self.tiles, self.K, self.fmt, self.scale = codes, tiles, K, fmt, float(scale)

    @property
    def shape(self):
        return self.codes.shape[0], self.codes.shape[1], self.K


def _row_stride(t: torch.Tensor, name: str) -> int:
    """Elements between the rows of a 2-d tensor whose rows are contiguous."""
    shape, st = t.shape, t.stride()
    if len(shape) != 2 or (shape[1] > 1 and st[1] != 1):
        raise ValueError(f"{name} must be 2-d with contiguous rows")
    ld = st[0] if shape[0] > 1 else shape[1]
    if ld < shape[1]:
        raise ValueError(f"{name} must not have overlapping rows")
    return ld


def mx4_quantize(x: torch.Tensor, fmt: int, scale: float = 1.0, rows: torch.Tensor | None = None,
                 swiglu: bool = False, out: Mx4 | None = None, stream=None) -> Mx4:
    """Rows of x [n, K] (bf16, fp16 or fp32; rows may be strided) to 4-bit codes
    with a scale per block. rows [R] int32 gathers source rows (a route map's
    rec_tok); swiglu takes x [n, 2K] as gate | up and quantises SiLU(gate) * up."""
    elem = _MX4_ELEM.get(x.dtype)
    if elem is None or not x.is_cuda:
        raise ValueError("x must be a bf16, fp16 or fp32 CUDA tensor")
    ld = _row_stride(x, "x")
    n, K = x.shape
    if swiglu:
        if K % 2:
            raise ValueError("swiglu needs an even number of columns (gate | up)")
        K //= 2
    b = mx4_block(fmt)
    if K < 1:
        raise ValueError("x must have at least one column")
    dev = x.device
    R, rp = n, None
    if rows is not None:
        if rows.dim() != 1 or rows.dtype != torch.int32 or rows.device != dev:
            raise ValueError("rows must be a 1-d int32 tensor on x's device")
        R, rp = rows.numel(), _dptr(rows)
    if out is None:
        with _allocating(stream, dev):
            out = Mx4._empty(R, K, mx4_padded(K), b, fmt, scale, dev)
    elif out.shape != (R, K) or out.fmt != fmt or out.device != dev:
        raise ValueError(f"out must hold {R} rows of {K} in this format on x's device")
    else:
        out.scale = float(scale)
    cp, sp = out._ptrs()
    with _on(x):
        st = lib().estream_mx4_quantize(x.data_ptr(), elem, ld, n, R, K, rp, 1 if swiglu else 0, fmt, out.scale,
                                        cp, sp, _stream(stream, dev))
    if st:
        _check(st, "estream_mx4_quantize")
    return out


def mx4_dequantize(q: Mx4, dtype=torch.float32, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values [R, K] that quantised rows stand for (bf16, fp16 or fp32)."""
    R, K, dev = q._R, q.K, q.device
    if out is None:
        with _allocating(stream, dev):
            out, ld = torch.empty((R, K), dtype=dtype, device=dev), K
    else:
        if tuple(out.shape) != (R, K) or out.device != dev:
            raise ValueError(f"out must be [{R}, {K}] on the codes' device")
        ld = _row_stride(out, "out")
    elem = _MX4_ELEM.get(out.dtype)
    if elem is None:
        raise ValueError("out must be bf16, fp16 or fp32")
    cp, sp = q._ptrs()
    with _on(out):
        st = lib().estream_mx4_dequantize(cp, sp, q.fmt, q.scale, R, K,
                                          out.data_ptr(), elem, ld, _stream(stream, dev))
    if st:
        _check(st, "estream_mx4_dequantize")
    return out


def mx4_weights(codes: torch.Tensor, scales: torch.Tensor, K: int, fmt: int, scale: float = 1.0,
                stream=None) -> Mx4Weights:
    """Weights of mx4_product from quantised rows: codes [N, Kp/2] or [P, N, Kp/2]
    with their scales (the codes are kept, the scales laid out once)."""
    if codes.dim() == 2:
        codes, scales = codes.unsqueeze(0), scales.unsqueeze(0)
    Kp, b = mx4_padded(K), mx4_block(fmt)
    if codes.dim() != 3 or codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or K < 1:
        raise ValueError("codes and scales must be uint8 [P, N, ...]")
    P, N = codes.shape[:2]
    if P < 1 or N < 1 or tuple(codes.shape) != (P, N, Kp // 2) or tuple(scales.shape) != (P, N, Kp // b):
        raise ValueError(f"codes must be [P, N, {Kp // 2}] and scales [P, N, {Kp // b}] for K = {K}")
    if not codes.is_cuda or scales.device != codes.device:
        raise ValueError("codes and scales must be on one CUDA device")
    with _allocating(stream, codes.device):
        tiles = torch.empty(lib().estream_mx4_weight_scale_bytes(P, N, K), dtype=torch.uint8, device=codes.device)
    with _on(codes):
        _check(lib().estream_mx4_weight_scales(_dptr(scales), P, N, K, fmt, _dptr(tiles),
                                               _stream(stream, codes.device)), "estream_mx4_weight_scales")
    if not codes.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return Mx4Weights(codes, tiles, K, fmt, scale)


def mx4_product(x: Mx4, w: Mx4Weights, offsets: torch.Tensor | None = None, out: torch.Tensor | None = None,
                out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """x [R, K] times w [P, N, K] transposed, both quantised in one format:
    [R, N] in bf16 or fp32. With offsets [P + 1] int32 (a route map's), rows
    [offsets[p], offsets[p + 1]) meet w[p], and rows outside every slot are zero."""
    R, K, dev = x._R, x.K, x.device
    P, N = w.codes.shape[:2]
    if K != w.K or x.fmt != w.fmt or w.codes.device != dev:
        raise ValueError("x and w must have one width and format, on one device")
    op = None
    if offsets is not None:
        _need(offsets, P + 1, torch.int32, "offsets", dev)
        op = _dptr(offsets)
    elif P != 1:
        raise ValueError("weights of several slots need offsets")
    if out is None:
        with _allocating(stream, dev):
            out, ld = torch.empty((R, N), dtype=out_dtype, device=dev), N
    else:
        if tuple(out.shape) != (R, N) or out.device != dev:
            raise ValueError(f"out must be [{R}, {N}] on x's device")
        ld = _row_stride(out, "out")
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out must be bf16 or fp32")
    cp, sp = x._ptrs()
    with _on(out):
        st = lib().estream_mx4_product(cp, sp, R, w.codes.data_ptr(),
                                       w.tiles.data_ptr(), P, N, K, x.fmt, x.scale * w.scale, op, out.data_ptr(),
                                       _MX4_ELEM[out.dtype], ld, _stream(stream, dev))
    if st:
        _check(st, "estream_mx4_product")
    return out


def mx4_error(device=None, stream=None) -> int:
    """estream_mx4_error on `device` (default: the current one): the first error
    that product kernels recorded there since the last call."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        return lib().estream_mx4_error(_stream(stream, device))


# ---------------------------------------------------------------------------
# paged key-value cache
# ---------------------------------------------------------------------------

class PagedKV:
    """Keys and values in pages: k, v [pages, page_size, heads, dim] (bf16, fp16 or
    float8_e4m3fn; dim contiguous, the other strides any, so a cache stored head by
    head is given as a transposed view). With E4M3 the value of an element is the
    element times k_scale or v_scale. The tensors stay the caller's; they are kept
    alive by this object."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: float = 1.0, v_scale: float = 1.0):
        elem = _KV_ELEM.get(k.dtype)
        if elem is None or v.dtype != k.dtype or not k.is_cuda or v.device != k.device:
            raise ValueError("k and v must be bf16, fp16 or float8_e4m3fn, of one type on one CUDA device")
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must be [pages, page_size, heads, dim]")
        pages, page, heads, dim = k.shape
        if page < 1 or not 1 <= heads <= 1024 or dim % 16 or not 16 <= dim <= 256 or max(pages, page) > 1 << 30:
            raise ValueError("1 to 1024 heads, dim a multiple of 16 up to 256, and pages of at least one token")
        unit = 16 // k.element_size()
        for t in (k, v):
            if t.stride(3) != 1 or t.data_ptr() % 16 or any(
                    n > 1 and (s < dim or s % unit) for n, s in zip(t.shape[:3], t.stride()[:3])):
                raise ValueError("rows of dim must be contiguous, start on 16 bytes and not overlap")
        if not all(2.0 ** -100 <= s <= 2.0 ** 100 and (elem == KV_E4M3 or s == 1.0) for s in (k_scale, v_scale)):
            raise ValueError("scales must be between 2^-100 and 2^100, and 1 for 16-bit caches")
        self.k, self.v, self.k_scale, self.v_scale = k, v, float(k_scale), float(v_scale)
        self.dtype, self.device, self.heads, self.dim, self.page_size = k.dtype, k.device, heads, dim, page
        self._scale = dim ** -0.5
        self._desc = KvCache(k.data_ptr(), v.data_ptr(), elem, pages, page, heads, dim, k_scale, v_scale,
                             *k.stride()[:3], *v.stride()[:3])
        self._ref, self._address = ctypes.byref(self._desc), ctypes.addressof(self._desc)
        lib()
        self._workspaces = {}
        self._elem, self._index = elem, k.get_device()

    def attend_workspace_bytes(self, B: int, Hq: int, M: int, window: int = 0) -> int:
        """Bytes of kv_attend's workspace for B rows of Hq heads and tables of M pages."""
        n = self._workspaces.get((B, Hq, M, window))
        if n is None:
            with torch.cuda.device(self.device):
                n = lib().estream_kv_attend_workspace_bytes(self._ref, B, Hq, M, window)
            if len(self._workspaces) < 256:
                self._workspaces[B, Hq, M, window] = n
        return n


def _kv_bad(t: torch.Tensor, n: int, heads: int | None, cache: PagedKV, name: str, dtype):
    """Why a tensor is not [n, heads, dim] next to the cache."""
    if t.dim() != 3 or t.shape[0] != n or (heads is not None and t.shape[1] != heads) or t.shape[2] != cache.dim:
        return ValueError(f"{name} must be [{n}, {'heads' if heads is None else heads}, {cache.dim}]")
    if t.dtype is not dtype:
        return ValueError(f"{name} must be {dtype}, as the call's other rows")
    return ValueError(f"{name} must have contiguous rows of dim that do not overlap, on the cache's device")


def _kv_dtype(t: torch.Tensor, cache: PagedKV, name: str) -> int:
    """The element type of a call's rows."""
    elem = _KV_ELEM.get(t.dtype)
    if elem != cache._elem and (cache._elem != KV_E4M3 or elem is None):
        raise ValueError(f"{name} must be of the cache's type, or bf16 or fp16 next to an E4M3 cache")
    if elem == KV_E4M3:
        raise ValueError(f"{name} must be bf16 or fp16")
    return elem


def _kv_ints(t: torch.Tensor, n: int, name: str, cache: PagedKV) -> int:
    if t.dtype is not torch.int32 or t.shape != (n,) or t.get_device() != cache._index or not t.is_contiguous():
        raise ValueError(f"{name} must be [{n}] int32, contiguous, on the cache's device")
    return t.data_ptr()


def _kv_table(t: torch.Tensor, cache: PagedKV):
    """A page table's address, rows, columns and the elements between rows."""
    if t.dtype is not torch.int32 or t.dim() != 2 or t.get_device() != cache._index:
        raise ValueError("table must be [B, M] int32 on the cache's device")
    (B, M), (row, one) = t.shape, t.stride()
    if one != 1 and M > 1:
        raise ValueError("table must have contiguous rows")
    if max(B, M) > 1 << 30:
        raise ValueError("a table has at most 2^30 rows and columns")
    return t.data_ptr(), B, M, row


def _kv_run(name: str, index: int, args) -> None:
    """One call on the cache's device."""
    fn = getattr(_lib or lib(), name)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args)
    else:
        with torch.cuda.device(index):
            st = fn(*args)
    if st:
        _check(st, name)


def kv_append(cache: PagedKV, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, table: torch.Tensor,
              rows: torch.Tensor | None = None, q: torch.Tensor | None = None, inv_freq: torch.Tensor | None = None,
              interleaved: bool = False, q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Stores keys and values [T, heads, dim] of new tokens at their positions [T]
    int32 of the sequences whose pages are table [B, M] int32 (rows [T]: the
    tokens' table rows; without it token t has row t). With inv_freq [rot / 2]
    fp32 the keys, and q [T, Hq, dim], are rotated by position; returns the rotated
    queries (q_out, which may be q). A token with a negative position is skipped;
    one without a valid page is not stored and its queries become NaNs."""
    if stream is not None:
        with _current(stream, cache.device):
            return kv_append(cache, k, v, positions, table, rows, q, inv_freq, interleaved, q_out)
    if _fast is not None and (q_out is not None or q is None):
        st = _fast.kv_append(cache._address, cache._index, k, v, positions, table, rows, q, inv_freq, interleaved, q_out)
        if st == 0:
            return q_out
        if st is not None:
            _check(st, "estream_kv_append")
    elem, dt, heads, dim, index = _kv_dtype(k, cache, "k"), k.dtype, cache.heads, cache.dim, cache._index
    T = k.shape[0]
    if T > 1 << 30:
        raise ValueError("at most 2^30 tokens a call")
    k0, k1, k2 = k.stride() if k.dim() == 3 else (0, 0, 0)
    if k2 != 1 or k.shape != (T, heads, dim) or k.get_device() != index:
        raise _kv_bad(k, T, heads, cache, "k", dt)
    v0, v1, v2 = v.stride() if v.dim() == 3 else (0, 0, 0)
    if v2 != 1 or v.dtype is not dt or v.shape != (T, heads, dim) or v.get_device() != index:
        raise _kv_bad(v, T, heads, cache, "v", dt)
    tp, B, M, table_row = _kv_table(table, cache)
    if rows is None and B < T:
        raise ValueError("table must have a row for each token, or rows must name them")
    Hq = rot = q0 = q1 = o0 = o1 = 0
    qp = op = fp = None
    if q is not None:
        q0, q1, q2 = q.stride() if q.dim() == 3 else (0, 0, 0)
        Hq = q.shape[1] if q2 == 1 else 0
        if q2 != 1 or q.dtype is not dt or q.shape != (T, Hq, dim) or q.get_device() != index:
            raise _kv_bad(q, T, None, cache, "q", dt)
        if q_out is None:
            q_out = torch.empty((T, Hq, dim), dtype=dt, device=cache.device)
        o0, o1, o2 = q_out.stride() if q_out.dim() == 3 else (0, 0, 0)
        if o2 != 1 or q_out.dtype is not dt or q_out.shape != (T, Hq, dim) or q_out.get_device() != index \
                or (T > 1 and o0 < dim) or (Hq > 1 and o1 < dim):
            raise _kv_bad(q_out, T, Hq, cache, "q_out", dt)
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        if inv_freq.dtype is not torch.float32 or inv_freq.dim() != 1 or rot > dim \
                or inv_freq.get_device() != index or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be [rot / 2] fp32, contiguous, with rot at most dim, on the cache's device")
        fp = inv_freq.data_ptr()
    _kv_run("estream_kv_append", index, (
        cache._ref, elem, T, k.data_ptr(), k0, k1, v.data_ptr(), v0, v1, _kv_ints(positions, T, "positions", cache),
        None if rows is None else _kv_ints(rows, T, "rows", cache), tp, B, M, table_row, qp, q0, q1, Hq, op, o0, o1,
        fp, rot, 1 if interleaved else 0, _stream(None, cache.device)))
    return q_out


def kv_attend(cache: PagedKV, q: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, scale: float | None = None,
              window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of one new token per row, q [B, Hq, dim], over the first lens [B]
    int32 positions (the last `window` of them, if given) of the sequence whose
    pages are table [B, M] int32: [B, Hq, dim], and the logarithms of the sums of
    exponentials into lse [B, Hq] fp32. scale: 1 / sqrt(dim) unless given. Rows
    that share a sequence (the tokens of a prompt) may share a table row
    (table.expand). workspace: uint8, cache.attend_workspace_bytes(B, Hq, M,
    window) of them, for this call alone until it ends (allocated when not given)."""
    if stream is not None:
        with _current(stream, cache.device):
            return kv_attend(cache, q, table, lens, scale, window, out, lse, workspace)
    if _fast is not None and out is not None:
        st = _fast.kv_attend(cache._address, cache._index, q, table, lens, cache._scale if scale is None else scale, window,
                             out, lse, workspace)
        if st == 0:
            return out
        if st is not None:
            _check(st, "estream_kv_attend")
    elem, dt, dim, index = _kv_dtype(q, cache, "q"), q.dtype, cache.dim, cache._index
    if q.dim() != 3 or q.shape[2] != dim or q.shape[1] < 1 or q.shape[1] % cache.heads:
        raise ValueError(f"q must be [B, Hq, {dim}] with Hq a multiple of {cache.heads}")
    shape = B, Hq, _ = q.shape
    q0, q1, q2 = q.stride()
    if q2 != 1 or q.get_device() != index:
        raise _kv_bad(q, B, None, cache, "q", dt)
    tp, rows, M, table_row = _kv_table(table, cache)
    if rows != B:
        raise ValueError("table must have a row for each row of q")
    if not 0 <= window < 1 << 31:
        raise ValueError("window must be between 0 and 2^31 - 1")
    if out is None:
        out = torch.empty(shape, dtype=dt, device=cache.device)
    o0, o1, o2 = out.stride() if out.dim() == 3 else (0, 0, 0)
    if o2 != 1 or out.dtype is not dt or out.shape != shape or out.get_device() != index \
            or (B > 1 and o0 < dim) or (Hq > 1 and o1 < dim):
        raise _kv_bad(out, B, Hq, cache, "out", dt)
    ep = wp = None
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (B, Hq) or lse.get_device() != index or not lse.is_contiguous():
            raise ValueError(f"lse must be [{B}, {Hq}] fp32, contiguous, on the cache's device")
        ep = lse.data_ptr()
    n = cache.attend_workspace_bytes(B, Hq, M, window)
    if workspace is not None:
        if workspace.dtype is not torch.uint8 or workspace.numel() < n or workspace.get_device() != index \
                or not workspace.is_contiguous():
            raise ValueError(f"workspace must hold {n} bytes (uint8, contiguous) on the cache's device")
        wp = workspace.data_ptr()
    elif n:
        workspace = torch.empty(n, dtype=torch.uint8, device=cache.device)
        wp = workspace.data_ptr()
    _kv_run("estream_kv_attend", index, (
        cache._ref, elem, B, Hq, q.data_ptr(), q0, q1, tp, M, table_row, _kv_ints(lens, B, "lens", cache),
        cache._scale if scale is None else scale, window, out.data_ptr(), o0, o1, ep, wp, n, _stream(None, cache.device)))
    return out


# ---------------------------------------------------------------------------
# sampling
# ---------------------------------------------------------------------------

def _choice(x, B: int, dtype, name: str, device):
    """A choice of all rows, or a tensor with one for each: the number and the pointer."""
    if not isinstance(x, torch.Tensor):
        return x, None
    if x.dtype is not dtype or x.dim() != 1 or x.shape[0] != B or x.device != device or not x.is_contiguous():
        raise ValueError(f"{name} must be a number or [{B}] {dtype}, contiguous, on the logits' device")
    return 0, x.data_ptr()


def sample_tokens(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
                  out: torch.Tensor | None = None, prob: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The next token of each row of logits [B, V] (bf16, fp16 or fp32), [B] int32, from
    the random numbers u [B] fp32 in [0, 1): temperature, then the top_k largest (0:
    all), then of those the likeliest with top_p of the weight, then those with at
    least min_p of the largest's probability (rows may be one expanded row); the token is the first in the vocabulary's
    order whose cumulative probability exceeds u, and its probability goes to
    prob [B] fp32. Temperature 0 takes the largest logit. Each choice is a number or a
    tensor [B] (fp32; top_k int32). A row without a finite largest logit gives -1."""
    if stream is not None and logits.is_cuda:
        with _current(stream, logits.device):
            return sample_tokens(logits, u, temperature, top_k, top_p, min_p, out, prob)
    if _fast is not None and out is not None:
        st = _fast.sample(logits.get_device(), logits, u, temperature, top_k, top_p, min_p, out, prob)
        if st == 0:
            return out
        if st is not None:
            _check(st, "estream_sample_tokens")
    elem = _MX4_ELEM.get(logits.dtype)
    if elem is None or not logits.is_cuda:
        raise ValueError("logits must be a bf16, fp16 or fp32 CUDA tensor")
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be 2-d with contiguous rows")
    B, V = logits.shape
    ld, dev = logits.stride(0), logits.device
    if not 1 <= V <= SAMPLE_MAX_V:
        raise ValueError(f"a vocabulary must have 1 to {SAMPLE_MAX_V} tokens")
    if B > 1 << 30:
        raise ValueError("at most 2^30 rows a call")
    if not isinstance(top_k, torch.Tensor) and not -(1 << 31) <= top_k < 1 << 31:
        raise ValueError("top_k must fit in 32 bits")
    _, up = _choice(u, B, torch.float32, "u", dev)
    if up is None:
        raise ValueError("u must be a tensor with a random number for each row")
    choices = (*_choice(temperature, B, torch.float32, "temperature", dev), *_choice(top_k, B, torch.int32, "top_k", dev),
               *_choice(top_p, B, torch.float32, "top_p", dev), *_choice(min_p, B, torch.float32, "min_p", dev))
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=dev)
    elif out.dtype is not torch.int32 or tuple(out.shape) != (B,) or out.device != dev or not out.is_contiguous():
        raise ValueError(f"out must be [{B}] int32, contiguous, on the logits' device")
    pp = None if prob is None else _choice(prob, B, torch.float32, "prob", dev)[1]
    with _on(logits):
        st = lib().estream_sample_tokens(logits.data_ptr(), elem, ld, B, V, up, *choices, out.data_ptr(), pp,
                                         _stream(None, dev))
    if st:
        _check(st, "estream_sample_tokens")
    return out


def set_timing(ctx, on: bool) -> None:
    _check(lib().estream_set_timing(ctx, int(bool(on))), "estream_set_timing")


def reset_stats(ctx) -> None:
    _check(lib().estream_reset_stats(ctx), "estream_reset_stats")


def last_stats(ctx) -> dict:
    s = Stats()
    _check(lib().estream_last_stats(ctx, ctypes.byref(s)), "estream_last_stats")
    return {name: getattr(s, name) for name, _ in Stats._fields_}


def get_device_error(ctx) -> int:
    return lib().estream_get_device_error(ctx)


def poison_workspace(ctx, stream=None) -> None:
    """estream_poison_workspace (test aid): NaN / past-target fill of the
    context's per-call buffers on the stream, before a layer call."""
    _check(lib().estream_poison_workspace(ctx, _stream(stream)), "estream_poison_workspace")


def residency_trace(ctx, cap: int = 4096):
    buf = (ctypes.c_int32 * (4 * cap))()
    n = ctypes.c_int()
    _check(lib().estream_residency_trace(ctx, buf, cap, ctypes.byref(n)), "estream_residency_trace")
    m = min(n.value, cap)
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(m)]


def pipeline_trace(ctx, cap: int = 4096):
    """Per-group (a, d, s, f) times in ms of the last timed paged call, and
    the time routing finished."""
    import numpy as np
    buf = np.zeros((cap, 4), dtype=np.float64)
    n = ctypes.c_int()
    tne = ctypes.c_double()
    _check(lib().estream_pipeline_trace(ctx, buf.ctypes.data_as(ctypes.c_void_p), cap,
                                        ctypes.byref(n), ctypes.byref(tne)), "estream_pipeline_trace")
    return buf[:min(n.value, cap)].copy(), tne.value


def maxplus_pipeline(L, X, q: int, b: int, T_ne: float = 0.0):
    """Eq. 5: returns (T_pipe, adsf[K][4])."""
    import numpy as np
    L = np.ascontiguousarray(L, dtype=np.float64)
    X = np.ascontiguousarray(X, dtype=np.float64)
    K = len(L)
    out = np.zeros((max(K, 1), 4), dtype=np.float64)
    t = lib().estream_maxplus_pipeline(L.ctypes.data_as(ctypes.c_void_p), X.ctypes.data_as(ctypes.c_void_p),
                                       K, q, b, T_ne, out.ctypes.data_as(ctypes.c_void_p))
    return t, out[:K]


def bank_bound(g, M_max, M_other, W_e, N_e) -> int:
    return lib().estream_bank_bound(g, M_max, M_other, W_e, N_e)


def autoconfig(profiles: dict, T_ne: float, Q0: int, M_max: float, W_e: float, N_e: int,
               M_other: dict | None = None):
    """Eqs. 9-10 over {g: (L[], X[])}. Returns (G*, B*, T_pipe*)."""
    import numpy as np
    gs = list(profiles)
    Ls = [np.ascontiguousarray(profiles[g][0], dtype=np.float64) for g in gs]
    Xs = [np.ascontiguousarray(profiles[g][1], dtype=np.float64) for g in gs]
    g_arr = (ctypes.c_int * len(gs))(*gs)
    k_arr = (ctypes.c_int * len(gs))(*[len(x) for x in Ls])
    L_arr = (ctypes.c_void_p * len(gs))(*[x.ctypes.data for x in Ls])
    X_arr = (ctypes.c_void_p * len(gs))(*[x.ctypes.data for x in Xs])
    mo = None
    if M_other is not None:
        mo = (ctypes.c_double * len(gs))(*[float(M_other[g]) for g in gs])
    G, B, T = ctypes.c_int(), ctypes.c_int(), ctypes.c_double()
    _check(lib().estream_autoconfig(len(gs), g_arr, k_arr, L_arr, X_arr, T_ne, Q0, M_max, mo, W_e,
                                    N_e, ctypes.byref(G), ctypes.byref(B), ctypes.byref(T)),
           "estream_autoconfig")
    return G.value, B.value, T.value


def inject_expert_timeout(ctx) -> None:
    _check(lib().estream_inject_expert_timeout(ctx), "estream_inject_expert_timeout")


def inject_route_timeout(ctx) -> None:
    _check(lib().estream_inject_route_timeout(ctx), "estream_inject_route_timeout")


def inject_late_arrival(ctx, barrier: int) -> None:
    _check(lib().estream_inject_late_arrival(ctx, barrier), "estream_inject_late_arrival")


def inject_pager_fault(ctx, layer: int, group: int) -> None:
    _check(lib().estream_inject_pager_fault(ctx, layer, group), "estream_inject_pager_fault")


def unbind(ctx) -> None:
    if ctx:
        lib().estream_unbind(ctx)
