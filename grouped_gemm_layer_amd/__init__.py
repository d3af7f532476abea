"""Python binding of the MoE expert-layer HIP library (libmoe_gfx950.so).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  PyTorch provides device memory and the current stream.  The
binding raises if the built library is missing; there is no fallback.

Names follow the C ABI in include/moe.h:
    workspace_size(dims) -> (route_ws, saved, fwd_ws, bwd_ws)
    route(dims, logits, routing, ws)
    route_noalloc(dims, logits, routing)
    weight_codes_size(dims); quantize_weights(dims, w13, w2, codes)
    forward_cached(dims, x, w13, w2, codes, routing, y, saved, ws)
    backward_cached(dims, dy, x, codes, routing, saved, dx, dw13, dw2, dgate, dlogits, ws)
    forward(dims, x, w13, w2, routing, y, saved, ws)
    backward(dims, dy, x, w13, w2, routing, saved, dx, dw13, dw2, dgate, dlogits, ws)
    mxfp8_quantize(src, along, codes, scales)
    mxfp8_quantize_grouped(src, offsets, capacity, pad_off, codes, scales)
    sort_workspace_size(T, k, E); sort_tokens(routing, ws)
    permute(x, routing, xp, weights); permute_backward(dxp, routing, dx, weights, x, dweights)
    unpermute(rows, routing, y, weights); unpermute_backward(dy, routing, drows, weights, rows, dweights)
    mxfp4_quantize(src, codes, scales, along, swiglu); mxfp4_dequantize(codes, scales, out)
    mxfp4_product(a_codes, a_scales, b_codes, b_scales, c, k, a_format, offsets, row_map, row_div)
    grad_workspace_size(count); grad_norm(tensors, sumsq, ws); grad_clip(tensors, sumsq, max_norm, norm, out)
plus GradientList, which owns the buffers of a list of gradients, and
allocation helpers (alloc_routing, alloc_workspace) and MoeLayer, a
small holder that owns the buffers of one shape.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "MODE_FP32", "MODE_BF16", "MODE_MXFP8", "MODE_FP8_BWD", "Dims", "RoutingBuffers",
    "MoeError", "lib_path", "load_library", "workspace_size", "route", "forward", "backward",
    "alloc_routing", "alloc_workspace", "status_str", "MoeLayer", "num_kernels", "mxfp8_quantize",
    "mxfp8_quantize_grouped", "mxfp8_grouped_capacity", "route_noalloc", "weight_codes_size", "quantize_weights",
    "forward_cached", "backward_cached", "sort_workspace_size", "sort_tokens", "permute", "permute_backward",
    "unpermute", "unpermute_backward", "mxfp4_quantize", "mxfp4_dequantize", "mxfp4_product", "grad_workspace_size",
    "grad_norm", "grad_clip", "GradientList",
]

MODE_FP32, MODE_BF16, MODE_MXFP8, MODE_FP8_BWD = 0, 1, 2, 3
MODE_BY_NAME = {"fp32": MODE_FP32, "bf16": MODE_BF16, "mxfp8": MODE_MXFP8, "fp8_bwd": MODE_FP8_BWD}

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_NAME = "libmoe_gfx950.so"

SYMBOLS = ("moe_workspace_size", "moe_route", "moe_forward", "moe_backward", "moe_status_str")


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("mode", ctypes.c_int32)]

    @classmethod
    def of(cls, T, H, I, E, k, mode):
        if isinstance(mode, str):
            mode = MODE_BY_NAME[mode]
        return cls(T, H, I, E, k, mode)


class _CRouting(ctypes.Structure):
    _fields_ = [("topk_idx", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("sorted_to_flat", ctypes.c_void_p),
                ("flat_to_sorted", ctypes.c_void_p)]


class _CTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64), ("type", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)} (status {status})")


_lib = None


def lib_path() -> str:
    return os.path.join(_PKG, LIB_NAME)


def load_library():
    """Load the built HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    # torch's HIP runtime (same soname) must be the one in the process, so that
    # torch streams and device pointers are valid in the library's calls
    import torch  # noqa: F401
    path = lib_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with python -m grouped_gemm_layer_amd.build_lib")
    lib = ctypes.CDLL(path)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.moe_workspace_size.argtypes = [ctypes.POINTER(Dims)] + [ctypes.POINTER(sz)] * 4
    lib.moe_route.argtypes = [ctypes.POINTER(Dims), vp, ctypes.POINTER(_CRouting), vp, sz, vp]
    lib.moe_forward.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, ctypes.POINTER(_CRouting), vp, vp, vp, sz, vp]
    lib.moe_backward.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, vp, ctypes.POINTER(_CRouting), vp, vp,
                                 vp, vp, vp, vp, vp, sz, vp]
    for f in ("moe_workspace_size", "moe_route", "moe_forward", "moe_backward"):
        getattr(lib, f).restype = ctypes.c_int
    lib.moe_weight_codes_size.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(sz)]
    lib.moe_weight_codes_size.restype = ctypes.c_int
    lib.moe_quantize_weights.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, sz, vp]
    lib.moe_quantize_weights.restype = ctypes.c_int
    lib.moe_forward_cached.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, vp, ctypes.POINTER(_CRouting), vp, vp, vp,
                                       sz, vp]
    lib.moe_forward_cached.restype = ctypes.c_int
    lib.moe_backward_cached.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, ctypes.POINTER(_CRouting), vp, vp, vp, vp,
                                        vp, vp, vp, sz, vp]
    lib.moe_backward_cached.restype = ctypes.c_int
    lib.moe_route_noalloc.argtypes = [ctypes.POINTER(Dims), vp, ctypes.POINTER(_CRouting), vp]
    lib.moe_route_noalloc.restype = ctypes.c_int
    lib.moe_route_project.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, ctypes.POINTER(_CRouting), vp, sz, vp]
    lib.moe_route_project.restype = ctypes.c_int
    lib.moe_router_backward.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(_CRouting), vp, vp, vp, vp, vp, vp]
    lib.moe_router_backward.restype = ctypes.c_int
    lib.moe_backward_accumulate.argtypes = lib.moe_backward.argtypes
    lib.moe_backward_accumulate.restype = ctypes.c_int
    lib.moe_forward_recompute.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, ctypes.POINTER(_CRouting), vp, vp, sz,
                                          vp]
    lib.moe_forward_recompute.restype = ctypes.c_int
    lib.moe_forward_timed.argtypes = lib.moe_forward.argtypes + [vp, ctypes.c_int]
    lib.moe_backward_timed.argtypes = lib.moe_backward.argtypes + [vp, ctypes.c_int]
    lib.moe_forward_timed.restype = ctypes.c_int
    lib.moe_backward_timed.restype = ctypes.c_int
    lib.moe_num_kernels.argtypes = [ctypes.POINTER(Dims), ctypes.c_int]
    lib.moe_num_kernels.restype = ctypes.c_int
    i32 = ctypes.c_int32
    lib.moe_mxfp8_quantize.argtypes = [vp, i32, i32, i32, vp, vp, vp]
    lib.moe_mxfp8_quantize.restype = ctypes.c_int
    lib.moe_mxfp8_quantize_grouped.argtypes = [vp, i32, i32, vp, i32, i32, vp, vp, vp, vp]
    lib.moe_mxfp8_quantize_grouped.restype = ctypes.c_int
    lib.moe_mxfp8_grouped_capacity.argtypes = [i32, i32]
    lib.moe_mxfp8_grouped_capacity.restype = sz
    lib.moe_status_str.argtypes = [ctypes.c_int]
    lib.moe_status_str.restype = ctypes.c_char_p
    i64, f32, psz = ctypes.c_int64, ctypes.c_float, ctypes.POINTER(sz)
    for f, args in (
            ("moe_sort_workspace_size", [i32, i32, i32, psz]),
            ("moe_sort_tokens", [vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
            ("moe_permute", [vp, i64, i32, i32, i32, i32, vp, vp, vp, i64, i32, vp]),
            ("moe_permute_backward", [vp, i64, i32, i32, i32, i32, i32, vp, vp, vp, i64, vp, i64, vp, vp]),
            ("moe_unpermute", [vp, i64, i32, i32, i32, i32, i32, vp, vp, vp, i64, vp]),
            ("moe_unpermute_backward", [vp, i64, i32, i32, i32, i32, vp, vp, vp, i64, vp, i64, i32, vp, vp]),
            ("moe_mxfp4_quantize", [vp, i64, i32, i32, i32, i32, i32, i32, vp, vp, vp]),
            ("moe_mxfp4_dequantize", [vp, vp, i32, i32, vp, i64, i32, vp]),
            ("moe_mxfp4_product", [vp, vp, i32, i32, vp, vp, i32, i32, i32, vp, vp, i32, vp, i64, i32, i32, vp]),
            ("moe_grad_workspace_size", [i32, psz]),
            ("moe_grad_norm", [vp, i32, vp, vp, sz, vp]),
            ("moe_grad_clip", [vp, i32, vp, f32, vp, vp])):
        getattr(lib, f).argtypes = args
        getattr(lib, f).restype = ctypes.c_int
    lib.moe_wgrad_chunk_rows.argtypes = []
    lib.moe_wgrad_chunk_rows.restype = ctypes.c_int32
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load_library().moe_status_str(status).decode()


def wgrad_chunk_rows() -> int:
    """Rows per weight-gradient chunk (experts with more rows are split)."""
    return int(load_library().moe_wgrad_chunk_rows())


def _check(st: int, what: str):
    if st != 0:
        raise MoeError(st, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def workspace_size(dims: Dims):
    lib = load_library()
    out = [ctypes.c_size_t(0) for _ in range(4)]
    _check(lib.moe_workspace_size(ctypes.byref(dims), *[ctypes.byref(o) for o in out]), "moe_workspace_size")
    return tuple(o.value for o in out)


class RoutingBuffers:
    """Device tensors of the routing state (torch int32/float32)."""

    def __init__(self, topk_idx, gate, counts, offsets, sorted_to_flat, flat_to_sorted):
        self.topk_idx, self.gate, self.counts = topk_idx, gate, counts
        self.offsets, self.sorted_to_flat, self.flat_to_sorted = offsets, sorted_to_flat, flat_to_sorted

    def c(self) -> _CRouting:
        return _CRouting(self.topk_idx.data_ptr(), self.gate.data_ptr(), self.counts.data_ptr(),
                         self.offsets.data_ptr(), self.sorted_to_flat.data_ptr(), self.flat_to_sorted.data_ptr())


def alloc_routing(dims: Dims, device="cuda") -> RoutingBuffers:
    import torch
    T, k, E = dims.T, dims.k, dims.E
    i32 = dict(dtype=torch.int32, device=device)
    return RoutingBuffers(torch.empty((T, k), **i32), torch.empty((T, k), dtype=torch.float32, device=device),
                          torch.empty((E,), **i32), torch.empty((E + 1,), **i32),
                          torch.empty((T * k,), **i32), torch.empty((T * k,), **i32))


def alloc_workspace(nbytes: int, device="cuda"):
    import torch
    return torch.empty((max(int(nbytes), 1),), dtype=torch.uint8, device=device)


def route(dims: Dims, logits, routing: RoutingBuffers, ws, stream=None):
    lib = load_library()
    r = routing.c()
    _check(lib.moe_route(ctypes.byref(dims), _ptr(logits), ctypes.byref(r), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_route")


def route_noalloc(dims: Dims, logits, routing: RoutingBuffers, stream=None):
    """moe_route_noalloc: routing without a workspace (the library's static
    per-device scratch; calls that overlap on one GPU race)."""
    lib = load_library()
    r = routing.c()
    _check(lib.moe_route_noalloc(ctypes.byref(dims), _ptr(logits), ctypes.byref(r), _stream(stream)),
           "moe_route_noalloc")


def route_project(dims: Dims, x, w_router, logits, routing: RoutingBuffers, ws, stream=None):
    """logits = x w_router^T (written to `logits`), then route (moe_route_project)."""
    lib = load_library()
    r = routing.c()
    _check(lib.moe_route_project(ctypes.byref(dims), _ptr(x), _ptr(w_router), _ptr(logits), ctypes.byref(r),
                                 _ptr(ws), ws.numel(), _stream(stream)), "moe_route_project")


def router_backward(dims: Dims, routing: RoutingBuffers, dlogits, x, w_router, dx, dw_router, stream=None):
    """dx += dlogits w_router; dw_router = dlogits^T x (moe_router_backward)."""
    lib = load_library()
    r = routing.c()
    _check(lib.moe_router_backward(ctypes.byref(dims), ctypes.byref(r), _ptr(dlogits), _ptr(x), _ptr(w_router),
                                   _ptr(dx), _ptr(dw_router), _stream(stream)), "moe_router_backward")


def forward(dims: Dims, x, w13, w2, routing: RoutingBuffers, y, saved, ws, stream=None, events=None):
    """events: optional ctypes array of hipEvent_t (moe_forward_timed)."""
    lib = load_library()
    r = routing.c()
    args = [ctypes.byref(dims), _ptr(x), _ptr(w13), _ptr(w2), ctypes.byref(r), _ptr(y), _ptr(saved), _ptr(ws),
            ws.numel(), _stream(stream)]
    if events is None:
        _check(lib.moe_forward(*args), "moe_forward")
    else:
        _check(lib.moe_forward_timed(*args, events, len(events)), "moe_forward_timed")


def forward_recompute(dims: Dims, x, w13, w2, routing: RoutingBuffers, saved, ws, stream=None):
    """moe_forward_recompute: restore `saved` for the backward without computing y."""
    lib = load_library()
    r = routing.c()
    _check(lib.moe_forward_recompute(ctypes.byref(dims), _ptr(x), _ptr(w13), _ptr(w2), ctypes.byref(r),
                                     _ptr(saved), _ptr(ws), ws.numel(), _stream(stream)), "moe_forward_recompute")


def backward(dims: Dims, dy, x, w13, w2, routing: RoutingBuffers, saved, dx, dw13, dw2, dgate, dlogits, ws,
             stream=None, events=None, accumulate=False):
    """events: optional ctypes array of hipEvent_t (moe_backward_timed).
    accumulate: add the weight gradients to dw13 / dw2 (moe_backward_accumulate)."""
    lib = load_library()
    r = routing.c()
    args = [ctypes.byref(dims), _ptr(dy), _ptr(x), _ptr(w13), _ptr(w2), ctypes.byref(r), _ptr(saved), _ptr(dx),
            _ptr(dw13), _ptr(dw2), _ptr(dgate), _ptr(dlogits), _ptr(ws), ws.numel(), _stream(stream)]
    if accumulate:
        if events is not None:
            raise ValueError("timed accumulate-into is not provided")
        _check(lib.moe_backward_accumulate(*args), "moe_backward_accumulate")
    elif events is None:
        _check(lib.moe_backward(*args), "moe_backward")
    else:
        _check(lib.moe_backward_timed(*args, events, len(events)), "moe_backward_timed")


def weight_codes_size(dims: Dims) -> int:
    """Bytes of the MXFP8 weight copies of an fp8 mode (moe_weight_codes_size)."""
    out = ctypes.c_size_t(0)
    _check(load_library().moe_weight_codes_size(ctypes.byref(dims), ctypes.byref(out)), "moe_weight_codes_size")
    return out.value


def quantize_weights(dims: Dims, w13, w2, codes, stream=None):
    """MXFP8 copies of the weights into `codes` (uint8 tensor, moe_quantize_weights)."""
    _check(load_library().moe_quantize_weights(ctypes.byref(dims), _ptr(w13), _ptr(w2), _ptr(codes), codes.numel(),
                                               _stream(stream)), "moe_quantize_weights")


def forward_cached(dims: Dims, x, w13, w2, codes, routing: RoutingBuffers, y, saved, ws, stream=None):
    """moe_forward_cached: the MXFP8 GEMMs take their weights from `codes`."""
    r = routing.c()
    _check(load_library().moe_forward_cached(ctypes.byref(dims), _ptr(x), _ptr(w13), _ptr(w2), _ptr(codes),
                                             ctypes.byref(r), _ptr(y), _ptr(saved), _ptr(ws), ws.numel(),
                                             _stream(stream)), "moe_forward_cached")


def backward_cached(dims: Dims, dy, x, codes, routing: RoutingBuffers, saved, dx, dw13, dw2, dgate, dlogits, ws,
                    stream=None):
    """moe_backward_cached: the MXFP8 GEMMs take their weights from `codes`."""
    r = routing.c()
    _check(load_library().moe_backward_cached(ctypes.byref(dims), _ptr(dy), _ptr(x), _ptr(codes), ctypes.byref(r),
                                              _ptr(saved), _ptr(dx), _ptr(dw13), _ptr(dw2), _ptr(dgate),
                                              _ptr(dlogits), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_backward_cached")


def num_kernels(dims: Dims, which: str) -> int:
    n = load_library().moe_num_kernels(ctypes.byref(dims), {"route": 0, "forward": 1, "backward": 2}[which])
    if n < 0:
        raise MoeError(2, "moe_num_kernels")
    return n


def mxfp8_quantize(src, along: int, codes, scales, stream=None):
    """src: bf16 [rows, cols]; along=1 -> codes [rows, cols], scales [rows, cols/32];
    along=0 -> codes [cols, rows], scales [cols, rows/32] (uint8 tensors)."""
    rows, cols = src.shape
    _check(load_library().moe_mxfp8_quantize(_ptr(src), rows, cols, along, _ptr(codes), _ptr(scales),
                                             _stream(stream)), "moe_mxfp8_quantize")


def mxfp8_grouped_capacity(rows: int, E: int) -> int:
    return int(load_library().moe_mxfp8_grouped_capacity(rows, E))


def mxfp8_quantize_grouped(src, offsets, capacity: int, pad_off, codes, scales, stream=None):
    """src: bf16 [rows, cols] in expert order (offsets int32 [E+1]); codes
    [cols, capacity], scales [cols, capacity/32] (uint8), pad_off int32 [E+1]."""
    rows, cols = src.shape
    E = offsets.numel() - 1
    _check(load_library().moe_mxfp8_quantize_grouped(_ptr(src), rows, cols, _ptr(offsets), E, capacity,
                                                     _ptr(pad_off), _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_mxfp8_quantize_grouped")


# ---------------------------------------------------------------------------
# Operators beside the layer
# ---------------------------------------------------------------------------
def _type_of(t) -> int:
    """The moe_type of a tensor's elements."""
    import torch
    if t.dtype is torch.bfloat16:
        return 1
    if t.dtype is torch.float32:
        return 0
    raise ValueError(f"float32 or bfloat16 values expected, got {t.dtype}")


def _matrix(t, name):
    """(rows, cols, row pitch) of a 2-D operand whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{name}: a matrix expected, got shape {tuple(t.shape)}")
    rows, cols = t.shape
    ld = t.stride(0) if rows > 1 else cols
    if (cols > 1 and t.stride(1) != 1) or ld < cols:
        raise ValueError(f"{name}: rows must be contiguous and must not overlap (strides {t.stride()})")
    return rows, cols, ld


def _plain(t, name, dtype, numel=None):
    """Checks a contiguous tensor of `dtype` (and of `numel` elements)."""
    if t.dtype is not dtype or not t.is_contiguous() or (numel is not None and t.numel() != numel):
        raise ValueError(f"{name}: a contiguous {dtype} tensor{'' if numel is None else f' of {numel} elements'} "
                         f"expected, got {t.dtype} {tuple(t.shape)}")


def _enqueue(what, stream, tensors, *args):
    """Calls the library's function `what` on the tensors' device: on `stream`,
    or on that device's current one.  None of `tensors` may live elsewhere.
    (Plain device numbers and the raw stream: the torch.device and Stream
    objects cost 2 us more, a third of a small call.)"""
    import torch
    lib = _lib or load_library()
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if d < 0:
                    raise ValueError(f"moe_{what}: device tensors expected, got one on {t.device}")
                if dev is not None:
                    raise ValueError(f"moe_{what}: tensors on devices {dev} and {d}")
                dev = d
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    else:
        if stream.device.index != dev:
            raise ValueError(f"moe_{what}: a stream of {stream.device} for tensors on device {dev}")
        raw = stream.cuda_stream
    f = getattr(lib, "moe_" + what)
    if dev == torch.cuda.current_device():
        st = f(*args, raw)
    else:   # kernels launch on the current device
        with torch.cuda.device(dev):
            st = f(*args, raw)
    if st != 0:
        raise MoeError(st, "moe_" + what)


def _addr(t):
    return None if t is None else t.data_ptr()


def sort_workspace_size(T: int, k: int, E: int) -> int:
    """Bytes of sort_tokens' workspace (moe_sort_workspace_size)."""
    out = ctypes.c_size_t(0)
    _check(load_library().moe_sort_workspace_size(T, k, E, ctypes.byref(out)), "moe_sort_workspace_size")
    return out.value


def sort_tokens(routing: RoutingBuffers, ws, stream=None):
    """Writes routing's counts, offsets and maps from its topk_idx [T, k]
    (moe_sort_tokens); an index outside [0, E) marks a slot without an expert."""
    import torch
    idx = routing.topk_idx
    if idx.dim() != 2:
        raise ValueError(f"topk_idx: [T, k] expected, got shape {tuple(idx.shape)}")
    (T, k), E = idx.shape, routing.counts.numel()
    _plain(idx, "topk_idx", torch.int32)
    _plain(routing.counts, "counts", torch.int32)
    _plain(routing.offsets, "offsets", torch.int32, E + 1)
    _plain(routing.sorted_to_flat, "sorted_to_flat", torch.int32, T * k)
    _plain(routing.flat_to_sorted, "flat_to_sorted", torch.int32, T * k)
    _plain(ws, "ws", torch.uint8)
    _enqueue("sort_tokens", stream,
             (idx, routing.counts, routing.offsets, routing.sorted_to_flat, routing.flat_to_sorted, ws),
             idx.data_ptr(), T, k, E, routing.counts.data_ptr(), routing.offsets.data_ptr(),
             routing.sorted_to_flat.data_ptr(), routing.flat_to_sorted.data_ptr(), ws.data_ptr(), ws.numel())


def _rows_call(tokens, rows, routing, weights, dweights, other, other_like):
    """Shared checks of the four row calls: (T, H, k, type, row pitches of
    tokens, rows and other)."""
    import torch
    T, H, ldt = _matrix(tokens, "token rows")
    n, H2, ldr = _matrix(rows, "expert rows")
    typ = _type_of(tokens)
    f2s = routing.flat_to_sorted
    k = routing.topk_idx.shape[1] if T == 0 else f2s.numel() // T
    _plain(f2s, "flat_to_sorted", torch.int32, T * k)
    if H != H2 or rows.dtype is not tokens.dtype:
        raise ValueError(f"token rows {tuple(tokens.shape)} {tokens.dtype} and expert rows {tuple(rows.shape)} "
                         f"{rows.dtype} do not match")
    if weights is not None:
        _plain(weights, "weights", torch.float32, T * k)
    ldo = 0
    if dweights is not None:
        _plain(dweights, "dweights", torch.float32, T * k)
        if other is None or other.shape != other_like.shape or other.dtype is not tokens.dtype:
            raise ValueError("dweights needs the forward's rows, of their shape and type")
        ldo = _matrix(other, "forward rows")[2]
    return T, H, n, k, typ, ldt, ldr, ldo


def permute(x, routing: RoutingBuffers, xp, weights=None, stream=None):
    """xp[row of slot (t, j)] = weights[t, j] x[t] (moe_permute); rows no slot names stay as they are."""
    T, H, n, k, typ, ldx, ldp, _ = _rows_call(x, xp, routing, weights, None, None, None)
    f2s = routing.flat_to_sorted
    _enqueue("permute", stream, (x, xp, f2s, weights), x.data_ptr(), ldx, T, H, k, typ, f2s.data_ptr(),
             _addr(weights), xp.data_ptr(), ldp, n)


def permute_backward(dxp, routing: RoutingBuffers, dx, weights=None, x=None, dweights=None, stream=None):
    """dx[t] = sum_j weights[t, j] dxp[row]; dweights[t, j] = <x[t], dxp[row]> (moe_permute_backward)."""
    T, H, n, k, typ, lddx, ldp, ldx = _rows_call(dx, dxp, routing, weights, dweights, x, dx)
    f2s = routing.flat_to_sorted
    other = x if dweights is not None else None
    _enqueue("permute_backward", stream, (dxp, dx, f2s, weights, other, dweights), dxp.data_ptr(), ldp, n, T, H, k, typ,
             f2s.data_ptr(), _addr(weights), _addr(other), ldx, dx.data_ptr(), lddx, _addr(dweights))


def unpermute(rows, routing: RoutingBuffers, y, weights=None, stream=None):
    """y[t] = sum_j weights[t, j] rows[row of slot (t, j)] (moe_unpermute)."""
    T, H, n, k, typ, ldy, ldo, _ = _rows_call(y, rows, routing, weights, None, None, None)
    f2s = routing.flat_to_sorted
    _enqueue("unpermute", stream, (rows, y, f2s, weights), rows.data_ptr(), ldo, n, T, H, k, typ, f2s.data_ptr(),
             _addr(weights), y.data_ptr(), ldy)


def unpermute_backward(dy, routing: RoutingBuffers, drows, weights=None, rows=None, dweights=None, stream=None):
    """drows[row] = weights[t, j] dy[t]; dweights[t, j] = <dy[t], rows[row]> (moe_unpermute_backward)."""
    T, H, n, k, typ, lddy, lddr, ldo = _rows_call(dy, drows, routing, weights, dweights, rows, drows)
    f2s = routing.flat_to_sorted
    other = rows if dweights is not None else None
    _enqueue("unpermute_backward", stream, (dy, drows, f2s, weights, other, dweights), dy.data_ptr(), lddy, T, H, k, typ,
             f2s.data_ptr(), _addr(weights), _addr(other), ldo, drows.data_ptr(), lddr, n, _addr(dweights))


def mxfp4_quantize(src, codes, scales, along: int = 1, swiglu: bool = False, stream=None):
    """MXFP4 codes and scales (uint8) of src [rows, cols] or [batch, rows, cols]
    (moe_mxfp4_quantize): along=1 by rows, codes [.., rows, KB*16] and scales
    [.., rows, KB]; along=0 transposed, [.., cols, KB*16] and [.., cols, KB].
    swiglu: src rows are [g1 | g3] and SiLU(g1) * g3 is quantised."""
    import torch
    if src.dim() not in (2, 3):
        raise ValueError(f"src: [rows, cols] or [batch, rows, cols] expected, got shape {tuple(src.shape)}")
    batch = src.shape[0] if src.dim() == 3 else 1
    rows, width = src.shape[-2:]
    ld = src.stride(-2) if rows > 1 else (src.stride(0) if src.dim() == 3 and batch > 1 else width)
    if (width > 1 and src.stride(-1) != 1) or ld < width or (
            src.dim() == 3 and batch > 1 and rows > 0 and src.stride(0) != rows * ld):
        raise ValueError(f"src: contiguous rows at one pitch expected, got strides {src.stride()}")
    if swiglu and width % 2:
        raise ValueError(f"src: rows of [g1 | g3] expected, got {width} columns")
    cols = width // 2 if swiglu else width
    r, n = (rows, cols) if along else (cols, rows)
    kb = -(-n // 32)
    _plain(codes, "codes", torch.uint8, batch * r * kb * 16)
    _plain(scales, "scales", torch.uint8, batch * r * kb)
    _enqueue("mxfp4_quantize", stream, (src, codes, scales), src.data_ptr(), ld, batch, rows, cols, _type_of(src), along,
             int(swiglu), codes.data_ptr(), scales.data_ptr())


def mxfp4_dequantize(codes, scales, out, stream=None):
    """The values of MXFP4 codes and scales as out [.., cols] holds them (moe_mxfp4_dequantize)."""
    import torch
    m = out if out.dim() == 2 else out.view(-1, out.shape[-1]) if out.is_contiguous() else None
    if m is None:
        raise ValueError("out: a matrix or a contiguous tensor expected")
    rows, cols, ld = _matrix(m, "out")
    kb = -(-cols // 32)
    _plain(codes, "codes", torch.uint8, rows * kb * 16)
    _plain(scales, "scales", torch.uint8, rows * kb)
    _enqueue("mxfp4_dequantize", stream, (codes, scales, out), codes.data_ptr(), scales.data_ptr(), rows, cols,
             m.data_ptr(), ld, _type_of(out))


MX_FORMATS = {"mxfp4": 0, "mxfp8": 1}


def mxfp4_product(a_codes, a_scales, b_codes, b_scales, c, k: int, a_format: str = "mxfp4", offsets=None, row_map=None,
                  row_div: int = 1, stream=None):
    """c[r] = a[row_map[r] // row_div] b[e]^T for rows r of expert e
    (moe_mxfp4_product).  a: [a_rows, ..] in a_format, b: MXFP4 [E, N, ..] (or
    [N, ..] without offsets), rows of k values; c: [rows, N] float32 or
    bfloat16; offsets: int32 [E+1]; row_map: int32 [rows]."""
    import torch
    fmt = MX_FORMATS.get(a_format)
    if fmt is None:
        raise ValueError(f"a_format: one of {sorted(MX_FORMATS)} expected, got {a_format!r}")
    rows, N, ldc = _matrix(c, "c")
    kb = -(-k // 32)
    E = offsets.numel() - 1 if offsets is not None else 1
    a_rows = a_codes.shape[0]
    _plain(a_codes, "a_codes", torch.uint8, a_rows * (kb * 16 if fmt == 0 else k))
    _plain(a_scales, "a_scales", torch.uint8, a_rows * kb)
    _plain(b_codes, "b_codes", torch.uint8, E * N * kb * 16)
    _plain(b_scales, "b_scales", torch.uint8, E * N * kb)
    if offsets is not None:
        _plain(offsets, "offsets", torch.int32)
    if row_map is not None:
        _plain(row_map, "row_map", torch.int32, rows)
    elif a_rows < rows:
        raise ValueError(f"c has {rows} rows, a {a_rows}")
    _enqueue("mxfp4_product", stream, (a_codes, a_scales, b_codes, b_scales, c, offsets, row_map), a_codes.data_ptr(),
             a_scales.data_ptr(), a_rows, fmt, b_codes.data_ptr(), b_scales.data_ptr(), E, N, k, _addr(offsets),
             _addr(row_map), row_div, c.data_ptr(), ldc, rows, _type_of(c))


def _tensor_table(tensors, out):
    """The C array (moe_tensor) of a list of gradients and of their outputs: four
    64-bit words each, the type in the low half of the last."""
    import array
    for name, ts in (("gradient", tensors), ("output", out or ())):
        if not all([t.is_contiguous() for t in ts]):
            i = [t.is_contiguous() for t in ts].index(False)
            raise ValueError(f"{name} {i}: a contiguous tensor expected, got strides {ts[i].stride()}")
    n = [t.numel() for t in tensors]
    kinds = [t.dtype for t in tensors]
    code = {dt: _type_of(tensors[kinds.index(dt)]) for dt in set(kinds)}
    table = array.array("q", bytes(32 * max(len(tensors), 1)))
    if tensors:
        table[0::4] = array.array("q", [t.data_ptr() for t in tensors])
        table[2::4] = array.array("q", n)
        table[3::4] = array.array("q", [code[dt] for dt in kinds])
    if out is not None:
        if len(out) != len(tensors):
            raise ValueError(f"{len(tensors)} gradients and {len(out)} outputs")
        if [t.numel() for t in out] != n or [t.dtype for t in out] != kinds:
            raise ValueError("every output needs its gradient's size and type")
        if out:
            table[1::4] = array.array("q", [t.data_ptr() for t in out])
    return table


def grad_workspace_size(count: int) -> int:
    """Bytes of grad_norm's workspace for `count` tensors (moe_grad_workspace_size)."""
    out = ctypes.c_size_t(0)
    _check(load_library().moe_grad_workspace_size(count, ctypes.byref(out)), "moe_grad_workspace_size")
    return out.value


def _scalar(t, name, dtype):
    _plain(t, name, dtype, 1)


def grad_norm(tensors, sumsq, ws, stream=None):
    """sumsq (float64, one element) = sum of squares of all tensors (moe_grad_norm)."""
    import torch
    _scalar(sumsq, "sumsq", torch.float64)
    _plain(ws, "ws", torch.uint8)
    table = _tensor_table(tensors, None)
    _enqueue("grad_norm", stream, (sumsq, ws, *tensors), table.buffer_info()[0], len(tensors), sumsq.data_ptr(),
             ws.data_ptr(), ws.numel())


def grad_clip(tensors, sumsq, max_norm: float, norm=None, out=None, stream=None):
    """Scales the tensors by min(1, max_norm / sqrt(sumsq)), in place or into
    `out`; norm (float32, one element) = sqrt(sumsq) (moe_grad_clip)."""
    import torch
    _scalar(sumsq, "sumsq", torch.float64)
    if norm is not None:
        _scalar(norm, "norm", torch.float32)
    table = _tensor_table(tensors, out)
    _enqueue("grad_clip", stream, (sumsq, norm, *tensors, *(out or ())), table.buffer_info()[0], len(tensors),
             sumsq.data_ptr(), max_norm, _addr(norm))


class GradientList:
    """The gradients of a step (contiguous float32 or bfloat16 tensors of one
    device), with the buffers of their norm and the table the library reads.
    The tensors stay where they are while the list is used; out: where the
    clipped gradients go (default: in place)."""

    def __init__(self, tensors, out=None):
        import torch
        self.tensors = list(tensors)
        self.out = None if out is None else list(out)
        if not self.tensors:
            raise ValueError("at least one gradient expected")
        dev = self.tensors[0].device
        self._table = _tensor_table(self.tensors, self.out)
        at = {t.get_device() for t in (*self.tensors, *(self.out or ()))}
        if len(at) > 1 or min(at) < 0:
            raise ValueError(f"gradients and outputs on one GPU expected, got devices {sorted(at)}")
        self.sumsq = torch.empty(1, dtype=torch.float64, device=dev)
        self.norm = torch.empty((), dtype=torch.float32, device=dev)
        self.ws = alloc_workspace(grad_workspace_size(len(self.tensors)), dev)

    def sum_squares(self, stream=None):
        """sumsq (float64 [1]) of these tensors; ranks add theirs up before scale()."""
        _enqueue("grad_norm", stream, (self.sumsq,), self._table.buffer_info()[0], len(self.tensors),
                 self.sumsq.data_ptr(), self.ws.data_ptr(), self.ws.numel())
        return self.sumsq

    def scale(self, max_norm: float, stream=None):
        """Clips by the norm sqrt(sumsq); returns the norm (float32 tensor)."""
        _enqueue("grad_clip", stream, (self.sumsq,), self._table.buffer_info()[0], len(self.tensors),
                 self.sumsq.data_ptr(), max_norm, self.norm.data_ptr())
        return self.norm

    def clip(self, max_norm: float, stream=None):
        """Norm and clipping in one go; returns the norm (float32 tensor)."""
        self.sum_squares(stream)
        return self.scale(max_norm, stream)


class MoeLayer:
    """Owns the routing state, saved buffer, outputs and workspaces of one shape.

    Weights and activations are passed per call; all buffers are torch device
    tensors allocated once here (never inside route/forward/backward)."""

    def __init__(self, T, H, I, E, k, mode="bf16", device="cuda"):
        import torch
        self.dims = Dims.of(T, H, I, E, k, mode)
        self.device = device
        self.act_dtype = torch.float32 if self.dims.mode == MODE_FP32 else torch.bfloat16
        rws, saved, fws, bws = workspace_size(self.dims)
        self.routing = alloc_routing(self.dims, device)
        self.route_ws = alloc_workspace(rws, device)
        self.saved = alloc_workspace(saved, device)
        self.fwd_ws = alloc_workspace(fws, device)
        self.bwd_ws = alloc_workspace(bws, device)
        self.y = torch.empty((T, H), dtype=self.act_dtype, device=device)
        self.dx = torch.empty((T, H), dtype=self.act_dtype, device=device)
        self.dw13 = torch.empty((E, 2 * I, H), dtype=torch.float32, device=device)
        self.dw2 = torch.empty((E, H, I), dtype=torch.float32, device=device)
        self.dgate = torch.empty((T, k), dtype=torch.float32, device=device)
        self.dlogits = torch.empty((T, E), dtype=torch.float32, device=device)

    def route(self, logits, stream=None):
        route(self.dims, logits, self.routing, self.route_ws, stream)

    def route_project(self, x, w_router, stream=None):
        """Router projection logits = x w_router^T (kept in self.logits), then route."""
        import torch
        if getattr(self, "logits", None) is None:
            self.logits = torch.empty((self.dims.T, self.dims.E), dtype=torch.float32, device=self.device)
        route_project(self.dims, x, w_router, self.logits, self.routing, self.route_ws, stream)
        return self.logits

    def router_backward(self, x, w_router, dw_router, stream=None):
        """After backward(want_dlogits=True): dx += dlogits w_router, dw_router = dlogits^T x."""
        router_backward(self.dims, self.routing, self.dlogits, x, w_router, self.dx, dw_router, stream)

    def forward(self, x, w13, w2, stream=None, events=None, keep_saved=True):
        """keep_saved=False: keep no state for a backward (checkpointing's first forward)."""
        forward(self.dims, x, w13, w2, self.routing, self.y, self.saved if keep_saved else None, self.fwd_ws,
                stream, events)
        return self.y

    def forward_recompute(self, x, w13, w2, stream=None):
        """Second forward of activation checkpointing: `saved` as forward() writes it, y untouched."""
        forward_recompute(self.dims, x, w13, w2, self.routing, self.saved, self.fwd_ws, stream)

    def quantize_weights(self, w13, w2, stream=None):
        """MXFP8 copies of the weights (fp8 modes), kept in self.wcodes for the cached calls."""
        if getattr(self, "wcodes", None) is None:
            self.wcodes = alloc_workspace(weight_codes_size(self.dims), self.device)
        quantize_weights(self.dims, w13, w2, self.wcodes, stream)
        return self.wcodes

    def forward_cached(self, x, w13, w2, stream=None):
        forward_cached(self.dims, x, w13, w2, self.wcodes, self.routing, self.y, self.saved, self.fwd_ws, stream)
        return self.y

    def backward_cached(self, dy, x, want_dlogits=True, stream=None):
        backward_cached(self.dims, dy, x, self.wcodes, self.routing, self.saved, self.dx, self.dw13, self.dw2,
                        self.dgate, self.dlogits if want_dlogits else None, self.bwd_ws, stream)
        return self.dx, self.dw13, self.dw2, self.dgate, (self.dlogits if want_dlogits else None)

    def backward(self, dy, x, w13, w2, want_dlogits=True, stream=None, events=None, accumulate=False):
        backward(self.dims, dy, x, w13, w2, self.routing, self.saved, self.dx, self.dw13, self.dw2, self.dgate,
                 self.dlogits if want_dlogits else None, self.bwd_ws, stream, events, accumulate)
        return self.dx, self.dw13, self.dw2, self.dgate, (self.dlogits if want_dlogits else None)
