"""B200-native (sm_100a) Mixture-of-Experts layer forward.

Python binding of the C ABI in ``include/moe.h`` (``libmoe.so``, built in-tree by
``mixture_experts_layer_logits_b200/build.py``).  The functions here only marshal
arguments -- device pointers, the shape struct and the current CUDA stream --
into the library; every step of the layer runs in its CUDA kernels.  There is no
fallback: if the library is missing or a call fails, an exception is raised.

torch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

__all__ = [
    "MoeError", "Shape", "moe_workspace_size", "moe_route", "moe_permute", "moe_grouped_ffn",
    "moe_combine", "moe_forward", "moe_forward_timed", "moe_forward_kernel_count",
    "moe_forward_fused", "moe_forward_w8", "moe_forward_w8_supported", "moe_selftest_wait_timeout",
    "moe_device_status", "library_path", "load_library",
    "MOE_OK", "MOE_ERR_INVALID_ARG", "MOE_ERR_UNSUPPORTED_SHAPE", "MOE_ERR_MISALIGNED",
    "MOE_ERR_WORKSPACE_TOO_SMALL", "MOE_ERR_CUDA", "MOE_ERR_DEVICE_TIMEOUT",
    "MOE_ERR_DEVICE_BOUNDS", "debug_library_path",
    "MmShape", "moe_quantize_mx", "moe_add_rmsnorm", "moe_grouped_mm_workspace_size",
    "moe_grouped_mm_mx4", "moe_mx4_workspace_size", "moe_grouped_ffn_mx4", "moe_forward_mx4",
    "workspace_mx4",
]

(MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED_SHAPE, MOE_ERR_MISALIGNED,
 MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_CUDA, MOE_ERR_DEVICE_TIMEOUT,
 MOE_ERR_DEVICE_BOUNDS) = range(8)

_HERE = os.path.dirname(os.path.abspath(__file__))
# libmoe_debug.so: the same library with the kernels' input-index checks compiled
# in (moe_device_status then reports MOE_ERR_DEVICE_BOUNDS); MOE_LIBRARY=debug in
# the environment selects it at import.
debug_library_path = os.path.join(_HERE, "libmoe_debug.so")
library_path = (debug_library_path if os.environ.get("MOE_LIBRARY", "") == "debug"
                else os.path.join(_HERE, "libmoe.so"))


class Shape(ctypes.Structure):
    """moe_shape_t: T tokens, E experts, top_k, H hidden, I intermediate."""

    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("H", ctypes.c_int32), ("I", ctypes.c_int32)]

    def __repr__(self):
        return f"Shape(T={self.T}, E={self.E}, top_k={self.top_k}, H={self.H}, I={self.I})"


class MmShape(ctypes.Structure):
    """moe_mm_shape_t: R token rows, E experts, N outputs, K inputs."""

    _fields_ = [("R", ctypes.c_int32), ("E", ctypes.c_int32), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = load_library()
        msg = lib.moe_status_string(status).decode()
        if status == MOE_ERR_CUDA:
            msg += f" (cudaError {lib.moe_last_cuda_error()})"
        super().__init__(f"{where}: {msg}")
        self.status = status


_lib = None
_vp = ctypes.c_void_p


def load_library():
    """Load the library at library_path (raises OSError if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise OSError(f"{library_path} is missing: run mixture_experts_layer_logits_b200/build.py")
    lib = ctypes.CDLL(library_path)
    lib.moe_workspace_size.argtypes = [Shape]
    lib.moe_workspace_size.restype = ctypes.c_size_t
    lib.moe_route.argtypes = [_vp, Shape, _vp, _vp, _vp]
    lib.moe_permute.argtypes = [_vp, Shape, _vp, _vp, _vp, ctypes.c_size_t, _vp]
    lib.moe_grouped_ffn.argtypes = [_vp, _vp, _vp, _vp, _vp, Shape, _vp, _vp, ctypes.c_size_t, _vp]
    lib.moe_combine.argtypes = [_vp, _vp, Shape, _vp, _vp]
    lib.moe_forward.argtypes = [_vp, _vp, _vp, _vp, Shape, _vp, _vp, _vp, _vp, _vp, _vp,
                                ctypes.c_size_t, _vp]
    lib.moe_forward_timed.argtypes = [_vp, _vp, _vp, _vp, Shape, _vp, _vp, _vp, _vp, _vp, _vp,
                                      ctypes.c_size_t, _vp, ctypes.POINTER(_vp), ctypes.c_int]
    lib.moe_forward_w8.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, Shape, _vp, _vp, _vp, _vp, _vp,
                                   _vp, ctypes.c_size_t, _vp]
    lib.moe_forward_w8_timed.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, Shape, _vp, _vp, _vp, _vp,
                                         _vp, _vp, ctypes.c_size_t, _vp, ctypes.POINTER(_vp),
                                         ctypes.c_int]
    lib.moe_forward_w8_supported.argtypes = [Shape]
    lib.moe_forward_w8_supported.restype = ctypes.c_int
    lib.moe_forward_kernel_count.argtypes = [Shape]
    lib.moe_forward_kernel_count.restype = ctypes.c_int
    lib.moe_forward_fused.argtypes = [Shape]
    lib.moe_forward_fused.restype = ctypes.c_int
    lib.moe_selftest_wait_timeout.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint,
                                              ctypes.c_void_p]
    lib.moe_selftest_wait_timeout.restype = ctypes.c_int
    lib.moe_device_status.argtypes = [_vp, ctypes.c_size_t, _vp]
    i64, sz = ctypes.c_int64, ctypes.c_size_t
    lib.moe_quantize_mx.argtypes = [_vp, ctypes.c_int, i64, i64, ctypes.c_int, _vp, _vp, _vp]
    lib.moe_add_rmsnorm.argtypes = [_vp, _vp, _vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_float,
                                    _vp, _vp, _vp, _vp, _vp]
    lib.moe_grouped_mm_workspace_size.argtypes = [MmShape]
    lib.moe_grouped_mm_workspace_size.restype = sz
    lib.moe_grouped_mm_mx4.argtypes = [_vp] * 5 + [MmShape, _vp, _vp, sz, _vp]
    lib.moe_mx4_workspace_size.argtypes = [Shape]
    lib.moe_mx4_workspace_size.restype = sz
    lib.moe_grouped_ffn_mx4.argtypes = [_vp] * 8 + [Shape, _vp, _vp, sz, _vp]
    lib.moe_forward_mx4.argtypes = [_vp] * 7 + [Shape] + [_vp] * 6 + [sz, _vp]
    for fn in (lib.moe_quantize_mx, lib.moe_add_rmsnorm, lib.moe_grouped_mm_mx4,
               lib.moe_grouped_ffn_mx4, lib.moe_forward_mx4):
        fn.restype = ctypes.c_int
    for fn in (lib.moe_route, lib.moe_permute, lib.moe_grouped_ffn, lib.moe_combine,
               lib.moe_forward, lib.moe_forward_timed, lib.moe_forward_w8,
               lib.moe_forward_w8_timed, lib.moe_device_status):
        fn.restype = ctypes.c_int
    lib.moe_status_string.argtypes = [ctypes.c_int]
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_last_cuda_error.argtypes = []
    lib.moe_last_cuda_error.restype = ctypes.c_int
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _need(t: torch.Tensor, name: str, dtype, shape):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous CUDA {dtype} {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def moe_workspace_size(T: int, E: int, top_k: int, H: int = 0, I: int = 0) -> int:
    return int(load_library().moe_workspace_size(Shape(T, E, top_k, H, I)))


def workspace(T: int, E: int, top_k: int, H: int = 0, I: int = 0, device="cuda") -> torch.Tensor:
    """A device workspace big enough for the shape (uint8)."""
    n = moe_workspace_size(T, E, top_k, H, I)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_route(logits: torch.Tensor, top_k: int, topk_ids=None, topk_weights=None):
    T, E = logits.shape
    _need(logits, "logits", torch.float32, (T, E))
    ids = topk_ids if topk_ids is not None else torch.empty(T, top_k, dtype=torch.int32,
                                                            device=logits.device)
    w = topk_weights if topk_weights is not None else torch.empty(T, top_k, dtype=torch.float32,
                                                                  device=logits.device)
    _need(ids, "topk_ids", torch.int32, (T, top_k))
    _need(w, "topk_weights", torch.float32, (T, top_k))
    _check(load_library().moe_route(_ptr(logits), Shape(T, E, top_k, 0, 0), _ptr(ids), _ptr(w),
                                    _stream(logits)), "moe_route")
    return ids, w


def moe_permute(topk_ids: torch.Tensor, E: int, ws: torch.Tensor = None, expert_offsets=None,
                permuted_rows=None):
    T, k = topk_ids.shape
    _need(topk_ids, "topk_ids", torch.int32, (T, k))
    dev = topk_ids.device
    if ws is None:
        ws = workspace(T, E, k, device=dev)
    off = expert_offsets if expert_offsets is not None else torch.empty(E + 1, dtype=torch.int32,
                                                                        device=dev)
    rows = permuted_rows if permuted_rows is not None else torch.empty(T * k, dtype=torch.int32,
                                                                       device=dev)
    _need(off, "expert_offsets", torch.int32, (E + 1,))
    _need(rows, "permuted_rows", torch.int32, (T * k,))
    _check(load_library().moe_permute(_ptr(topk_ids), Shape(T, E, k, 0, 0), _ptr(off), _ptr(rows),
                                      _ptr(ws), ws.numel(), _stream(topk_ids)), "moe_permute")
    return off, rows


def moe_grouped_ffn(x, w13, w2, expert_offsets, permuted_rows, top_k: int, ws=None, y=None):
    T, H = x.shape
    E, twoI, _ = w13.shape
    I = twoI // 2
    dev = x.device
    _need(x, "x", torch.bfloat16, (T, H))
    _need(w13, "w13", torch.bfloat16, (E, 2 * I, H))
    _need(w2, "w2", torch.bfloat16, (E, H, I))
    _need(expert_offsets, "expert_offsets", torch.int32, (E + 1,))
    _need(permuted_rows, "permuted_rows", torch.int32, (T * top_k,))
    if ws is None:
        ws = workspace(T, E, top_k, H, I, device=dev)
    if y is None:
        y = torch.empty(T * top_k, H, dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, (T * top_k, H))
    _check(load_library().moe_grouped_ffn(_ptr(x), _ptr(w13), _ptr(w2), _ptr(expert_offsets),
                                          _ptr(permuted_rows), Shape(T, E, top_k, H, I), _ptr(y),
                                          _ptr(ws), ws.numel(), _stream(x)), "moe_grouped_ffn")
    return y


def moe_combine(y, topk_weights, out=None):
    T, k = topk_weights.shape
    H = y.shape[1]
    _need(y, "y", torch.bfloat16, (T * k, H))
    _need(topk_weights, "topk_weights", torch.float32, (T, k))
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=y.device)
    _need(out, "out", torch.bfloat16, (T, H))
    _check(load_library().moe_combine(_ptr(y), _ptr(topk_weights), Shape(T, k, k, H, 0),
                                      _ptr(out), _stream(y)), "moe_combine")
    return out


def _forward(x, logits, w13, w2, top_k, ws, out, topk_ids, topk_weights, expert_offsets,
             permuted_rows, events, scales=None):
    T, H = x.shape
    E = logits.shape[1]
    I = w13.shape[1] // 2
    dev = x.device
    wdt = torch.bfloat16 if scales is None else torch.uint8
    _need(x, "x", torch.bfloat16, (T, H))
    _need(logits, "logits", torch.float32, (T, E))
    _need(w13, "w13", wdt, (E, 2 * I, H))
    _need(w2, "w2", wdt, (E, H, I))
    if scales is not None:
        _need(scales[0], "w13_scale", torch.float32, (E, 2 * I))
        _need(scales[1], "w2_scale", torch.float32, (E, H))
    if ws is None:
        ws = workspace(T, E, top_k, H, I, device=dev)
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, (T, H))
    for t, name, dt, shp in ((topk_ids, "topk_ids", torch.int32, (T, top_k)),
                             (topk_weights, "topk_weights", torch.float32, (T, top_k)),
                             (expert_offsets, "expert_offsets", torch.int32, (E + 1,)),
                             (permuted_rows, "permuted_rows", torch.int32, (T * top_k,))):
        if t is not None:
            _need(t, name, dt, shp)
    weights = ((_ptr(w13), _ptr(w2)) if scales is None else
               (_ptr(w13), _ptr(scales[0]), _ptr(w2), _ptr(scales[1])))
    args = (_ptr(x), _ptr(logits), *weights, Shape(T, E, top_k, H, I), _ptr(out),
            _ptr(topk_ids), _ptr(topk_weights), _ptr(expert_offsets), _ptr(permuted_rows),
            _ptr(ws), ws.numel(), _stream(x))
    lib = load_library()
    name = "moe_forward" if scales is None else "moe_forward_w8"
    if events is None:
        _check(getattr(lib, name)(*args), name)
    else:
        arr = (_vp * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
        _check(getattr(lib, name + "_timed")(*args, arr, len(events)), name + "_timed")
    return out


def moe_forward(x, logits, w13, w2, top_k: int, ws=None, out=None, topk_ids=None,
                topk_weights=None, expert_offsets=None, permuted_rows=None):
    return _forward(x, logits, w13, w2, top_k, ws, out, topk_ids, topk_weights, expert_offsets,
                    permuted_rows, None)


def moe_forward_timed(x, logits, w13, w2, top_k: int, events, ws=None, out=None, topk_ids=None,
                      topk_weights=None, expert_offsets=None, permuted_rows=None):
    """moe_forward that records the 5 torch.cuda.Event objects in `events` at the
    stage boundaries (before routing, after permute, after w13, after w2, after
    combine)."""
    if len(events) != 5:
        raise ValueError("moe_forward_timed needs 5 events")
    return _forward(x, logits, w13, w2, top_k, ws, out, topk_ids, topk_weights, expert_offsets,
                    permuted_rows, events)


def moe_forward_w8(x, logits, w13, w13_scale, w2, w2_scale, top_k: int, ws=None, out=None,
                   topk_ids=None, topk_weights=None, expert_offsets=None, permuted_rows=None,
                   events=None):
    """The layer with FP8 (E4M3) expert weights: w13 / w2 uint8 codes [E, 2I, H] /
    [E, H, I], w13_scale / w2_scale fp32 [E, 2I] / [E, H] (one scale per weight
    row).  Other arguments and outputs as moe_forward; `events` (5
    torch.cuda.Event, optional) as moe_forward_timed."""
    if events is not None and len(events) != 5:
        raise ValueError("moe_forward_w8 needs 5 events")
    return _forward(x, logits, w13, w2, top_k, ws, out, topk_ids, topk_weights, expert_offsets,
                    permuted_rows, events, scales=(w13_scale, w2_scale))


def moe_forward_w8_supported(T: int, E: int, top_k: int, H: int, I: int) -> bool:
    return bool(load_library().moe_forward_w8_supported(Shape(T, E, top_k, H, I)))


def moe_forward_kernel_count(T: int, E: int, top_k: int, H: int, I: int) -> int:
    return int(load_library().moe_forward_kernel_count(Shape(T, E, top_k, H, I)))


def moe_forward_fused(T: int, E: int, top_k: int, H: int, I: int) -> bool:
    """True if moe_forward runs the FFN and the combine as one persistent launch."""
    return bool(load_library().moe_forward_fused(Shape(T, E, top_k, H, I)))


# ------------------------------------------------------------------ microscaled operators
#
# These calls run on the current stream of their tensors' device, whichever device is
# current, and check that all tensors are on that one.  The word that moe_device_status reads lies
# in the workspace: a program that wants to know of a bounded wait that ran out passes `ws`
# (without one the call allocates its own and drops it).

_MX_FORMATS = {"e2m1": 0, "e4m3": 1}
_MX_SOURCES = {torch.bfloat16: 0, torch.float32: 1}


def _same(t: torch.Tensor, name: str, dtype, shape, device):
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


# A call of one of these on a few rows takes the host longer than the GPU, so the checks and
# allocations below are the cheapest forms that torch has.


def _out(t, name, like, dtype, shape):
    """The given output tensor, checked, or a new one on the device of `like`."""
    if t is None:
        return like.new_empty(*shape, dtype=dtype)
    _same(t, name, dtype, shape, like.device)
    return t


def _out_like(t, name, like, dtype):
    """_out of the shape of `like`."""
    if t is None:
        return torch.empty_like(like) if dtype is like.dtype else torch.empty_like(like, dtype=dtype)
    _same(t, name, dtype, like.shape, like.device)
    return t


# The current device and a device's current stream without torch's wrappers around them, or the
# public forms where a build of torch has no such entry.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, where, device, *args):
    """fn(*args, current stream of `device`) with that device current."""
    if device.type != "cuda":
        raise ValueError(f"{where}: expected CUDA tensors, got {device}")
    index = device.index
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != MOE_OK:
        raise MoeError(status, where)


def moe_quantize_mx(src: torch.Tensor, fmt: str = "e2m1", codes=None, scales=None):
    """(codes, scales): src (bf16 or fp32 [..., cols], cols a multiple of 32) in microscaled
    blocks of 32 columns.  fmt "e2m1": codes uint8 [..., cols / 2], the lower column in
    the low nibble; "e4m3": codes uint8 [..., cols].  scales uint8 [..., cols / 32],
    2^(code - 127)."""
    if fmt not in _MX_FORMATS:
        raise ValueError(f"fmt: expected 'e2m1' or 'e4m3', got {fmt!r}")
    if src.dtype not in _MX_SOURCES or src.dim() < 1 or not src.is_contiguous():
        raise ValueError(f"src: expected a contiguous bf16 or fp32 matrix, got {src.dtype} "
                         f"{tuple(src.shape)}")
    *lead, cols = src.shape
    if cols < 32 or cols % 32 or src.numel() == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_quantize_mx")
    dev = src.device
    codes = _out(codes, "codes", src, torch.uint8, (*lead, cols // 2 if fmt == "e2m1" else cols))
    scales = _out(scales, "scales", src, torch.uint8, (*lead, cols // 32))
    _call(load_library().moe_quantize_mx, "moe_quantize_mx", dev, src.data_ptr(),
          _MX_SOURCES[src.dtype], src.numel() // cols, cols, _MX_FORMATS[fmt], codes.data_ptr(),
          scales.data_ptr())
    return codes, scales


def moe_add_rmsnorm(x, weight, eps: float = 1e-6, residual=None, quantize: bool = False,
                    sum_out=None, out=None, codes=None, scales=None):
    """(h, out, codes, scales): h = bf16(x + residual) and its root-mean-square norm times
    weight, as bf16 `out` and, with quantize=True, in microscaled E4M3 blocks (codes uint8
    [T, H], scales uint8 [T, H / 32]); codes and scales are None without it.  x, residual bf16
    [T, H], weight bf16 [H].  Without a residual h is None and x itself is normed.
    sum_out may be the residual, which is then updated in place."""
    if x.dim() != 2:
        raise ValueError(f"x: expected [T, H], got {tuple(x.shape)}")
    shape, dev = x.shape, x.device
    T, H = shape
    if T < 1 or H < 32 or H % 32:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_add_rmsnorm")
    bf16 = torch.bfloat16
    px = _same(x, "x", bf16, shape, dev)
    pw = _same(weight, "weight", bf16, (H,), dev)
    pr = ps = pc = psc = None
    if residual is not None:
        pr = _same(residual, "residual", bf16, shape, dev)
        sum_out = _out_like(sum_out, "sum_out", x, bf16)
        ps = sum_out.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out: there is no residual to add")
    out = _out_like(out, "out", x, bf16)
    if quantize:
        codes = _out_like(codes, "codes", x, torch.uint8)
        scales = _out(scales, "scales", x, torch.uint8, (T, H // 32))
        pc, psc = codes.data_ptr(), scales.data_ptr()
    elif codes is not None or scales is not None:
        raise ValueError("codes, scales: given without quantize=True")
    _call(load_library().moe_add_rmsnorm, "moe_add_rmsnorm", dev, px, pr, pw, T, H, eps, ps,
          out.data_ptr(), pc, psc)
    return sum_out, out, codes, scales


@functools.lru_cache(maxsize=4096)
def _mm_plan(R, E, N, K):
    """(MmShape, workspace bytes)."""
    shape = MmShape(R, E, N, K)
    return shape, int(load_library().moe_grouped_mm_workspace_size(shape))


def moe_grouped_mm_workspace_size(R: int, E: int, N: int, K: int) -> int:
    return _mm_plan(R, E, N, K)[1]


def moe_grouped_mm_mx4(a, a_scale, w, w_scale, expert_offsets, ws=None, y=None):
    """y bf16 [R, N]: rows expert_offsets[e] .. expert_offsets[e + 1] of a (microscaled E4M3
    codes uint8 [R, K], scales uint8 [R, K / 32]) times w[e] transposed (E2M1 codes uint8
    [E, N, K / 2], scales uint8 [E, N, K / 32]).  Rows behind expert_offsets[E] are not
    written."""
    if a.dim() != 2 or w.dim() != 3:
        raise ValueError(f"a, w: expected [R, K] and [E, N, K / 2], got {tuple(a.shape)} and "
                         f"{tuple(w.shape)}")
    R, K = a.shape
    E, N, _ = w.shape
    dev, u8 = a.device, torch.uint8
    shape, need = _mm_plan(R, E, N, K)
    if need == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_grouped_mm_mx4")
    ptrs = (_same(a, "a", u8, (R, K), dev),
            _same(a_scale, "a_scale", u8, (R, K // 32), dev),
            _same(w, "w", u8, (E, N, K // 2), dev),
            _same(w_scale, "w_scale", u8, (E, N, K // 32), dev),
            _same(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev))
    y = _out(y, "y", a, torch.bfloat16, (R, N))
    ws = _workspace_of(ws, need, a)
    _call(load_library().moe_grouped_mm_mx4, "moe_grouped_mm_mx4", dev, *ptrs, shape,
          y.data_ptr(), ws.data_ptr(), ws.numel())
    return y


@functools.lru_cache(maxsize=4096)
def _mx4_plan(T, E, top_k, H, I):
    """(Shape, workspace bytes)."""
    shape = Shape(T, E, top_k, H, I)
    return shape, int(load_library().moe_mx4_workspace_size(shape))


def moe_mx4_workspace_size(T: int, E: int, top_k: int, H: int, I: int) -> int:
    return _mx4_plan(T, E, top_k, H, I)[1]


def workspace_mx4(T: int, E: int, top_k: int, H: int, I: int, device="cuda") -> torch.Tensor:
    """A device workspace of moe_grouped_ffn_mx4 and moe_forward_mx4 for the shape (uint8)."""
    n = moe_mx4_workspace_size(T, E, top_k, H, I)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_mx4_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _workspace_of(ws, need, like):
    if ws is None:
        return like.new_empty(need, dtype=torch.uint8)
    if ws.dtype is not torch.uint8 or ws.device != like.device or not ws.is_contiguous():
        raise ValueError(f"ws: expected contiguous uint8 on {like.device}, got {ws.dtype} on "
                         f"{ws.device}")
    return ws


def _mx4_operands(where, x, x_scale, w13, w13_scale, w2, w2_scale, top_k):
    """(Shape, workspace bytes, pointers) of the checked x and weights."""
    if x.dim() != 2 or w13.dim() != 3 or w2.dim() != 3:
        raise ValueError(f"{where}: expected x [T, H], w13 [E, 2I, H / 2] and w2 [E, H, I / 2]")
    T, H = x.shape
    E = w13.shape[0]
    I = w13.shape[1] // 2
    shape, need = _mx4_plan(T, E, top_k, H, I)
    if need == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, where)
    dev, u8 = x.device, torch.uint8
    return shape, need, (
        _same(x, "x", u8, (T, H), dev),
        _same(x_scale, "x_scale", u8, (T, H // 32), dev),
        _same(w13, "w13", u8, (E, 2 * I, H // 2), dev),
        _same(w13_scale, "w13_scale", u8, (E, 2 * I, H // 32), dev),
        _same(w2, "w2", u8, (E, H, I // 2), dev),
        _same(w2_scale, "w2_scale", u8, (E, H, I // 32), dev))


def moe_grouped_ffn_mx4(x, x_scale, w13, w13_scale, w2, w2_scale, expert_offsets, permuted_rows,
                        top_k: int, ws=None, y=None):
    """moe_grouped_ffn on microscaled operands: x E4M3 codes uint8 [T, H], w13 and w2 E2M1
    codes uint8 [E, 2I, H / 2] and [E, H, I / 2], each with its uint8 scales
    [..., cols / 32]; y bf16 [T*k, H].  act is microscaled E4M3 between the two products."""
    shape, need, ptrs = _mx4_operands("moe_grouped_ffn_mx4", x, x_scale, w13, w13_scale, w2,
                                      w2_scale, top_k)
    dev, R = x.device, shape.T * top_k
    off = _same(expert_offsets, "expert_offsets", torch.int32, (shape.E + 1,), dev)
    rows = _same(permuted_rows, "permuted_rows", torch.int32, (R,), dev)
    y = _out(y, "y", x, torch.bfloat16, (R, shape.H))
    ws = _workspace_of(ws, need, x)
    _call(load_library().moe_grouped_ffn_mx4, "moe_grouped_ffn_mx4", dev, *ptrs, off, rows, shape,
          y.data_ptr(), ws.data_ptr(), ws.numel())
    return y


def moe_forward_mx4(x, x_scale, logits, w13, w13_scale, w2, w2_scale, top_k: int, ws=None,
                    out=None, topk_ids=None, topk_weights=None, expert_offsets=None,
                    permuted_rows=None):
    """The whole layer on microscaled operands (see moe_grouped_ffn_mx4), any T.  Other
    arguments and outputs as moe_forward; ws of workspace_mx4."""
    shape, need, ptrs = _mx4_operands("moe_forward_mx4", x, x_scale, w13, w13_scale, w2, w2_scale,
                                      top_k)
    dev, T, E = x.device, shape.T, shape.E
    plog = _same(logits, "logits", torch.float32, (T, E), dev)
    extra = [None if t is None else _same(t, name, dt, shp, dev)
             for t, name, dt, shp in ((topk_ids, "topk_ids", torch.int32, (T, top_k)),
                                      (topk_weights, "topk_weights", torch.float32, (T, top_k)),
                                      (expert_offsets, "expert_offsets", torch.int32, (E + 1,)),
                                      (permuted_rows, "permuted_rows", torch.int32, (T * top_k,)))]
    out = _out(out, "out", x, torch.bfloat16, (T, shape.H))
    ws = _workspace_of(ws, need, x)
    _call(load_library().moe_forward_mx4, "moe_forward_mx4", dev, *ptrs[:2], plog, *ptrs[2:],
          shape, out.data_ptr(), *extra, ws.data_ptr(), ws.numel())
    return out


def moe_selftest_wait_timeout(ws: torch.Tensor, limit_us: int) -> None:
    """Queue the failure-detection self-test: two unsatisfiable bounded waits that
    give up after limit_us and record a timeout in ws (see moe_device_status)."""
    _check(load_library().moe_selftest_wait_timeout(_ptr(ws), ws.numel(), int(limit_us),
                                                    _stream(ws)), "moe_selftest_wait_timeout")


def moe_device_status(ws: torch.Tensor) -> int:
    """Synchronise the current stream and return (and clear) the device error status."""
    return int(load_library().moe_device_status(_ptr(ws), ws.numel(), _stream(ws)))
