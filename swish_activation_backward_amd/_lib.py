"""ctypes binding of libswiglu_bwd.so: argument marshalling only.

Each function has the name of the C entry point it calls and takes torch CUDA (HIP)
tensors: it checks shapes and dtypes, turns tensors into device pointers and sizes,
passes torch's current stream, and raises ``SwgError`` on a non-zero status.  All
arithmetic happens in the library's HIP kernels; there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading
from typing import NamedTuple, Optional

import torch

__all__ = ["SwgError", "load_library", "library_path", "swish_grad", "swish_grad_strided",
           "swiglu_bwd_b", "swiglu_bwd_b_noalloc", "swiglu_bwd_w", "swiglu_bwd_x", "swiglu_fwd",
           "swiglu_bwd_b_workspace_size", "swiglu_bwd_w_workspace_size", "swg_version",
           "swg_time_next_call", "swiglu_bwd_wx", "swiglu_bwd_wx_workspace_size",
           "swiglu_bwd_gemm_tile", "swg_set_gemm_tile", "DTYPE_CODE", "STATUS",
           "layer_norm_fwd", "layer_norm_bwd", "layer_norm_bwd_workspace_size", "TokenLogprobs",
           "token_logprobs", "token_logprobs_bwd", "token_logprobs_workspace_size", "distill_fwd",
           "distill_bwd", "distill_fwd_bwd", "distill_workspace_size", "MAX_TOP", "MAX_TEACHER"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libswiglu_bwd.so"

DTYPE_CODE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
STATUS = {0: "SWG_OK", 1: "SWG_ERR_NULLPTR", 2: "SWG_ERR_INVALID", 3: "SWG_ERR_UNSUPPORTED",
          4: "SWG_ERR_WORKSPACE", 5: "SWG_ERR_HIP"}

_lock = threading.Lock()
_lib = None


class SwgError(RuntimeError):
    def __init__(self, call: str, status: int, lib):
        self.status = status
        msg = lib.swg_status_string(status).decode()
        if status == 5:
            msg += f" (hipError_t {lib.swg_last_hip_error()})"
        super().__init__(f"{call}: {msg}")


def library_path() -> str:
    return os.environ.get("SWIGLU_BWD_LIB", os.path.join(_HERE, _LIB_NAME))


def load_library():
    """Load the HIP library (raises if it has not been built: no fallback exists)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m swish_activation_backward_amd.build`"
                " (the SwiGLU backward has no CPU fallback)")
        lib = ctypes.CDLL(path)
        vp, i64, sz, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
        lib.swish_grad.argtypes = [vp, vp, vp, i64, i32, ctypes.POINTER(ctypes.c_float), vp]
        lib.swish_grad.restype = i32
        pi64 = ctypes.POINTER(ctypes.c_int64)
        lib.swish_grad_strided.argtypes = [vp, vp, vp, i32, pi64, pi64, pi64, pi64, i32,
                                           ctypes.POINTER(ctypes.c_float), vp]
        lib.swish_grad_strided.restype = i32
        lib.swiglu_bwd_b.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, vp, sz, vp]
        lib.swiglu_bwd_b.restype = i32
        lib.swiglu_bwd_b_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, vp]
        lib.swiglu_bwd_b_noalloc.restype = i32
        lib.swiglu_bwd_b_workspace_size.argtypes = [i64, i64, i32]
        lib.swiglu_bwd_b_workspace_size.restype = sz
        lib.swiglu_bwd_w.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, sz, vp]
        lib.swiglu_bwd_w.restype = i32
        lib.swiglu_bwd_w_workspace_size.argtypes = [i64, i64, i64, i32]
        lib.swiglu_bwd_w_workspace_size.restype = sz
        lib.swiglu_bwd_x.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp]
        lib.swiglu_bwd_x.restype = i32
        lib.swiglu_bwd_wx.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp,
                                      sz, vp]
        lib.swiglu_bwd_wx.restype = i32
        lib.swiglu_bwd_wx_workspace_size.argtypes = [i64, i64, i64, i32]
        lib.swiglu_bwd_wx_workspace_size.restype = sz
        lib.swiglu_bwd_gemm_tile.argtypes = [i32, i64, i64, i64, i32]
        lib.swiglu_bwd_gemm_tile.restype = i32
        lib.swg_set_gemm_tile.argtypes = [i32]
        lib.swg_set_gemm_tile.restype = i32
        lib.swiglu_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp]
        lib.swiglu_fwd.restype = i32
        f32 = ctypes.c_float
        lib.layer_norm_fwd.argtypes = [vp, i64, vp, vp, vp, i64, vp, vp, i64, i64, f32, i32, i32,
                                       vp]
        lib.layer_norm_fwd.restype = i32
        lib.layer_norm_bwd.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, vp, i32, i64,
                                       i64, i32, i32, vp, sz, vp]
        lib.layer_norm_bwd.restype = i32
        lib.layer_norm_bwd_workspace_size.argtypes = [i64, i64, i32]
        lib.layer_norm_bwd_workspace_size.restype = sz
        lib.token_logprobs.argtypes = [vp, i64, vp, vp, vp, vp, vp, vp, i64, i64, i64, f32, i64,
                                       i32, vp, sz, vp]
        lib.token_logprobs.restype = i32
        lib.token_logprobs_workspace_size.argtypes = [i64, i64, i64, i32]
        lib.token_logprobs_workspace_size.restype = sz
        lib.token_logprobs_bwd.argtypes = [vp, i64, vp, vp, vp, vp, vp, vp, i64, i64, i64, f32,
                                           i64, i32, vp]
        lib.token_logprobs_bwd.restype = i32
        lib.distill_fwd.argtypes = [vp, i64, vp, vp, i64, vp, vp, i64, i64, f32, i32, i32, vp, sz,
                                    vp]
        lib.distill_fwd.restype = i32
        lib.distill_workspace_size.argtypes = [i64, i64, i64, i32]
        lib.distill_workspace_size.restype = sz
        lib.distill_bwd.argtypes = [vp, i64, vp, vp, i64, vp, vp, vp, i64, i64, i64, f32, i32, i32,
                                    vp]
        lib.distill_bwd.restype = i32
        lib.distill_fwd_bwd.argtypes = [vp, i64, vp, vp, i64, vp, vp, vp, vp, i64, i64, i64, f32,
                                        i32, i32, vp, sz, vp]
        lib.distill_fwd_bwd.restype = i32
        lib.swg_status_string.argtypes = [i32]
        lib.swg_status_string.restype = ctypes.c_char_p
        lib.swg_last_hip_error.argtypes = []
        lib.swg_last_hip_error.restype = i32
        lib.swg_time_next_call.argtypes = [vp, vp]
        lib.swg_time_next_call.restype = i32
        lib.swg_version.argtypes = []
        lib.swg_version.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _ptr(t):
    """Device pointer of a GPU tensor; host tensors are refused (the kernels would
    dereference host addresses)."""
    if t is None:
        return None
    if t.device.type != "cuda":
        raise ValueError(f"tensor on {t.device}: the library computes on the GPU only "
                         f"(move inputs and outputs to a cuda device)")
    return ctypes.c_void_p(t.data_ptr())


def _on_device(device):
    """Context that makes ``device`` HIP's current device for the launch (the library
    launches on the current device); host tensors are refused."""
    if device.type != "cuda":
        raise ValueError(f"tensor on {device}: the library computes on the GPU only "
                         f"(move inputs and outputs to a cuda device)")
    if device.index == torch.cuda.current_device():
        return _SAME_DEVICE
    return torch.cuda.device(device)


_SAME_DEVICE = contextlib.nullcontext()


def _check_stream(stream, device):
    """A stream of another device cannot order work on the tensors' one."""
    if stream.device != device:
        raise ValueError(f"stream of {stream.device}, expected one of {device}")


def _stream(stream, device):
    """The stream handle to launch on: ``stream``, else torch's current stream of the
    tensors' device."""
    if stream is None:
        # the handle itself: a torch.cuda.Stream object costs about a microsecond
        return torch._C._cuda_getCurrentRawStream(device.index)
    _check_stream(stream, device)
    return stream.cuda_stream


def _on_stream(stream, t):
    """Context that makes ``stream`` torch's current one for a call on ``t``'s device."""
    if isinstance(t, torch.Tensor) and t.device.type == "cuda":   # others are refused inside
        _check_stream(stream, t.device)
    return torch.cuda.stream(stream)


def _check(call, status, lib):
    if status != 0:
        raise SwgError(call, status, lib)


def _dense(name, t, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _dtype_code(t):
    if t.dtype not in DTYPE_CODE:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return DTYPE_CODE[t.dtype]


def _workspace(nbytes, workspace, device, stream):
    """The caller's workspace (checked), or a new one from torch's allocator.  A new one is
    marked as used on ``stream`` so that the allocator does not hand its memory out again
    before the kernels queued there have finished with it."""
    if nbytes == 0:
        return workspace
    if workspace is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        if stream is not None:
            ws.record_stream(stream)
        return ws
    if workspace.numel() * workspace.element_size() < nbytes or not workspace.is_contiguous():
        raise ValueError(f"workspace needs {nbytes} contiguous bytes")
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, expected {device}")
    return workspace


def swg_version() -> str:
    return load_library().swg_version().decode()


def swg_time_next_call(start, stop):
    """Attach two ``torch.cuda.Event`` (timing enabled, each recorded at least once so that
    torch has created it) to the kernels of the next library call on this thread: after it,
    ``start.elapsed_time(stop)`` is the span from its first kernel's start to its last
    kernel's end.  ``None, None`` cancels."""
    lib = load_library()
    handles = []
    for name, e in (("start", start), ("stop", stop)):
        if e is None:
            handles.append(None)
            continue
        h = e.cuda_event
        if not h:
            raise ValueError(f"{name} event has no HIP event yet: record it once first")
        handles.append(ctypes.c_void_p(h))
    _check("swg_time_next_call", lib.swg_time_next_call(*handles), lib)


def _same_kind(name, t, dtype, shape, device):
    """dtype, shape and device checks without a layout requirement (strided calls)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def swish_grad(grad, x, grad_x=None, beta=None, stream=None):
    """grad_x = grad * sigma(beta x) * (1 + beta x (1 - sigma(beta x)))  (elementwise, any
    shape).  ``beta`` None means 1.0; ``grad_x`` may be ``grad`` or ``x`` (in place).
    Contiguous tensors go to ``swish_grad``; any other layout (transposed, sliced,
    broadcast inputs, a non-contiguous output) to ``swish_grad_strided``."""
    _same_kind("x", x, grad.dtype, grad.shape, grad.device)
    if grad_x is None:
        grad_x = torch.empty(grad.shape, dtype=grad.dtype, device=grad.device)
    _same_kind("grad_x", grad_x, grad.dtype, grad.shape, grad.device)
    if not (grad.is_contiguous() and x.is_contiguous() and grad_x.is_contiguous()):
        return swish_grad_strided(grad, x, grad_x, beta=beta, stream=stream)
    lib = load_library()
    b = None if beta is None else ctypes.byref(ctypes.c_float(beta))
    with _on_device(grad.device):
        st = lib.swish_grad(_ptr(grad), _ptr(x), _ptr(grad_x), grad.numel(), _dtype_code(grad),
                            b, _stream(stream, grad.device))
    _check("swish_grad", st, lib)
    return grad_x


def swish_grad_strided(grad, x, grad_x, beta=None, stream=None):
    """The Swish gradient over tensors of one shape with any strides (the C entry point
    of the same name: passes torch's sizes and element strides)."""
    _same_kind("x", x, grad.dtype, grad.shape, grad.device)
    _same_kind("grad_x", grad_x, grad.dtype, grad.shape, grad.device)
    lib = load_library()
    nd = grad.dim()
    arr = ctypes.c_int64 * max(nd, 1)
    sizes = arr(*grad.shape)
    sg, sx, so = arr(*grad.stride()), arr(*x.stride()), arr(*grad_x.stride())
    b = None if beta is None else ctypes.byref(ctypes.c_float(beta))
    with _on_device(grad.device):
        st = lib.swish_grad_strided(_ptr(grad), _ptr(x), _ptr(grad_x), nd, sizes, sg, sx, so,
                                    _dtype_code(grad), b, _stream(stream, grad.device))
    _check("swish_grad_strided", st, lib)
    return grad_x


def swiglu_bwd_b_workspace_size(M: int, N: int, dtype) -> int:
    return int(load_library().swiglu_bwd_b_workspace_size(M, N, DTYPE_CODE[dtype]))


def swiglu_bwd_w_workspace_size(M: int, K: int, N: int, dtype) -> int:
    return int(load_library().swiglu_bwd_w_workspace_size(M, K, N, DTYPE_CODE[dtype]))


def swiglu_bwd_b(dy, g, fc, dg, dfc, db_g, db_fc, workspace=None, stream=None):
    """b stage: writes dg, dfc [M, N]; accumulates db_g, db_fc [N] (+=)."""
    lib = load_library()
    if dy.dim() != 2:
        raise ValueError("dy must be [M, N]")
    M, N = dy.shape
    dt, dev = dy.dtype, dy.device
    for name, t in (("dy", dy), ("g", g), ("fc", fc), ("dg", dg), ("dfc", dfc)):
        _dense(name, t, dt, (M, N), dev)
    for name, t in (("db_g", db_g), ("db_fc", db_fc)):
        if t.numel() != N:
            raise ValueError(f"{name} must hold N = {N} elements")
        _dense(name, t, dt, t.shape, dev)
    code = _dtype_code(dy)
    nbytes = int(lib.swiglu_bwd_b_workspace_size(M, N, code))
    with _on_device(dev):
        ws = _workspace(nbytes, workspace, dev, stream)
        st = lib.swiglu_bwd_b(_ptr(dy), _ptr(g), _ptr(fc), _ptr(dg), _ptr(dfc), _ptr(db_g),
                              _ptr(db_fc), M, N, code, _ptr(ws), 0 if ws is None else
                              ws.numel() * ws.element_size(), _stream(stream, dev))
    _check("swiglu_bwd_b", st, lib)


def swiglu_bwd_b_noalloc(dy, g, fc, dg, dfc, db_g, db_fc, stream=None):
    """b stage with the column partials in the library's static device array (no
    workspace, no allocation); same results as ``swiglu_bwd_b``."""
    lib = load_library()
    if dy.dim() != 2:
        raise ValueError("dy must be [M, N]")
    M, N = dy.shape
    dt, dev = dy.dtype, dy.device
    for name, t in (("dy", dy), ("g", g), ("fc", fc), ("dg", dg), ("dfc", dfc)):
        _dense(name, t, dt, (M, N), dev)
    for name, t in (("db_g", db_g), ("db_fc", db_fc)):
        if t.numel() != N:
            raise ValueError(f"{name} must hold N = {N} elements")
        _dense(name, t, dt, t.shape, dev)
    with _on_device(dev):
        st = lib.swiglu_bwd_b_noalloc(_ptr(dy), _ptr(g), _ptr(fc), _ptr(dg), _ptr(dfc),
                                      _ptr(db_g), _ptr(db_fc), M, N, _dtype_code(dy),
                                      _stream(stream, dev))
    _check("swiglu_bwd_b_noalloc", st, lib)


def swiglu_bwd_w(x, dg, dfc, dw_g, dw_fc, workspace=None, stream=None):
    """w stage: [dw_g | dw_fc] (each [K, N]) += x^T [dg | dfc]."""
    lib = load_library()
    if x.dim() != 2 or dg.dim() != 2:
        raise ValueError("x must be [M, K] and dg [M, N]")
    M, K = x.shape
    N = dg.shape[1]
    dt, dev = x.dtype, x.device
    _dense("x", x, dt, (M, K), dev)
    for name, t in (("dg", dg), ("dfc", dfc)):
        _dense(name, t, dt, (M, N), dev)
    for name, t in (("dw_g", dw_g), ("dw_fc", dw_fc)):
        _dense(name, t, dt, (K, N), dev)
    code = _dtype_code(x)
    nbytes = int(lib.swiglu_bwd_w_workspace_size(M, K, N, code))
    with _on_device(dev):
        ws = _workspace(nbytes, workspace, dev, stream)
        st = lib.swiglu_bwd_w(_ptr(x), _ptr(dg), _ptr(dfc), _ptr(dw_g), _ptr(dw_fc), M, K, N,
                              code, _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                              _stream(stream, dev))
    _check("swiglu_bwd_w", st, lib)


def swiglu_bwd_x(dg, dfc, w_g, w_fc, dx, stream=None):
    """x stage: dx [M, K] = dg W_g^T + dfc W_fc^T (overwritten)."""
    lib = load_library()
    if dg.dim() != 2 or w_g.dim() != 2:
        raise ValueError("dg must be [M, N] and w_g [K, N]")
    M, N = dg.shape
    K = w_g.shape[0]
    dt, dev = dg.dtype, dg.device
    for name, t in (("dg", dg), ("dfc", dfc)):
        _dense(name, t, dt, (M, N), dev)
    for name, t in (("w_g", w_g), ("w_fc", w_fc)):
        _dense(name, t, dt, (K, N), dev)
    _dense("dx", dx, dt, (M, K), dev)
    with _on_device(dev):
        st = lib.swiglu_bwd_x(_ptr(dg), _ptr(dfc), _ptr(w_g), _ptr(w_fc), _ptr(dx), M, K, N,
                              _dtype_code(dg), _stream(stream, dev))
    _check("swiglu_bwd_x", st, lib)


def swiglu_bwd_wx_workspace_size(M: int, K: int, N: int, dtype) -> int:
    return int(load_library().swiglu_bwd_wx_workspace_size(M, K, N, DTYPE_CODE[dtype]))


_GEMM_STAGE = {"w": 0, "x": 1, "wx": 2}


def swiglu_bwd_gemm_tile(stage: str, M: int, K: int, N: int, dtype) -> int:
    """Output tile edge (256 or 128) the planner picks for stage "w", "x" or "wx" (the fused
    pass) at this shape; 0 where the stage does not use the bf16 / fp16 tiles."""
    return int(load_library().swiglu_bwd_gemm_tile(_GEMM_STAGE[stage], M, K, N,
                                                   DTYPE_CODE[dtype]))


def swg_set_gemm_tile(edge: int) -> None:
    """Make the GEMM calls (and workspace queries) on this thread use tile edge 256 or 128
    instead of the planner's choice; 0 restores the planner."""
    lib = load_library()
    _check("swg_set_gemm_tile", lib.swg_set_gemm_tile(int(edge)), lib)


def swiglu_bwd_wx(x, dg, dfc, w_g, w_fc, dw_g, dw_fc, dx, workspace=None, stream=None):
    """Fused w + x pass: [dw_g | dw_fc] += x^T [dg | dfc] and dx = [dg | dfc] [W_g | W_fc]^T
    (overwritten) in one launch over [dg | dfc]."""
    lib = load_library()
    if x.dim() != 2 or dg.dim() != 2 or w_g.dim() != 2:
        raise ValueError("x must be [M, K], dg [M, N] and w_g [K, N]")
    M, K = x.shape
    N = dg.shape[1]
    dt, dev = x.dtype, x.device
    _dense("x", x, dt, (M, K), dev)
    for name, t in (("dg", dg), ("dfc", dfc)):
        _dense(name, t, dt, (M, N), dev)
    for name, t in (("w_g", w_g), ("w_fc", w_fc), ("dw_g", dw_g), ("dw_fc", dw_fc)):
        _dense(name, t, dt, (K, N), dev)
    _dense("dx", dx, dt, (M, K), dev)
    code = _dtype_code(x)
    nbytes = int(lib.swiglu_bwd_wx_workspace_size(M, K, N, code))
    with _on_device(dev):
        ws = _workspace(nbytes, workspace, dev, stream)
        st = lib.swiglu_bwd_wx(_ptr(x), _ptr(dg), _ptr(dfc), _ptr(w_g), _ptr(w_fc), _ptr(dw_g),
                               _ptr(dw_fc), _ptr(dx), M, K, N, code, _ptr(ws),
                               0 if ws is None else ws.numel() * ws.element_size(),
                               _stream(stream, dev))
    _check("swiglu_bwd_wx", st, lib)


def swiglu_fwd(x, w_g, w_fc, b_g, b_fc, g, fc, y, stream=None):
    """SwiGLU forward: g = x W_g + b_g, fc = x W_fc + b_fc, y = SiLU(g) fc (all three
    [M, N] outputs overwritten).  ``b_g`` / ``b_fc`` may be None (no bias)."""
    lib = load_library()
    if x.dim() != 2 or w_g.dim() != 2:
        raise ValueError("x must be [M, K] and w_g [K, N]")
    M, K = x.shape
    N = w_g.shape[1]
    dt, dev = x.dtype, x.device
    _dense("x", x, dt, (M, K), dev)
    for name, t in (("w_g", w_g), ("w_fc", w_fc)):
        _dense(name, t, dt, (K, N), dev)
    for name, t in (("b_g", b_g), ("b_fc", b_fc)):
        if t is not None:
            _dense(name, t, dt, (N,), dev)
    for name, t in (("g", g), ("fc", fc), ("y", y)):
        _dense(name, t, dt, (M, N), dev)
    with _on_device(dev):
        st = lib.swiglu_fwd(_ptr(x), _ptr(w_g), _ptr(w_fc), _ptr(b_g), _ptr(b_fc), _ptr(g),
                            _ptr(fc), _ptr(y), M, K, N, _dtype_code(x), _stream(stream, dev))
    _check("swiglu_fwd", st, lib)


# ---------------------------------------------------------------- row operators
MAX_TOP = 128          # SWG_MAX_TOP
MAX_TEACHER = 1024     # SWG_MAX_TEACHER


# A call on few rows is bound by the host, so the checks below test everything at once and leave
# it to the slow ones to say what is wrong, outputs that nobody gave are made in one go, and the
# device is switched only where it is not the current one.
def _gpu(device):
    if device.type != "cuda":
        raise ValueError(f"tensor on {device}: the library computes on the GPU only "
                         f"(move inputs and outputs to a cuda device)")


def _call(name, fn, device, *args):
    """Calls an entry point on the tensors' device and torch's current stream there.  A call
    given a stream makes it the current one first, so that what it allocates belongs to it."""
    index = device.index
    handle = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st != 0:
        raise SwgError(name, st, load_library())


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(query, *args):
    return int(getattr(load_library(), query)(*args))


def _rows(name, t, dtype, shape, device):
    """Checks a matrix whose rows are contiguous (any row stride that keeps them apart) and
    returns the row stride."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape
            and t.device == device):
        _same_kind(name, t, dtype, shape, device)
    R, C = shape
    ld, inner = t.stride()
    if (C > 1 and inner != 1) or (R > 1 and ld < C):
        raise ValueError(f"{name}: strides {t.stride()} (each row must be contiguous and rows "
                         f"may not overlap)")
    return max(ld, C)


def _packed(name, t, dtype, shape, device):
    """Checks a contiguous tensor and returns its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape
            and t.device == device and t.is_contiguous()):
        _dense(name, t, dtype, shape, device)
    return t.data_ptr()


def _matrix(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected two dimensions")
    return t.shape


def _out(name, t, dtype, shape, device):
    """A contiguous output: the caller's (checked) or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _packed(name, t, dtype, shape, device)
    return t


def _addr(t):
    return None if t is None else t.data_ptr()


def _size(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


def _affine(dtype, N, device, **named):
    """The type of a norm's w, b, dw and db (the given ones agree); ``dtype`` if none is given."""
    wdtype = None
    for name, t in named.items():
        if t is None:
            continue
        if wdtype is None:
            wdtype = t.dtype
        _packed(name, t, wdtype, (N,), device)
    wdtype = dtype if wdtype is None else wdtype
    if wdtype not in DTYPE_CODE:
        raise ValueError(f"unsupported dtype {wdtype}")
    return wdtype


def layer_norm_fwd(x, w, b, y=None, mean=None, rstd=None, eps=1e-5, stream=None):
    """Layer norm over the rows of x [M, N]: y = (x - mean) rstd w + b.  ``w`` and ``b`` [N] (or
    None) have x's dtype or fp32.  Returns y [M, N], and the fp32 mean and rstd [M] that
    ``layer_norm_bwd`` takes; outputs that are not given are allocated."""
    if stream is not None:
        with _on_stream(stream, x):
            return layer_norm_fwd(x, w, b, y, mean, rstd, eps)
    lib = load_library()
    shape = _matrix("x", x)
    M, N = shape
    dt, dev = x.dtype, x.device
    code = _dtype_code(x)
    ldx = _rows("x", x, dt, shape, dev)
    wdt = _affine(dt, N, dev, w=w, b=b)
    _gpu(dev)
    if y is None:
        y = torch.empty(shape, dtype=dt, device=dev)
    ldy = _rows("y", y, dt, shape, dev)
    mean = _out("mean", mean, torch.float32, (M,), dev)
    rstd = _out("rstd", rstd, torch.float32, (M,), dev)
    _call("layer_norm_fwd", lib.layer_norm_fwd, dev, x.data_ptr(), ldx, _addr(w), _addr(b),
          y.data_ptr(), ldy, mean.data_ptr(), rstd.data_ptr(), M, N, eps, code, DTYPE_CODE[wdt])
    return y, mean, rstd


def layer_norm_bwd_workspace_size(M: int, N: int, dtype) -> int:
    return int(load_library().layer_norm_bwd_workspace_size(M, N, DTYPE_CODE[dtype]))


def layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db, accumulate=False, workspace=None,
                   stream=None):
    """Gradients of ``layer_norm_fwd``: writes dx [M, N], dw and db [N] (each may be None);
    with ``accumulate`` dw and db are added to (+=)."""
    if stream is not None:
        with _on_stream(stream, dy):
            return layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db, accumulate, workspace)
    lib = load_library()
    shape = _matrix("dy", dy)
    M, N = shape
    dt, dev = dy.dtype, dy.device
    code = _dtype_code(dy)
    lddy = _rows("dy", dy, dt, shape, dev)
    ldx = _rows("x", x, dt, shape, dev)
    lddx = N if dx is None else _rows("dx", dx, dt, shape, dev)
    wdt = _affine(dt, N, dev, w=w, dw=dw, db=db)
    mean_at = _packed("mean", mean, torch.float32, (M,), dev)
    rstd_at = _packed("rstd", rstd, torch.float32, (M,), dev)
    _gpu(dev)
    ws = workspace
    if dw is not None or db is not None:
        ws = _workspace(_workspace_bytes("layer_norm_bwd_workspace_size", M, N, code), workspace,
                        dev, None)
    _call("layer_norm_bwd", lib.layer_norm_bwd, dev, dy.data_ptr(), lddy, x.data_ptr(),
          ldx, _addr(w), mean_at, rstd_at, _addr(dx), lddx, _addr(dw), _addr(db), int(accumulate),
          M, N, code, DTYPE_CODE[wdt], _addr(ws), _size(ws))


class TokenLogprobs(NamedTuple):
    """What ``token_logprobs`` returns, all fp32 but the int64 ids: logprob [R] (None without
    targets), entropy [R], lse [R], top_logprob and top_id [R, top] (None when top is 0)."""
    logprob: Optional[torch.Tensor]
    entropy: torch.Tensor
    lse: torch.Tensor
    top_logprob: Optional[torch.Tensor]
    top_id: Optional[torch.Tensor]


_NOTHING = TokenLogprobs(None, None, None, None, None)


def token_logprobs_workspace_size(R: int, V: int, top: int, dtype) -> int:
    return int(load_library().token_logprobs_workspace_size(R, V, top, DTYPE_CODE[dtype]))


def token_logprobs(logits, targets=None, top=0, temperature=1.0, ignore_index=-100, out=None,
                   workspace=None, stream=None):
    """Log probabilities of the ``targets`` [R] (int64) under softmax(logits / temperature),
    logits [R, V], with each row's entropy, log-sum-exp and its ``top`` likeliest entries
    (likeliest first, ties by rising id) with their log probabilities.  Returns
    ``TokenLogprobs``; ``out`` may hand back an earlier result of the same shape to be
    overwritten."""
    if stream is not None:
        with _on_stream(stream, logits):
            return token_logprobs(logits, targets, top, temperature, ignore_index, out, workspace)
    lib = load_library()
    shape = _matrix("logits", logits)
    R, V = shape
    dt, dev = logits.dtype, logits.device
    code = _dtype_code(logits)
    ld = _rows("logits", logits, dt, shape, dev)
    if targets is not None:
        _packed("targets", targets, torch.int64, (R,), dev)
    if out is None:
        out = _NOTHING
    _gpu(dev)
    f32 = torch.float32
    entropy = _out("out.entropy", out.entropy, f32, (R,), dev)
    lse = torch.empty_like(entropy) if out.lse is None else _out("out.lse", out.lse, f32, (R,), dev)
    logprob = top_lp = top_id = None
    if targets is not None:
        logprob = torch.empty_like(entropy) if out.logprob is None else _out(
            "out.logprob", out.logprob, f32, (R,), dev)
    if top > 0:
        top_lp = _out("out.top_logprob", out.top_logprob, f32, (R, top), dev)
        top_id = _out("out.top_id", out.top_id, torch.int64, (R, top), dev)
    ws = _workspace(_workspace_bytes("token_logprobs_workspace_size", R, V, top, code), workspace,
                    dev, None)
    _call("token_logprobs", lib.token_logprobs, dev, logits.data_ptr(), ld,
          _addr(targets), _addr(logprob), entropy.data_ptr(), lse.data_ptr(), _addr(top_lp),
          _addr(top_id), top, R, V, temperature, ignore_index, code, _addr(ws), _size(ws))
    return TokenLogprobs(logprob, entropy, lse, top_lp, top_id)


def token_logprobs_bwd(logits, targets, lse, entropy, dlogprob, dentropy, dlogits=None,
                       temperature=1.0, ignore_index=-100, stream=None):
    """Gradient of ``token_logprobs``'s logprob and entropy with respect to the logits, from
    dlogprob and dentropy [R] (fp32; either may be None, targets with dlogprob and entropy
    with dentropy).  ``dlogits`` [R, V] may be ``logits`` itself; it is returned."""
    if stream is not None:
        with _on_stream(stream, logits):
            return token_logprobs_bwd(logits, targets, lse, entropy, dlogprob, dentropy, dlogits,
                                      temperature, ignore_index)
    lib = load_library()
    shape = _matrix("logits", logits)
    R, V = shape
    dt, dev = logits.dtype, logits.device
    code = _dtype_code(logits)
    ld = _rows("logits", logits, dt, shape, dev)
    if targets is not None:
        _packed("targets", targets, torch.int64, (R,), dev)
    for name, t in (("lse", lse), ("entropy", entropy), ("dlogprob", dlogprob),
                    ("dentropy", dentropy)):
        if t is not None or name == "lse":
            _packed(name, t, torch.float32, (R,), dev)
    _gpu(dev)
    if dlogits is None:
        dlogits = torch.empty(shape, dtype=dt, device=dev)
    ldd = _rows("dlogits", dlogits, dt, shape, dev)
    _call("token_logprobs_bwd", lib.token_logprobs_bwd, dev, logits.data_ptr(), ld,
          _addr(targets), _addr(lse), _addr(entropy), _addr(dlogprob), _addr(dentropy),
          dlogits.data_ptr(), ldd, R, V, temperature, ignore_index, code)
    return dlogits


def _teacher(top, top_ids, R, dev):
    """Checks the teacher's entries [R, k]; returns k and the code of their type."""
    _, k = _matrix("top", top)
    _packed("top", top, top.dtype, (R, k), dev)
    _packed("top_ids", top_ids, torch.int64, (R, k), dev)
    return k, _dtype_code(top)


def distill_workspace_size(R: int, V: int, k: int, dtype) -> int:
    return int(load_library().distill_workspace_size(R, V, k, DTYPE_CODE[dtype]))


def _loss_and_lse(loss, lse, R, dev):
    loss = _out("loss", loss, torch.float32, (R,), dev)
    lse = torch.empty_like(loss) if lse is None else _out("lse", lse, torch.float32, (R,), dev)
    return loss, lse


def distill_fwd(logits, top, top_ids, temperature=1.0, loss=None, lse=None, workspace=None,
                stream=None):
    """Distillation loss of logits [R, V] against a teacher's entries: values ``top`` [R, k]
    (logits or log probabilities, bf16, fp16 or fp32) at ``top_ids`` [R, k] (int64; ids
    outside [0, V) are padding).  Returns the fp32 loss [R] (T^2 times the divergence from
    the teacher's renormalised distribution) and the lse [R] ``distill_bwd`` takes."""
    if stream is not None:
        with _on_stream(stream, logits):
            return distill_fwd(logits, top, top_ids, temperature, loss, lse, workspace)
    lib = load_library()
    shape = _matrix("logits", logits)
    R, V = shape
    dt, dev = logits.dtype, logits.device
    code = _dtype_code(logits)
    ld = _rows("logits", logits, dt, shape, dev)
    k, top_code = _teacher(top, top_ids, R, dev)
    _gpu(dev)
    loss, lse = _loss_and_lse(loss, lse, R, dev)
    ws = _workspace(_workspace_bytes("distill_workspace_size", R, V, k, code), workspace, dev, None)
    _call("distill_fwd", lib.distill_fwd, dev, logits.data_ptr(), ld, top.data_ptr(),
          top_ids.data_ptr(), k, loss.data_ptr(), lse.data_ptr(), R, V, temperature, code,
          top_code, _addr(ws), _size(ws))
    return loss, lse


def distill_bwd(logits, top, top_ids, lse, dloss, dlogits=None, temperature=1.0, stream=None):
    """Gradient of ``distill_fwd``'s loss with respect to the logits, from dloss [R] (fp32; 0
    for a masked row).  ``dlogits`` [R, V] may be ``logits`` itself; it is returned."""
    if stream is not None:
        with _on_stream(stream, logits):
            return distill_bwd(logits, top, top_ids, lse, dloss, dlogits, temperature)
    lib = load_library()
    shape = _matrix("logits", logits)
    R, V = shape
    dt, dev = logits.dtype, logits.device
    code = _dtype_code(logits)
    ld = _rows("logits", logits, dt, shape, dev)
    k, top_code = _teacher(top, top_ids, R, dev)
    lse_at = _packed("lse", lse, torch.float32, (R,), dev)
    dloss_at = _packed("dloss", dloss, torch.float32, (R,), dev)
    _gpu(dev)
    if dlogits is None:
        dlogits = torch.empty(shape, dtype=dt, device=dev)
    ldd = _rows("dlogits", dlogits, dt, shape, dev)
    _call("distill_bwd", lib.distill_bwd, dev, logits.data_ptr(), ld, top.data_ptr(),
          top_ids.data_ptr(), k, lse_at, dloss_at, dlogits.data_ptr(), ldd, R, V, temperature,
          code, top_code)
    return dlogits


def distill_fwd_bwd(logits, top, top_ids, dloss, dlogits=None, temperature=1.0, loss=None,
                    lse=None, workspace=None, stream=None):
    """``distill_fwd`` and ``distill_bwd`` in one call, for a training step that knows the row
    weights ``dloss`` [R] beforehand.  ``dlogits`` may be ``logits`` itself.  Returns
    (loss, lse, dlogits)."""
    if stream is not None:
        with _on_stream(stream, logits):
            return distill_fwd_bwd(logits, top, top_ids, dloss, dlogits, temperature, loss, lse,
                                   workspace)
    lib = load_library()
    shape = _matrix("logits", logits)
    R, V = shape
    dt, dev = logits.dtype, logits.device
    code = _dtype_code(logits)
    ld = _rows("logits", logits, dt, shape, dev)
    k, top_code = _teacher(top, top_ids, R, dev)
    dloss_at = _packed("dloss", dloss, torch.float32, (R,), dev)
    _gpu(dev)
    loss, lse = _loss_and_lse(loss, lse, R, dev)
    if dlogits is None:
        dlogits = torch.empty(shape, dtype=dt, device=dev)
    ldd = _rows("dlogits", dlogits, dt, shape, dev)
    ws = _workspace(_workspace_bytes("distill_workspace_size", R, V, k, code), workspace, dev, None)
    _call("distill_fwd_bwd", lib.distill_fwd_bwd, dev, logits.data_ptr(), ld,
          top.data_ptr(), top_ids.data_ptr(), k, dloss_at, loss.data_ptr(), lse.data_ptr(),
          dlogits.data_ptr(), ldd, R, V, temperature, code, top_code, _addr(ws), _size(ws))
    return loss, lse, dlogits
