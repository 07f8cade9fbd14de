"""ctypes binding of the C ABI in include/fp8blk.h (argument marshalling only).
The operators whose smallest calls last as long as their marshalling have it
compiled as well (csrc/host.cpp), for plain calls on the current stream.

Every function here has the name of the C entry point it calls.  Tensors are
torch CUDA tensors; outputs the caller does not pass are allocated with torch
(device memory only: the library itself never allocates), from the pool of the
stream the call runs on.  A non-zero status
raises Fp8Error.  The library must have been built (``python -m
blockwise_fp8_pretraining_b200.build``); there is no fallback.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import re
import warnings

import torch

from . import build as _build

ROWWISE, COLWISE, BOTH = 1, 2, 3
MAX_CONTRACTION_FPROP = 32768
GEMM_SPLIT_MIN_WORK_DEFAULT = 160      # FP8_GEMM_SPLIT_MIN_WORK_DEFAULT
MAX_NORM_COLS = 16384                  # FP8_MAX_NORM_COLS
MAX_TOPK = 32                          # FP8_MAX_TOPK
# The coefficients (a, b, c) of the steps published with the Muon optimiser.
NEWTON_SCHULZ_COEFFICIENTS = ((3.4445, -4.7750, 2.0315),) * 5

_lib = None
_host = None                           # the compiled host side, where it was built for this torch


class Fp8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        msg = f"{where}: {status_string(status)} (status {status})"
        if status == 5:
            msg += f": {fp8_last_cuda_error()}"
        super().__init__(msg)


def lib_path() -> str:
    return _build.LIB


def header_functions() -> list[str]:
    """Names of the functions include/fp8blk.h declares."""
    with open(_build.HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(fp8_\w+)\s*\(", text, flags=re.M)


def load() -> ctypes.CDLL:
    """Load libfp8blk.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise OSError(f"{path} is missing: build it with python -m blockwise_fp8_pretraining_b200.build")
    lib = ctypes.CDLL(path)
    p, i64, i32, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int
    sz = ctypes.c_size_t
    sig = {
        "fp8_quantize_act_1x128": [p, i64, i64, i32, p, p, p, p, p],
        "fp8_quantize_weight_128x128": [p, i64, i64, p, p, p, p],
        "fp8_swiglu_quantize_1x128": [p, i64, i64, i32, p, p, p, p, p],
        "fp8_rmsnorm_rstd": [p, i64, i64, ctypes.c_float, p, p],
        "fp8_rmsnorm_quantize_1x128": [p, i64, i64, p, p, i32, p, p, p, p, p],
        "fp8_add_rmsnorm_quantize_1x128": [p, p, i64, i64, ctypes.c_float, p, i32, p, p, p, p, p, p, p],
        "fp8_rmsnorm_backward": [p, p, p, p, p, i64, i64, p, p, i32, p, sz, p],
        "fp8_rmsnorm_backward_workspace_bytes": [i64, i64, p],
        "fp8_token_logprobs": [p, i32, i64, i64, i64, p, i32, p, p, p, p, p, p],
        "fp8_token_logprobs_backward": [p, i32, i64, i64, i64, p, p, p, p, p, p, i64, p],
        "fp8_newton_schulz": [p, i32, i64, i64, i64, p, i32, ctypes.c_float, p, p, sz, p],
        "fp8_newton_schulz_workspace_bytes": [i64, i64, i64, p],
        "fp8_selftest_silu_bf16": [p, p],
        "fp8_block_gemm_fprop": [p, p, p, p, p, i64, i64, i64, p, sz, p],
        "fp8_block_gemm_dgrad": [p, p, p, p, p, i64, i64, i64, p, sz, p],
        "fp8_block_gemm_wgrad": [p, p, p, p, p, i64, i64, i64, p, sz, p],
        "fp8_block_gemm_wgrad_accum_f32": [p, p, p, p, p, i64, i64, i64, p, sz, p],
        "fp8_block_gemm_wgrad_reduce_scatter_f32": [p, p, p, p, p, i32, i64, i64, i64, p, sz, p],
        "fp8_gemm_workspace_bytes": [p],
        "fp8_block_gemm_wgrad_static_ws": [p, p, p, p, p, i64, i64, i64, p],
        "fp8_get_error": [],
        "fp8_clear_error": [],
        "fp8_set_wait_timeout_ns": [ctypes.c_uint64],
        "fp8_set_gemm_split_min_work": [ctypes.c_int64],
        "fp8_cast_e4m3_scaled": [p, ctypes.c_float, p, i64, p],
        "fp8_selftest_wait_timeout": [p],
        "fp8_selftest_stall_next": [i32],
        "fp8_selftest_gemm_schedule": [i64, i64, i64, i32, i32, p, i64, p],
        "fp8_selftest_division": [p, p],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = st
    lib.fp8_status_string.argtypes = [st]
    lib.fp8_status_string.restype = ctypes.c_char_p
    lib.fp8_last_cuda_error.argtypes = []
    lib.fp8_last_cuda_error.restype = ctypes.c_char_p
    _load_host(lib)
    _lib = lib
    return lib


def _load_host(lib) -> None:
    """The compiled host side, if it is there and fits the running torch."""
    global _host
    if not os.path.exists(_build.HOST_LIB):
        return
    loader = importlib.machinery.ExtensionFileLoader("_fp8blk_host", _build.HOST_LIB)
    try:
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_fp8blk_host", loader))
        loader.exec_module(module)
    except ImportError as e:
        warnings.warn(f"the binding's compiled host side does not load, its Python one serves: {e}", RuntimeWarning)
        return
    module.bind(*(ctypes.cast(fn, ctypes.c_void_p).value for fn in (
        lib.fp8_add_rmsnorm_quantize_1x128, lib.fp8_rmsnorm_backward, lib.fp8_rmsnorm_backward_workspace_bytes,
        lib.fp8_token_logprobs, lib.fp8_token_logprobs_backward)))
    _host = module


def _plain(function: str, where: str, *args):
    """The compiled host side's result, or None where the call is not plain
    (see csrc/host.cpp) and goes through the checks below."""
    out = getattr(_host, function)(*args)
    if type(out) is int:
        raise Fp8Error(out, where)
    return out


def status_string(status: int) -> str:
    try:
        return load().fp8_status_string(int(status)).decode()
    except OSError:
        return "library not loaded"


def _check(status: int, where: str):
    if status != 0:
        raise Fp8Error(status, where)


def _stream(stream) -> int:
    if stream is None:                 # the handle alone: a torch Stream object costs a microsecond
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check_devices(named, current: int, stream=None) -> None:
    """The library launches on the current CUDA device, so every tensor (and
    an explicit torch stream) must live there; a pointer into another GPU's
    memory would be dereferenced by the wrong device."""
    for name, t in named:
        if t is not None and t.device.index != current:
            raise ValueError(f"{name} is on {t.device} but the current CUDA device is cuda:{current}; "
                             f"call inside torch.cuda.device({t.device.index})")
    if isinstance(stream, torch.cuda.Stream) and stream.device.index != current:
        raise ValueError(f"stream is on {stream.device} but the current CUDA device is cuda:{current}")


def _launch_checks(named, stream) -> None:
    _check_devices(named, torch.cuda.current_device(), stream)


def _elsewhere(function, stream, *args, **kwargs):
    """function(*args, **kwargs) with `stream` (a torch stream, or a handle on the
    current device) as the current one.

    What the call allocates then comes from that stream's pool, where whatever
    used the memory before is ordered ahead of the kernel; memory freed on the
    caller's stream may have work of that stream on it that is still to run.  New
    outputs are also tied to the caller's stream, which will read them: when they
    are freed, they are not reused before what is queued there has run."""
    dev = torch.cuda.current_device()
    launch = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=dev)
    _check_devices((), dev, launch)
    caller = torch.cuda.current_stream()
    if caller.cuda_stream == launch.cuda_stream:
        return function(*args, **kwargs)
    torch.cuda.set_stream(launch)
    try:
        out = function(*args, **kwargs)
    finally:
        torch.cuda.set_stream(caller)
    for t in out if isinstance(out, tuple) else (out,):
        if isinstance(t, torch.Tensor) and not any(t is given for given in args):
            t.record_stream(caller)
    return out


def _ptr(t: torch.Tensor | None) -> int:
    return 0 if t is None else t.data_ptr()


def _want(t: torch.Tensor, dtype, shape, name):
    if t.is_cuda and t.dtype == dtype and t.shape == shape and t.is_contiguous():
        return t
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _out(t, dtype, shape, device, name):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _want(t, dtype, shape, name)


# ------------------------------------------------------------------ kernels

def fp8_quantize_act_1x128(x, mode=BOTH, q_row=None, s_row=None, q_colT=None, s_col=None,
                           stream=None):
    """Quantize a bf16 activation [rows, cols].  Returns (q_row, s_row,
    q_colT, s_col); entries of a grouping the mode leaves out are None."""
    if stream is not None:
        return _elsewhere(fp8_quantize_act_1x128, stream, x, mode, q_row, s_row, q_colT, s_col)
    lib = load()
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise TypeError("x must be a 2-D bfloat16 tensor")
    rows, cols = x.shape
    _want(x, torch.bfloat16, (rows, cols), "x")
    dev = x.device
    if mode & ROWWISE:
        q_row = _out(q_row, torch.uint8, (rows, cols), dev, "q_row")
        s_row = _out(s_row, torch.float32, (cols // 128, rows), dev, "s_row")
    else:
        q_row = s_row = None
    if mode & COLWISE:
        q_colT = _out(q_colT, torch.uint8, (cols, rows), dev, "q_colT")
        s_col = _out(s_col, torch.float32, (rows // 128, cols), dev, "s_col")
    else:
        q_colT = s_col = None
    _launch_checks([("x", x), ("q_row", q_row), ("s_row", s_row), ("q_colT", q_colT), ("s_col", s_col)],
                   stream)
    _check(lib.fp8_quantize_act_1x128(_ptr(x), rows, cols, int(mode), _ptr(q_row), _ptr(s_row),
                                      _ptr(q_colT), _ptr(s_col), _stream(stream)),
           "fp8_quantize_act_1x128")
    return q_row, s_row, q_colT, s_col


def fp8_swiglu_quantize_1x128(gate_up, mode=BOTH, q_row=None, s_row=None, q_colT=None, s_col=None,
                              stream=None):
    """Quantize H = silu(gate) * up (bf16 roundings as the unfused path) of
    a bf16 gate_up activation [rows, 2 * ffn] without forming H in memory.
    Returns (q_row, s_row, q_colT, s_col) of H [rows, ffn]; entries of a
    grouping the mode leaves out are None."""
    if stream is not None:
        return _elsewhere(fp8_swiglu_quantize_1x128, stream, gate_up, mode, q_row, s_row, q_colT, s_col)
    lib = load()
    if gate_up.dtype != torch.bfloat16 or gate_up.dim() != 2 or gate_up.shape[1] % 2:
        raise TypeError("gate_up must be a 2-D bfloat16 tensor with an even number of columns")
    rows, cols2 = gate_up.shape
    ffn = cols2 // 2
    _want(gate_up, torch.bfloat16, (rows, cols2), "gate_up")
    dev = gate_up.device
    if mode & ROWWISE:
        q_row = _out(q_row, torch.uint8, (rows, ffn), dev, "q_row")
        s_row = _out(s_row, torch.float32, (ffn // 128, rows), dev, "s_row")
    else:
        q_row = s_row = None
    if mode & COLWISE:
        q_colT = _out(q_colT, torch.uint8, (ffn, rows), dev, "q_colT")
        s_col = _out(s_col, torch.float32, (rows // 128, ffn), dev, "s_col")
    else:
        q_colT = s_col = None
    outs = (q_row, s_row, q_colT, s_col)
    _launch_checks([("gate_up", gate_up), ("q_row", q_row), ("s_row", s_row), ("q_colT", q_colT),
                    ("s_col", s_col)], stream)
    _check(lib.fp8_swiglu_quantize_1x128(_ptr(gate_up), rows, ffn, int(mode), _ptr(q_row), _ptr(s_row),
                                         _ptr(q_colT), _ptr(s_col), _stream(stream)),
           "fp8_swiglu_quantize_1x128")
    return outs


def fp8_rmsnorm_rstd(x, eps=1e-6, rstd=None, stream=None):
    """RMSNorm's rstd[i] = 1 / sqrt(mean(x[i]^2) + eps) (float32 [rows]) of a
    bf16 x [rows, cols]."""
    if stream is not None and rstd is None:
        return _elsewhere(fp8_rmsnorm_rstd, stream, x, eps, rstd)
    lib = load()
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise TypeError("x must be a 2-D bfloat16 tensor")
    rows, cols = x.shape
    _want(x, torch.bfloat16, (rows, cols), "x")
    rstd = _out(rstd, torch.float32, (rows,), x.device, "rstd")
    _launch_checks([("x", x), ("rstd", rstd)], stream)
    _check(lib.fp8_rmsnorm_rstd(_ptr(x), rows, cols, float(eps), _ptr(rstd), _stream(stream)), "fp8_rmsnorm_rstd")
    return rstd


def fp8_rmsnorm_quantize_1x128(x, rstd, gamma, mode=BOTH, q_row=None, s_row=None, q_colT=None, s_col=None,
                               stream=None):
    """Quantize y = bf16(gamma * bf16(x * rstd)) (RMSNorm's output; rstd
    float32 [rows], gamma bf16 [cols]) of a bf16 x [rows, cols] without
    forming y in memory.  Returns (q_row, s_row, q_colT, s_col) of y;
    entries of a grouping the mode leaves out are None."""
    if stream is not None:
        return _elsewhere(fp8_rmsnorm_quantize_1x128, stream, x, rstd, gamma, mode, q_row, s_row, q_colT, s_col)
    lib = load()
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise TypeError("x must be a 2-D bfloat16 tensor")
    rows, cols = x.shape
    _want(x, torch.bfloat16, (rows, cols), "x")
    _want(rstd, torch.float32, (rows,), "rstd")
    _want(gamma, torch.bfloat16, (cols,), "gamma")
    dev = x.device
    if mode & ROWWISE:
        q_row = _out(q_row, torch.uint8, (rows, cols), dev, "q_row")
        s_row = _out(s_row, torch.float32, (cols // 128, rows), dev, "s_row")
    else:
        q_row = s_row = None
    if mode & COLWISE:
        q_colT = _out(q_colT, torch.uint8, (cols, rows), dev, "q_colT")
        s_col = _out(s_col, torch.float32, (rows // 128, cols), dev, "s_col")
    else:
        q_colT = s_col = None
    outs = (q_row, s_row, q_colT, s_col)
    _launch_checks([("x", x), ("rstd", rstd), ("gamma", gamma), ("q_row", q_row), ("s_row", s_row),
                    ("q_colT", q_colT), ("s_col", s_col)], stream)
    _check(lib.fp8_rmsnorm_quantize_1x128(_ptr(x), rows, cols, _ptr(rstd), _ptr(gamma), int(mode), _ptr(q_row),
                                          _ptr(s_row), _ptr(q_colT), _ptr(s_col), _stream(stream)),
           "fp8_rmsnorm_quantize_1x128")
    return outs


# The operators around the linears.  Their smallest calls take as long as the
# host does, so a tensor is checked (device included) in one go, tensors made here
# are not checked, and the messages are left to the checks above.

def _on(t, dtype, shape, dev, name):
    if t.get_device() == dev and t.dtype == dtype and t.shape == shape and t.is_contiguous():
        return t
    _want(t, dtype, shape, name)
    _check_devices([(name, t)], dev)
    return t


def _given(t, dtype, shape, like, dev, name):
    """t checked, or a new tensor (by the cheapest call)."""
    if t is not None:
        return _on(t, dtype, shape, dev, name)
    if like.shape == shape and like.is_contiguous():
        return torch.empty_like(like) if like.dtype == dtype else torch.empty_like(like, dtype=dtype)
    return like.new_empty(shape) if like.dtype == dtype else like.new_empty(shape, dtype=dtype)


def _aligned(t):
    """t, or a copy on the current stream where t (a slice of a longer tensor) does
    not begin at a multiple of 16 bytes, as the library has it."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.clone()


def _aside(outputs):
    """Where the library may write the outputs: themselves, or a new tensor in the
    place of one that does not begin at a multiple of 16 bytes."""
    return [t if t is None or t.data_ptr() % 16 == 0 else torch.empty_like(t) for t in outputs]


def _bring(outputs, written):
    for t, w in zip(outputs, written):
        if w is not t:
            t.copy_(w)


def _current(dev):
    """The current stream's handle, once the tensors' device is known to be current."""
    if dev != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{dev} but the current CUDA device is "
                         f"cuda:{torch.cuda.current_device()}; call inside torch.cuda.device({dev})")
    return torch._C._cuda_getCurrentRawStream(dev)


def _scratch(workspace, bytes_, like, dev):
    """The workspace, allocated when left out, and its bytes."""
    if workspace is None:
        workspace = like.new_empty((bytes_(),), dtype=torch.uint8)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        _check_devices([("workspace", workspace)], dev)
    return workspace, workspace.numel() * workspace.element_size()


def fp8_add_rmsnorm_quantize_1x128(x, gamma, residual=None, eps=1e-6, mode=BOTH, sum_out=None, rstd=None, q_row=None,
                                   s_row=None, q_colT=None, s_col=None, stream=None):
    """s = bf16(x + residual) (s = x without a residual), RMSNorm of s with
    the weight gamma, and its output quantized.  Returns (s, rstd, q_row,
    s_row, q_colT, s_col); entries of a grouping the mode leaves out are None,
    and s is x itself without a residual.  sum_out may be x or residual (in
    place)."""
    if stream is not None:
        return _elsewhere(fp8_add_rmsnorm_quantize_1x128, stream, x, gamma, residual, eps, mode, sum_out, rstd,
                          q_row, s_row, q_colT, s_col)
    lib = _lib or load()
    if _host is not None:
        out = _plain("add_rmsnorm_quantize", "fp8_add_rmsnorm_quantize_1x128", x, gamma, residual, eps, mode, sum_out, rstd,
                     q_row, s_row, q_colT, s_col)
        if out is not None:
            return out
    bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    if x.dtype != bf16 or x.dim() != 2:
        raise TypeError("x must be a 2-D bfloat16 tensor")
    shape = x.shape
    rows, cols = shape
    dev = x.get_device()
    _on(x, bf16, shape, dev if dev >= 0 else None, "x")
    _on(gamma, bf16, (cols,), dev, "gamma")
    if residual is not None:
        _on(residual, bf16, shape, dev, "residual")
        sum_out = _given(sum_out, bf16, shape, x, dev, "sum_out")
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual: without one the sum is x itself")
    rstd = _given(rstd, f32, (rows,), x, dev, "rstd")
    if mode & ROWWISE:
        q_row = _given(q_row, u8, shape, x, dev, "q_row")
        s_row = _given(s_row, f32, (cols // 128, rows), rstd, dev, "s_row")
    else:
        q_row = s_row = None
    if mode & COLWISE:
        q_colT = _given(q_colT, u8, (cols, rows), x, dev, "q_colT")
        s_col = _given(s_col, f32, (rows // 128, cols), rstd, dev, "s_col")
    else:
        q_colT = s_col = None
    handle = _current(dev)
    st = lib.fp8_add_rmsnorm_quantize_1x128(x.data_ptr(), _ptr(residual), rows, cols, float(eps), gamma.data_ptr(),
                                            int(mode), _ptr(sum_out), rstd.data_ptr(), _ptr(q_row), _ptr(s_row), _ptr(q_colT),
                                            _ptr(s_col), handle)
    if st:
        raise Fp8Error(st, "fp8_add_rmsnorm_quantize_1x128")
    return (x if residual is None else sum_out), rstd, q_row, s_row, q_colT, s_col


def fp8_rmsnorm_backward_workspace_bytes(rows: int, cols: int) -> int:
    """Bytes of scratch fp8_rmsnorm_backward needs on the current device for
    the gradient of the norm weight (0: none)."""
    n = ctypes.c_size_t(0)
    _check(load().fp8_rmsnorm_backward_workspace_bytes(int(rows), int(cols), ctypes.byref(n)),
           "fp8_rmsnorm_backward_workspace_bytes")
    return int(n.value)


def fp8_rmsnorm_backward(dy, s, rstd, gamma, dresidual=None, ds=None, dgamma=None, accumulate=False, workspace=None,
                         stream=None):
    """Gradient through RMSNorm: (ds, dgamma) from dy (the gradient of the
    norm's output), the norm's input s, its rstd and weight, plus the
    residual path's gradient of s if there is one.  ds (bf16) may be dy or
    dresidual (in place); dgamma is float32 [cols], added to with
    accumulate=True (it must then be given)."""
    if stream is not None:
        return _elsewhere(fp8_rmsnorm_backward, stream, dy, s, rstd, gamma, dresidual, ds, dgamma, accumulate, workspace)
    lib = _lib or load()
    if _host is not None:
        out = _plain("rmsnorm_backward", "fp8_rmsnorm_backward", dy, s, rstd, gamma, dresidual, ds, dgamma, accumulate,
                     workspace)
        if out is not None:
            return out
    bf16, f32 = torch.bfloat16, torch.float32
    if s.dtype != bf16 or s.dim() != 2:
        raise TypeError("s must be a 2-D bfloat16 tensor")
    shape = s.shape
    rows, cols = shape
    dev = s.get_device()
    _on(s, bf16, shape, dev if dev >= 0 else None, "s")
    _on(dy, bf16, shape, dev, "dy")
    rstd = _aligned(_on(rstd, f32, (rows,), dev, "rstd"))
    _on(gamma, bf16, (cols,), dev, "gamma")
    if dresidual is not None:
        _on(dresidual, bf16, shape, dev, "dresidual")
    if accumulate and dgamma is None:
        raise ValueError("accumulate=True needs the dgamma to add to")
    ds = _given(ds, bf16, shape, s, dev, "ds")
    dgamma = _given(dgamma, f32, (cols,), rstd, dev, "dgamma")
    workspace, size = _scratch(workspace, lambda: fp8_rmsnorm_backward_workspace_bytes(rows, cols), s, dev)
    handle = _current(dev)
    st = lib.fp8_rmsnorm_backward(dy.data_ptr(), s.data_ptr(), rstd.data_ptr(), gamma.data_ptr(), _ptr(dresidual), rows,
                                  cols, ds.data_ptr(), dgamma.data_ptr(), 1 if accumulate else 0,
                                  workspace.data_ptr(), size, handle)
    if st:
        raise Fp8Error(st, "fp8_rmsnorm_backward")
    return ds, dgamma


_DTYPES = {torch.bfloat16: 0, torch.float32: 1}      # FP8_BF16, FP8_F32


def _logits(t, name, like=None):
    """(dtype code, row stride) of a 2-D bf16 or float32 CUDA tensor whose
    rows are contiguous (a view into a padded vocabulary will do)."""
    code = _DTYPES.get(t.dtype)
    if code is None or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D bfloat16 or float32 tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is not None and (t.dtype != like.dtype or t.shape != like.shape):
        raise ValueError(f"{name}: expected {like.dtype} {tuple(like.shape)}, got {t.dtype} {tuple(t.shape)}")
    rows, vocab = t.shape
    ld, one = t.stride()
    if rows <= 1:
        ld = max(vocab, ld)
    if (vocab > 1 and one != 1) or ld < vocab:
        raise ValueError(f"{name}: rows must be contiguous and must not overlap")
    return code, ld


def fp8_token_logprobs(logits, targets=None, topk=0, logprob=None, entropy=None, stats=None, top_logprob=None,
                       top_index=None, stream=None):
    """Log probability of each row's target token (int64 [rows]; negative:
    none), the entropy of each row's distribution, stats [rows, 2] (the row's
    maximum m and log sum exp(x - m)), and the topk most likely tokens (log
    probabilities and int64 indices [rows, topk], largest first, equal logits
    by index) of bf16 or float32 logits [rows, vocab].  Returns (logprob,
    entropy, stats, top_logprob, top_index); logprob is None without targets,
    the last two with topk = 0.  Per-row arguments may be slices of longer tensors
    (one that does not begin at a multiple of 16 bytes is copied)."""
    if stream is not None:
        return _elsewhere(fp8_token_logprobs, stream, logits, targets, topk, logprob, entropy, stats, top_logprob,
                          top_index)
    lib = _lib or load()
    if _host is not None:
        out = _plain("token_logprobs", "fp8_token_logprobs", logits, targets, topk, logprob, entropy, stats, top_logprob,
                     top_index)
        if out is not None:
            return out
    f32, i64 = torch.float32, torch.int64
    code, ld = _logits(logits, "logits")
    rows, vocab = logits.shape
    dev = logits.get_device()
    entropy = _given(entropy, f32, (rows,), logits, dev, "entropy")
    if targets is not None:
        targets = _aligned(_on(targets, i64, (rows,), dev, "targets"))
        logprob = _given(logprob, f32, (rows,), entropy, dev, "logprob")
    else:
        logprob = None
    stats = _given(stats, f32, (rows, 2), entropy, dev, "stats")
    if topk > 0:
        top_logprob = _given(top_logprob, f32, (rows, topk), entropy, dev, "top_logprob")
        top_index = _given(top_index, i64, (rows, topk), top_logprob, dev, "top_index")
    else:
        top_logprob = top_index = None
    handle = _current(dev)
    out = (logprob, entropy, stats, top_logprob, top_index)
    written = _aside(out)
    st = lib.fp8_token_logprobs(logits.data_ptr(), code, rows, vocab, ld, _ptr(targets), int(topk), *map(_ptr, written),
                                handle)
    if st:
        raise Fp8Error(st, "fp8_token_logprobs")
    _bring(out, written)
    return out


def fp8_token_logprobs_backward(logits, targets, stats, dlogprob=None, entropy=None, dentropy=None, dlogits=None,
                                stream=None):
    """Gradient of the logits from the gradients of fp8_token_logprobs's
    logprob and entropy (float32 [rows], either None); entropy is needed with
    dentropy.  dlogits (the logits' type) may be the logits themselves.  Per-row
    arguments may be slices, as in fp8_token_logprobs."""
    if stream is not None:
        return _elsewhere(fp8_token_logprobs_backward, stream, logits, targets, stats, dlogprob, entropy, dentropy,
                          dlogits)
    lib = _lib or load()
    if _host is not None:
        out = _plain("token_logprobs_backward", "fp8_token_logprobs_backward", logits, targets, stats, dlogprob, entropy,
                     dentropy, dlogits)
        if out is not None:
            return out
    f32 = torch.float32
    code, ld = _logits(logits, "logits")
    rows, vocab = logits.shape
    dev = logits.get_device()
    stats = _aligned(_on(stats, f32, (rows, 2), dev, "stats"))
    if dlogprob is not None:
        if targets is None:
            raise ValueError("dlogprob needs targets")
        dlogprob = _aligned(_on(dlogprob, f32, (rows,), dev, "dlogprob"))
    if targets is not None:
        targets = _aligned(_on(targets, torch.int64, (rows,), dev, "targets"))
    if dentropy is not None:
        if entropy is None:
            raise ValueError("dentropy needs the entropy")
        dentropy = _aligned(_on(dentropy, f32, (rows,), dev, "dentropy"))
        entropy = _aligned(_on(entropy, f32, (rows,), dev, "entropy"))
    if dlogits is None:
        dlogits = _given(None, logits.dtype, (rows, vocab), logits, dev, "dlogits")
        ld_out = vocab
    else:
        _, ld_out = _logits(dlogits, "dlogits", logits)
        _check_devices([("dlogits", dlogits)], dev)
    handle = _current(dev)
    st = lib.fp8_token_logprobs_backward(logits.data_ptr(), code, rows, vocab, ld, _ptr(targets), stats.data_ptr(),
                                         _ptr(dlogprob), _ptr(entropy), _ptr(dentropy), dlogits.data_ptr(), ld_out,
                                         handle)
    if st:
        raise Fp8Error(st, "fp8_token_logprobs_backward")
    return dlogits


def fp8_newton_schulz_workspace_bytes(batch: int, m: int, n: int) -> int:
    """Bytes of scratch fp8_newton_schulz needs for [batch, m, n]."""
    k = ctypes.c_size_t(0)
    _check(load().fp8_newton_schulz_workspace_bytes(int(batch), int(m), int(n), ctypes.byref(k)),
           "fp8_newton_schulz_workspace_bytes")
    return int(k.value)


def fp8_newton_schulz(g, coefficients=NEWTON_SCHULZ_COEFFICIENTS, eps=1e-7, out=None, workspace=None, stream=None):
    """Newton-Schulz orthogonalisation of each matrix of g ([m, n] or
    [batch, m, n], bf16 or float32), one step per (a, b, c) of coefficients.
    Returns a bf16 tensor of g's shape.  workspace: optional uint8 scratch of
    fp8_newton_schulz_workspace_bytes (allocated when left out)."""
    if stream is not None:
        return _elsewhere(fp8_newton_schulz, stream, g, coefficients, eps, out, workspace)
    lib = _lib or load()
    if g.dim() not in (2, 3) or g.dtype not in _DTYPES:
        raise TypeError("g must be a 2-D or 3-D bfloat16 or float32 tensor")
    shape = g.shape
    dev = g.get_device()
    _on(g, g.dtype, shape, dev if dev >= 0 else None, "g")
    batch, m, n = shape if g.dim() == 3 else (1, *shape)
    steps = len(coefficients)
    if any(len(step) != 3 for step in coefficients):
        raise ValueError("each step takes three coefficients")
    table = (ctypes.c_float * (3 * steps))(*[float(v) for step in coefficients for v in step])
    g = _aligned(g)
    out = _given(out, torch.bfloat16, shape, g, dev, "out")
    written, = _aside((out,))
    workspace, size = _scratch(workspace, lambda: fp8_newton_schulz_workspace_bytes(batch, m, n), g, dev)
    handle = _current(dev)
    _check(lib.fp8_newton_schulz(g.data_ptr(), _DTYPES[g.dtype], batch, m, n, ctypes.cast(table, ctypes.c_void_p),
                                 steps, float(eps), written.data_ptr(), workspace.data_ptr(), size, handle),
           "fp8_newton_schulz")
    _bring((out,), (written,))
    return out


def fp8_quantize_weight_128x128(w, wq=None, sw=None, wqT=None, transposed=True, stream=None):
    """Quantize a bf16 weight [n, k] in 128x128 blocks.  Returns (wq, sw, wqT);
    wqT is None when transposed is False and no buffer is passed."""
    if stream is not None:
        return _elsewhere(fp8_quantize_weight_128x128, stream, w, wq, sw, wqT, transposed)
    lib = load()
    if w.dtype != torch.bfloat16 or w.dim() != 2:
        raise TypeError("w must be a 2-D bfloat16 tensor")
    n, k = w.shape
    _want(w, torch.bfloat16, (n, k), "w")
    wq = _out(wq, torch.uint8, (n, k), w.device, "wq")
    sw = _out(sw, torch.float32, (n // 128, k // 128), w.device, "sw")
    if wqT is not None or transposed:
        wqT = _out(wqT, torch.uint8, (k, n), w.device, "wqT")
    _launch_checks([("w", w), ("wq", wq), ("sw", sw), ("wqT", wqT)], stream)
    _check(lib.fp8_quantize_weight_128x128(_ptr(w), n, k, _ptr(wq), _ptr(sw), _ptr(wqT),
                                           _stream(stream)),
           "fp8_quantize_weight_128x128")
    return wq, sw, wqT


def _workspace(ws):
    """(pointer, bytes) of an optional GEMM workspace tensor (see
    fp8_gemm_workspace_bytes): contiguous, on the current device, zeroed
    before its first use."""
    if ws is None:
        return ctypes.c_void_p(0), 0
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size()


def fp8_gemm_workspace_bytes() -> int:
    """Bytes of the GEMM workspace on the current device."""
    n = ctypes.c_size_t(0)
    _check(load().fp8_gemm_workspace_bytes(ctypes.byref(n)), "fp8_gemm_workspace_bytes")
    return int(n.value)


def fp8_gemm_workspace(device=None) -> torch.Tensor:
    """A zeroed GEMM workspace for the current (or given) device, allocated
    by torch.  One launch at a time may use it."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        return torch.zeros(fp8_gemm_workspace_bytes(), dtype=torch.uint8, device=dev)


def fp8_block_gemm_fprop(xq, sx, wq, sw, y=None, stream=None, workspace=None):
    """Y[M, N] = X W^T (bf16) from X codes [M, K] / scales [K/128, M] and W
    codes [N, K] / scales [N/128, K/128].  workspace: optional (see
    fp8_gemm_workspace)."""
    if stream is not None and y is None:
        return _elsewhere(fp8_block_gemm_fprop, stream, xq, sx, wq, sw, y, workspace=workspace)
    lib = load()
    M, K = xq.shape
    N = wq.shape[0]
    _want(xq, torch.uint8, (M, K), "xq")
    _want(sx, torch.float32, (K // 128, M), "sx")
    _want(wq, torch.uint8, (N, K), "wq")
    _want(sw, torch.float32, (N // 128, K // 128), "sw")
    y = _out(y, torch.bfloat16, (M, N), xq.device, "y")
    _launch_checks([("xq", xq), ("sx", sx), ("wq", wq), ("sw", sw), ("y", y), ("workspace", workspace)],
                   stream)
    _check(lib.fp8_block_gemm_fprop(_ptr(xq), _ptr(sx), _ptr(wq), _ptr(sw), _ptr(y), M, N, K,
                                    *_workspace(workspace), _stream(stream)),
           "fp8_block_gemm_fprop")
    return y


def fp8_block_gemm_dgrad(dyq, sdy, wqT, sw, dx=None, stream=None, workspace=None):
    """dX[M, K] = dY W (bf16) from dY codes [M, N] / scales [N/128, M], the
    transposed weight codes [K, N] and the weight scales [N/128, K/128]."""
    if stream is not None and dx is None:
        return _elsewhere(fp8_block_gemm_dgrad, stream, dyq, sdy, wqT, sw, dx, workspace=workspace)
    lib = load()
    M, N = dyq.shape
    K = wqT.shape[0]
    _want(dyq, torch.uint8, (M, N), "dyq")
    _want(sdy, torch.float32, (N // 128, M), "sdy")
    _want(wqT, torch.uint8, (K, N), "wqT")
    _want(sw, torch.float32, (N // 128, K // 128), "sw")
    dx = _out(dx, torch.bfloat16, (M, K), dyq.device, "dx")
    _launch_checks([("dyq", dyq), ("sdy", sdy), ("wqT", wqT), ("sw", sw), ("dx", dx),
                    ("workspace", workspace)], stream)
    _check(lib.fp8_block_gemm_dgrad(_ptr(dyq), _ptr(sdy), _ptr(wqT), _ptr(sw), _ptr(dx), M, N, K,
                                    *_workspace(workspace), _stream(stream)),
           "fp8_block_gemm_dgrad")
    return dx


def fp8_block_gemm_wgrad(dyqT, sdyT, xqT, sxT, dw=None, stream=None, workspace=None):
    """dW[N, K] = dY^T X (bf16) from along-token codes: dY^T [N, M] / scales
    [M/128, N] and X^T [K, M] / scales [M/128, K]."""
    if stream is not None and dw is None:
        return _elsewhere(fp8_block_gemm_wgrad, stream, dyqT, sdyT, xqT, sxT, dw, workspace=workspace)
    lib = load()
    N, M = dyqT.shape
    K = xqT.shape[0]
    _want(dyqT, torch.uint8, (N, M), "dyqT")
    _want(sdyT, torch.float32, (M // 128, N), "sdyT")
    _want(xqT, torch.uint8, (K, M), "xqT")
    _want(sxT, torch.float32, (M // 128, K), "sxT")
    dw = _out(dw, torch.bfloat16, (N, K), dyqT.device, "dw")
    _launch_checks([("dyqT", dyqT), ("sdyT", sdyT), ("xqT", xqT), ("sxT", sxT), ("dw", dw),
                    ("workspace", workspace)], stream)
    _check(lib.fp8_block_gemm_wgrad(_ptr(dyqT), _ptr(sdyT), _ptr(xqT), _ptr(sxT), _ptr(dw), N, K, M,
                                    *_workspace(workspace), _stream(stream)),
           "fp8_block_gemm_wgrad")
    return dw


def fp8_block_gemm_wgrad_accum_f32(dyqT, sdyT, xqT, sxT, dw, stream=None, workspace=None):
    """dW[N, K] += dY^T X in FP32, in place, from the same along-token codes
    as fp8_block_gemm_wgrad; dw is a float32 [N, K] tensor (the main
    gradient).  Returns dw."""
    lib = load()
    N, M = dyqT.shape
    K = xqT.shape[0]
    _want(dyqT, torch.uint8, (N, M), "dyqT")
    _want(sdyT, torch.float32, (M // 128, N), "sdyT")
    _want(xqT, torch.uint8, (K, M), "xqT")
    _want(sxT, torch.float32, (M // 128, K), "sxT")
    _want(dw, torch.float32, (N, K), "dw")
    _launch_checks([("dyqT", dyqT), ("sdyT", sdyT), ("xqT", xqT), ("sxT", sxT), ("dw", dw),
                    ("workspace", workspace)], stream)
    _check(lib.fp8_block_gemm_wgrad_accum_f32(_ptr(dyqT), _ptr(sdyT), _ptr(xqT), _ptr(sxT), _ptr(dw),
                                              N, K, M, *_workspace(workspace), _stream(stream)),
           "fp8_block_gemm_wgrad_accum_f32")
    return dw


MAX_SHARDS = 8


def fp8_block_gemm_wgrad_reduce_scatter_f32(dyqT, sdyT, xqT, sxT, shards, stream=None, workspace=None):
    """dW = dY^T X of this rank's tokens, added in FP32 into the owners'
    shards: rows [q N / R, (q + 1) N / R) of dW into shards[q], a float32
    [N / R, K] tensor of rank q (this GPU's, or a peer's mapped into this
    process, see exchange_shards).  After every rank's call and a
    synchronization each shard holds its old contents plus the sum over
    ranks.  Returns shards."""
    lib = load()
    N, M = dyqT.shape
    K = xqT.shape[0]
    R = len(shards)
    if not 1 <= R <= MAX_SHARDS or N % R:
        raise ValueError(f"need 1..{MAX_SHARDS} shards dividing N = {N}, got {R}")
    _want(dyqT, torch.uint8, (N, M), "dyqT")
    _want(sdyT, torch.float32, (M // 128, N), "sdyT")
    _want(xqT, torch.uint8, (K, M), "xqT")
    _want(sxT, torch.float32, (M // 128, K), "sxT")
    for q, t in enumerate(shards):            # peers' shards may live on other devices
        _want(t, torch.float32, (N // R, K), f"shards[{q}]")
    _launch_checks([("dyqT", dyqT), ("sdyT", sdyT), ("xqT", xqT), ("sxT", sxT), ("workspace", workspace)], stream)
    table = (ctypes.c_void_p * R)(*[t.data_ptr() for t in shards])
    _check(lib.fp8_block_gemm_wgrad_reduce_scatter_f32(_ptr(dyqT), _ptr(sdyT), _ptr(xqT), _ptr(sxT),
                                                       ctypes.cast(table, ctypes.c_void_p), R, N, K, M,
                                                       *_workspace(workspace), _stream(stream)),
           "fp8_block_gemm_wgrad_reduce_scatter_f32")
    return shards


def exchange_shards(local, group=None, share=None, rebuild=None):
    """The shards of a data-parallel group as seen from this rank: every
    rank passes its own main-gradient shard; returns the list in rank order,
    this rank's own tensor at its place and the others mapped into this
    process through CUDA IPC (torch's tensor sharing).  share(t) turns a
    tensor into a picklable handle and rebuild(handle) maps one back; they
    default to torch.multiprocessing's CUDA reductions."""
    import torch.distributed as dist

    if share is None or rebuild is None:
        from torch.multiprocessing.reductions import reduce_tensor

        share = share or (lambda t: reduce_tensor(t))
        rebuild = rebuild or (lambda h: h[0](*h[1]))
    world = dist.get_world_size(group)
    me = dist.get_rank(group)
    handles = [None] * world
    dist.all_gather_object(handles, share(local), group=group)
    return [local if q == me else rebuild(handles[q]) for q in range(world)]


def fp8_block_gemm_wgrad_static_ws(dyqT, sdyT, xqT, sxT, dw=None, stream=None):
    """dW = dY^T X (bf16) like fp8_block_gemm_wgrad, with the split
    schedule's workspace inside the library (no device buffer passed), for
    callers that cannot allocate one; calls must not overlap on the GPU."""
    if stream is not None and dw is None:
        return _elsewhere(fp8_block_gemm_wgrad_static_ws, stream, dyqT, sdyT, xqT, sxT, dw)
    lib = load()
    N, M = dyqT.shape
    K = xqT.shape[0]
    _want(dyqT, torch.uint8, (N, M), "dyqT")
    _want(sdyT, torch.float32, (M // 128, N), "sdyT")
    _want(xqT, torch.uint8, (K, M), "xqT")
    _want(sxT, torch.float32, (M // 128, K), "sxT")
    dw = _out(dw, torch.bfloat16, (N, K), dyqT.device, "dw")
    _launch_checks([("dyqT", dyqT), ("sdyT", sdyT), ("xqT", xqT), ("sxT", sxT), ("dw", dw)], stream)
    _check(lib.fp8_block_gemm_wgrad_static_ws(_ptr(dyqT), _ptr(sdyT), _ptr(xqT), _ptr(sxT), _ptr(dw), N, K, M,
                                              _stream(stream)),
           "fp8_block_gemm_wgrad_static_ws")
    return dw


def fp8_get_error() -> int:
    return int(load().fp8_get_error())


def fp8_clear_error() -> None:
    _check(load().fp8_clear_error(), "fp8_clear_error")


def fp8_set_wait_timeout_ns(ns: int) -> None:
    _check(load().fp8_set_wait_timeout_ns(int(ns)), "fp8_set_wait_timeout_ns")


def fp8_set_gemm_split_min_work(units_per_pair: int) -> None:
    _check(load().fp8_set_gemm_split_min_work(int(units_per_pair)), "fp8_set_gemm_split_min_work")


def fp8_status_string(status: int) -> str:
    return status_string(status)


def fp8_last_cuda_error() -> str:
    try:
        return load().fp8_last_cuda_error().decode()
    except OSError:
        return ""


def fp8_cast_e4m3_scaled(x, scale: float, q=None, stream=None):
    if stream is not None and q is None:
        return _elsewhere(fp8_cast_e4m3_scaled, stream, x, scale, q)
    lib = load()
    n = x.numel()
    _want(x, torch.float32, tuple(x.shape), "x")
    q = _out(q, torch.uint8, tuple(x.shape), x.device, "q")
    _launch_checks([("x", x), ("q", q)], stream)
    _check(lib.fp8_cast_e4m3_scaled(_ptr(x), ctypes.c_float(scale), _ptr(q), n, _stream(stream)),
           "fp8_cast_e4m3_scaled")
    return q


def fp8_selftest_division(stream=None):
    """Returns (code mismatches, first code mismatch, quotient-bit
    mismatches with |x/s| >= 2^-12, first such, quotient-bit mismatches
    below 2^-12)."""
    if stream is not None:
        return _elsewhere(fp8_selftest_division, stream)
    res = torch.zeros(6, dtype=torch.int64, device="cuda")
    _check(load().fp8_selftest_division(_ptr(res), _stream(stream)), "fp8_selftest_division")
    torch.cuda.synchronize()
    return tuple(res.cpu().tolist()[:5])


def fp8_selftest_wait_timeout(stream=None) -> None:
    _check(load().fp8_selftest_wait_timeout(_stream(stream)), "fp8_selftest_wait_timeout")


def fp8_selftest_stall_next(which: int) -> None:
    """Arm the next GEMM (1), tile quantizer (2) or both (3) launches to run
    into their bounded wait (test support)."""
    _check(load().fp8_selftest_stall_next(int(which)), "fp8_selftest_stall_next")


def fp8_selftest_silu_bf16(stream=None):
    """silu of every bfloat16 bit pattern as the fused SwiGLU producer
    computes it: a numpy uint16 array of 65536 bit patterns (index = input
    bits)."""
    if stream is not None:
        return _elsewhere(fp8_selftest_silu_bf16, stream)
    out = torch.empty(65536, dtype=torch.int16, device="cuda")
    _check(load().fp8_selftest_silu_bf16(_ptr(out), _stream(stream)), "fp8_selftest_silu_bf16")
    torch.cuda.synchronize()
    return out.cpu().numpy().view("uint16")


def fp8_selftest_gemm_schedule(M: int, N: int, K: int, pairs: int, split: bool):
    """The GEMMs' work schedule as the library computes it (host code shared
    with the kernel): a list of (pair, tile, kb0, kb1, add_first, add_end)."""
    import numpy as np

    cap = 1 << 16
    rows = np.zeros((cap, 5), dtype=np.int32)
    n = ctypes.c_int64(0)
    _check(load().fp8_selftest_gemm_schedule(int(M), int(N), int(K), int(pairs), int(bool(split)),
                                            ctypes.c_void_p(rows.ctypes.data), cap, ctypes.byref(n)),
           "fp8_selftest_gemm_schedule")
    out = []
    for r in rows[: n.value]:
        out.append((int(r[0]), int(r[1]), int(r[2]), int(r[3]), int(r[4]) >> 16, int(r[4]) & 0xFFFF))
    return out
