"""Binding of the dense products with bias, activation and residual in their epilogue, and of
their gradients (C ABI in include/mgg/linear.h). It marshals as layer_ops.py does."""

from __future__ import annotations

import ctypes

import moe_grouped_gemm_nt_amd as _mgg
from moe_grouped_gemm_nt_amd import layer_ops as _ops

_FUNC = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "swiglu": 4}


class MggLinear(ctypes.Structure):
    """mgg_linear of include/mgg/linear.h."""
    _fields_ = [("dtype", ctypes.c_int), ("out_dt", ctypes.c_int), ("bias_dt", ctypes.c_int),
                ("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("func", ctypes.c_int), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("w", ctypes.c_void_p), ("ldw", ctypes.c_int64), ("bias", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("ld_res", ctypes.c_int64)]


def declare(lib: ctypes.CDLL):
    """Argument and result types of the entry points."""
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    linear = ctypes.POINTER(MggLinear)
    lib.linear_act.argtypes = [linear, vp, vp, vp, sz, vp]
    lib.linear_act_backward.argtypes = [linear, vp, i64, vp, i64, vp, vp, i32, vp, vp, sz, vp]
    lib.linear_act.restype = lib.linear_act_backward.restype = ctypes.c_int
    lib.linear_act_workspace.argtypes = [linear]
    lib.linear_act_backward_workspace.argtypes = [linear, vp, i64, vp, i64, vp, vp, vp]
    lib.linear_act_workspace.restype = lib.linear_act_backward_workspace.restype = sz


def _linear(x, w, bias, func, residual, out_dtype):
    """mgg_linear of a call, checked, and the columns of its output; the tensors stay alive with
    the caller."""
    import torch
    _mgg._require(x.dim() == 2 and w.dim() == 2, "x must be [M, K] and w [N, K]")
    (M, K), N = x.shape, w.shape[0]
    dt = _ops._act(x, "x")
    ldx = _ops._rows(x, M, K, x.dtype, "x")
    ldw = _ops._rows(w, N, K, x.dtype, "w")
    if func not in _FUNC:
        raise ValueError(f"func must be one of {sorted(_FUNC)}, got {func!r}")
    C = N
    if func == "swiglu":
        _mgg._require(N % 2 == 0, "swiglu needs as many up rows as gate rows in w")
        C = N // 2
    bias_dt = _ops.MGG_ACT_F32
    if bias is not None:
        if bias.shape != (N,) or not bias.is_contiguous():
            raise ValueError(f"bias must be contiguous [{N}]")
        bias_dt = _ops._act(bias, "bias")
    out_dt = dt
    if out_dtype != x.dtype:
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"the output must be bfloat16 or float32, got {out_dtype}")
        out_dt = _ops.MGG_ACT_BF16 if out_dtype == torch.bfloat16 else _ops.MGG_ACT_F32
    ld_res = C if residual is None else _ops._rows(residual, M, C, out_dtype, "residual")
    return MggLinear(dt, out_dt, bias_dt, M, N, K, _FUNC[func], x.data_ptr(), ldx, w.data_ptr(),
                     ldw, _ops._ptr(bias), _ops._ptr(residual), ld_res), C


def _room(ws, size, like):
    """The workspace's address: the caller's, a new one, or none where none is needed."""
    return None if size == 0 else _ops._workspace(ws, size, like)


def linear_act(x, w, bias=None, func="none", residual=None, keep_z=False, out=None,
               out_dtype=None, workspace=None):
    """out = f(x w^T + bias) + residual for x[M, K] and w[N, K] (both bf16 or both float32), bias
    [N] in either. func: "none", "relu", "gelu" (by erf), "silu", or "swiglu": silu of the first
    N/2 columns times the others. out [M, N] (swiglu: [M, N/2]) and residual have out_dtype (bf16
    or float32, x's by default). Returns out, with keep_z (out, z): z = x w^T + bias in x's type,
    what linear_act_backward takes."""
    out_dtype = out.dtype if out is not None else (out_dtype or x.dtype)
    linear, C = _linear(x, w, bias, func, residual, out_dtype)
    lib = _mgg.load_library()
    _ops._same_device(x, w, bias, residual, out, workspace)
    out = _ops._given(out, (linear.M, C), out_dtype, "out", x)
    z = x.new_empty((linear.M, linear.N)) if keep_z else None
    ref = ctypes.byref(linear)
    size = lib.linear_act_workspace(ref)
    workspace = _room(workspace, size, x)
    _ops._run(lib.linear_act, x.device, ref, out.data_ptr(), _ops._ptr(z), _ops._ptr(workspace),
              size)
    return (out, z) if keep_z else out


def linear_act_backward(x, w, d_out, z=None, func="none", need_x=True, need_w=True,
                        need_bias=False, dw_dtype=None, workspace=None):
    """Gradients of linear_act from that of its output, d_out (bf16 or float32), and its z (None
    exactly for func "none"): (d_x [M, K], d_w [N, K], d_bias float32 [N]), None where not
    needed. d_x has x's type, d_w dw_dtype (bf16 or float32, w's by default). With
    dz = d_out f'(z) held in x's type: d_x = dz w, d_w = dz^T x, d_bias the sums of dz. The
    residual's gradient is d_out."""
    import torch
    _mgg._require(need_x or need_w or need_bias, "one gradient must be needed")
    linear, C = _linear(x, w, None, func, None, d_out.dtype)
    M, N, K = linear.M, linear.N, linear.K
    ldd = _ops._rows(d_out, M, C, d_out.dtype, "d_out")
    _mgg._require((z is None) == (func == "none"), "z goes with a function, and only with one")
    ldz = N if z is None else _ops._rows(z, M, N, x.dtype, "z")
    lib = _mgg.load_library()
    _ops._same_device(x, w, d_out, z, workspace)
    d_x = x.new_empty((M, K)) if need_x else None
    d_w = x.new_empty((N, K), dtype=dw_dtype or w.dtype) if need_w else None
    dw_dt = _ops._act(d_w, "d_w") if need_w else 0
    d_bias = x.new_empty(N, dtype=torch.float32) if need_bias else None
    ref, ptr = ctypes.byref(linear), _ops._ptr
    args = (ref, ptr(z), ldz, d_out.data_ptr(), ldd, ptr(d_x), ptr(d_w))
    size = lib.linear_act_backward_workspace(*args, ptr(d_bias))
    workspace = _room(workspace, size, x)
    _ops._run(lib.linear_act_backward, x.device, *args, dw_dt, ptr(d_bias), ptr(workspace), size)
    return d_x, d_w, d_bias
