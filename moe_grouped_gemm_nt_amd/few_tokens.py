"""Binding of the MoE layer for the few tokens of a decoding step (C ABI in
include/mgg/few_tokens.h). It marshals as layer_ops.py does."""

from __future__ import annotations

import ctypes

import moe_grouped_gemm_nt_amd as _mgg
from moe_grouped_gemm_nt_amd import layer_ops as _ops

MGG_WEIGHT_BF16, MGG_WEIGHT_FP8, MGG_WEIGHT_FP4 = 0, 1, 2


def declare(lib: ctypes.CDLL):
    """Argument and result types of the entry points."""
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.moe_few_tokens.argtypes = [i32, i32, i32, i32, i32, i32, vp, i64, vp, vp, vp, vp, vp, vp,
                                   i32, i32, i32, vp, i64, vp, vp, sz, vp]
    lib.moe_few_tokens.restype = ctypes.c_int
    lib.moe_few_tokens_workspace.argtypes = [i32, i32, i32, i32]
    lib.moe_few_tokens_workspace.restype = sz


_WEIGHT = {}  # torch element type -> mgg_weight, filled when torch is first needed


def _weight(w13, w2, G, H, I):
    """mgg_weight of a call from its weight tensors."""
    import torch
    if not _WEIGHT:
        _WEIGHT.update({torch.bfloat16: MGG_WEIGHT_BF16, torch.uint8: MGG_WEIGHT_FP8,
                        torch.float8_e4m3fn: MGG_WEIGHT_FP8})
        fp4 = getattr(torch, "float4_e2m1fn_x2", None)
        if fp4 is not None:
            _WEIGHT[fp4] = MGG_WEIGHT_FP4
    code = _WEIGHT.get(w13.dtype)
    if code is None:
        raise TypeError(f"w13 must be bfloat16, FP8 bytes or packed FP4, got {w13.dtype}")
    row13, row2 = w13.shape[2], w2.shape[2]
    if w13.dtype == torch.uint8 and 2 * row13 == H:
        code = MGG_WEIGHT_FP4
    packed = 2 if code == MGG_WEIGHT_FP4 else 1
    if row13 * packed != H or w2.shape[:2] != (G, H) or row2 * packed != I or \
            w2.dtype != w13.dtype:
        raise ValueError("w13 must be [G, 2I, H] and w2 [G, H, I] of one element type "
                         "(FP4: half as many bytes a row)")
    return code


def _scales(s, G, N, K, code, gran, like, name):
    import torch
    if s is None:
        raise ValueError(f"FP8 and FP4 weights need {name}")
    want = {"block128": (G, -(-N // 128), K // 128), "channel": (G, K // 128, N),
            "block32": (G, K // 128, N, 4)}[gran]
    if s.shape != want or s.dtype != like.dtype or \
            (s.dtype != torch.uint8 and s.dtype != torch.float32):
        raise ValueError(f"{name} ({gran}) must be float32 or uint8 {list(want)}, both scales of "
                         f"one type; got {s.dtype} {list(s.shape)}")


def moe_few_tokens(x, ids, weights, w13, w2, s13=None, s2=None, sfb_gran=None, residual=None,
                   out=None, out_dtype=None, workspace=None):
    """A whole MoE layer for few tokens (at most 128):
        out[t] = residual[t] + sum_j weights[t, j] * w2[e] (silu(g) * u),  [g; u] = w13[e] x[t],
    e = ids[t, j], ids outside [0, G) skipped. x bf16 [T, H]; ids int32 and weights float32
    [T, k] (route_topk's); w13 [G, 2I, H] (gate rows, then up rows) and w2 [G, H, I] in bf16, FP8
    bytes or packed FP4 with the grouped products' scales s13, s2 and granularity sfb_gran
    ("block128" by default, "channel", for FP4 "block32"). residual [T, H] has the output's type,
    out_dtype (bf16 by default, or float32)."""
    import torch
    _mgg._require(x.dim() == 2 and ids.dim() == 2 and w13.dim() == 3 and w2.dim() == 3,
                  "x must be [T, H], ids [T, k], w13 [G, 2I, H], w2 [G, H, I]")
    T, H = x.shape
    k, G = ids.shape[1], w13.shape[0]
    _mgg._require(w13.shape[1] % 2 == 0, "w13 must hold as many up rows as gate rows")
    I = w13.shape[1] // 2
    if x.dtype != torch.bfloat16:
        raise TypeError(f"x must be bfloat16, got {x.dtype}")
    ldx = _ops._rows(x, T, H, x.dtype, "x")
    if ids.shape[0] != T or ids.dtype != torch.int32:
        raise ValueError("ids must be int32 [T, k]")
    if weights.shape != ids.shape or weights.dtype != torch.float32:
        raise ValueError("weights must be float32 [T, k]")
    code = _weight(w13, w2, G, H, I)
    gran = sfb_gran or ("block32" if code == MGG_WEIGHT_FP4 else "block128")
    allowed = ("block32",) if code == MGG_WEIGHT_FP4 else ("block128", "channel")
    if gran not in allowed:
        raise ValueError(f"weight-scale granularity {gran!r} does not fit these weights "
                         f"(expected one of {list(allowed)})")
    if code == MGG_WEIGHT_BF16:
        _mgg._require(s13 is None and s2 is None, "bf16 weights take no scales")
    else:
        _scales(s13, G, 2 * I, H, code, gran, s13, "s13")
        _scales(s2, G, H, I, code, gran, s13, "s2")
    out_dtype = out.dtype if out is not None else (out_dtype or torch.bfloat16)
    lib = _mgg.load_library()
    _ops._same_device(x, ids, weights, w13, w2, s13, s2, residual, out, workspace)
    _mgg._contig(ids, weights, w13, w2, s13, s2)
    out = _ops._given(out, (T, H), out_dtype, "out", x)
    out_code = _ops._act(out, "out")
    ld_res = _ops._rows(residual, T, H, out_dtype, "residual") if residual is not None else H
    size = lib.moe_few_tokens_workspace(T, k, G, I)
    workspace = _ops._workspace(workspace, size, x)
    _ops._run(lib.moe_few_tokens, x.device, code, T, k, G, H, I, x.data_ptr(), ldx,
              ids.data_ptr(), weights.data_ptr(), w13.data_ptr(), _ops._ptr(s13), w2.data_ptr(),
              _ops._ptr(s2), _mgg._sf_fmt(s13), _mgg._GRAN[gran], out_code, _ops._ptr(residual),
              ld_res, out.data_ptr(), workspace.data_ptr(), size)
    return out
