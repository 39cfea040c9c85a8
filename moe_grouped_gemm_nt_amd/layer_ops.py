"""Binding of the operators that stand around the grouped products of an MoE layer (C ABI in
include/mgg/layer_ops.h): routing, the norms around a block, and the orthogonalised update of
expert weights.

As the grouped products' binding, it only marshals: sizes come from tensor shapes, kernels run
on the current stream of the tensors' device, outputs (and workspaces) are allocated here when
not given, and a non-OK status raises. Rows may be strided (last dimension contiguous) where a
tensor is read; outputs are contiguous. Activations are bfloat16 or float32.
"""

from __future__ import annotations

import ctypes

import moe_grouped_gemm_nt_amd as _mgg

MGG_ACT_BF16, MGG_ACT_F32 = 0, 1
MGG_SCORE_SOFTMAX, MGG_SCORE_SIGMOID = 0, 1
MGG_GATE_NONE, MGG_GATE_TOKEN, MGG_GATE_ELEMENT = 0, 1, 2
_SCORE = {"softmax": MGG_SCORE_SOFTMAX, "sigmoid": MGG_SCORE_SIGMOID}


class MggBlock(ctypes.Structure):
    """mgg_block of include/mgg/layer_ops.h."""
    _fields_ = [("dtype", ctypes.c_int), ("param", ctypes.c_int), ("T", ctypes.c_int),
                ("H", ctypes.c_int), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("gate_kind", ctypes.c_int),
                ("gate", ctypes.c_void_p), ("ld_gate", ctypes.c_int64),
                ("scale", ctypes.c_void_p), ("w_after", ctypes.c_void_p),
                ("w_before", ctypes.c_void_p), ("alpha", ctypes.c_float),
                ("beta", ctypes.c_float), ("eps", ctypes.c_float)]


def declare(lib: ctypes.CDLL):
    """Argument and result types of the entry points."""
    vp, i32, i64, sz, f32 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                             ctypes.c_float)
    block = ctypes.POINTER(MggBlock)
    lib.route_topk.argtypes = [i32, i32, i32, i32, vp, i64, vp, i32, i32, f32, i32, vp, vp, vp,
                               vp, vp, vp, vp, sz, vp]
    lib.route_topk_backward.argtypes = [i32, i32, i32, i32, vp, i64, i32, i32, f32, i32, vp, vp,
                                        vp, vp, vp, vp, vp, vp]
    lib.block_residual_norm.argtypes = [block, vp, vp, vp]
    lib.block_residual_norm_backward.argtypes = [block, vp, i64, vp, i64, vp, vp, vp, vp, vp,
                                                 vp, vp, sz, vp]
    lib.block_norm.argtypes = [i32, i32, i32, i32, vp, i64, vp, f32, vp, vp]
    lib.block_norm_backward.argtypes = [i32, i32, i32, i32, vp, i64, vp, f32, vp, i64, vp, i64,
                                        vp, vp, vp, sz, vp]
    lib.grouped_newton_schulz.argtypes = [i32, i32, i32, i32, i32, vp, vp, i32,
                                          ctypes.POINTER(f32), f32, f32, vp, sz, vp]
    for f in (lib.route_topk, lib.route_topk_backward, lib.block_residual_norm,
              lib.block_residual_norm_backward, lib.block_norm, lib.block_norm_backward,
              lib.grouped_newton_schulz):
        f.restype = ctypes.c_int
    lib.route_topk_workspace.argtypes = [i32, i32, i32]
    lib.block_residual_norm_backward_workspace.argtypes = [i32, i32]
    lib.grouped_newton_schulz_workspace.argtypes = [i32, i32, i32]
    for f in (lib.route_topk_workspace, lib.block_residual_norm_backward_workspace,
              lib.grouped_newton_schulz_workspace):
        f.restype = sz


def _ptr(t):
    """Address of a tensor, None for none (ctypes takes either for a pointer)."""
    return None if t is None else t.data_ptr()


def _same_device(first, *rest):
    """Every tensor that is given on the first one's GPU."""
    device = first.device
    ok = device.type == "cuda"
    for t in rest:
        if t is not None and t.device != device:
            ok = False
    _mgg._require(ok, "all tensors must be on the same GPU")
    return device


_raw_stream = _current_device = None


def _torch_calls():
    """Looks up, once, the current device and the handle of its current stream (without a Stream
    object where torch offers that: a tenth of the time of a small call)."""
    global _raw_stream, _current_device
    import torch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda i: torch.cuda.current_stream(i).cuda_stream)
    _current_device = torch.cuda.current_device


def _run(fn, device, *args):
    """Calls an entry point on the device's current stream, and raises on a non-OK status. The
    device is made current only when it is not: small calls are bound by this host code."""
    if _raw_stream is None:
        _torch_calls()
    index = device.index
    if _current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        import torch
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _mgg._check(status)


_ACTS = {}  # torch element type -> mgg_act, filled when torch is first needed


def _act(t, name) -> int:
    code = _ACTS.get(t.dtype)
    if code is None:
        import torch
        _ACTS.update({torch.bfloat16: MGG_ACT_BF16, torch.float32: MGG_ACT_F32})
        if t.dtype not in _ACTS:
            raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
        code = _ACTS[t.dtype]
    return code


def _rows(t, T, H, dtype, name) -> int:
    """Row stride of a [T, H] tensor that is read."""
    if t.shape != (T, H):
        raise ValueError(f"{name} must be [{T}, {H}], got {list(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    row, col = t.stride()
    if H > 1 and col != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if T <= 1:
        return H
    if row < H:
        raise ValueError(f"{name}: rows must not overlap")
    return row


def _given(t, shape, dtype, name, like):
    """An output: the caller's, checked, or a new one."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {list(shape)}")
    _mgg._contig(t)
    return t


def _workspace(ws, size, like):
    import torch
    if ws is None:
        return like.new_empty(size, dtype=torch.uint8)
    if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.numel() < size:
        raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {size} bytes")
    return ws


def _sequences(seq_ends):
    import torch
    if seq_ends is None:
        return 1
    _mgg._require(seq_ends.dtype == torch.int32 and seq_ends.dim() == 1 and seq_ends.numel() >= 1,
                  "seq_ends must be int32 [S]")
    _mgg._contig(seq_ends)
    return seq_ends.numel()


def _score_code(score) -> int:
    if score not in _SCORE:
        raise ValueError(f"score must be one of {sorted(_SCORE)}, got {score!r}")
    return _SCORE[score]


def route_topk(logits, topk, bias=None, seq_ends=None, score="softmax", renormalize=True,
               scale=1.0, balance=True, workspace=None):
    """Top-k routing of logits[T, G] (bf16 or float32): (ids int32 [T, k], weights float32
    [T, k], counts int32 [S, G], tokens int32 [S], loss float32 [S]), or (ids, weights) with
    balance=False. seq_ends int32 [S] on the device: cumulative row ends of the sequences, rows
    past the last are padding (ids -1); None: one sequence. bias float32 [G] (sigmoid scores
    only) enters the selection, not the weights. loss is each sequence's balance loss, 1 when
    counts and probabilities are even."""
    import torch
    _mgg._require(logits.dim() == 2, "logits must be [T, G]")
    T, G = logits.shape
    dt, code, k = _act(logits, "logits"), _score_code(score), int(topk)
    ld = _rows(logits, T, G, logits.dtype, "logits")
    _mgg._require(1 <= k <= min(G, 32), "topk must be in [1, min(G, 32)]")
    S = _sequences(seq_ends)
    if bias is not None:
        _mgg._require(code == MGG_SCORE_SIGMOID, "a selection bias goes with sigmoid scores")
        _mgg._require(bias.dtype == torch.float32 and bias.shape == (G,),
                      "bias must be float32 [G]")
        _mgg._contig(bias)
    lib = _mgg.load_library()
    _same_device(logits, bias, seq_ends, workspace)
    ids = logits.new_empty((T, k), dtype=torch.int32)
    weights = logits.new_empty((T, k), dtype=torch.float32)
    counts = tokens = loss = None
    size = 0
    if balance:
        counts = logits.new_empty((S, G), dtype=torch.int32)
        tokens = logits.new_empty(S, dtype=torch.int32)
        loss = logits.new_empty(S, dtype=torch.float32)
        size = lib.route_topk_workspace(T, G, S)
        workspace = _workspace(workspace, size, logits)
    _run(lib.route_topk, logits.device, dt, T, G, k, _ptr(logits), ld, _ptr(bias), code,
         int(bool(renormalize)), float(scale), S, _ptr(seq_ends), _ptr(ids), _ptr(weights),
         _ptr(counts), _ptr(tokens), _ptr(loss), _ptr(workspace) if balance else None, size)
    return (ids, weights, counts, tokens, loss) if balance else (ids, weights)


def route_topk_backward(logits, ids, counts=None, tokens=None, d_weights=None, d_balance=None,
                        seq_ends=None, score="softmax", renormalize=True, scale=1.0,
                        d_logits=None):
    """Gradient of the logits [T, G] from those of route_topk's weights (d_weights float32
    [T, k]) and losses (d_balance float32 [S], which needs counts and tokens); either may be
    None. seq_ends, score, renormalize and scale as in the forward call."""
    import torch
    _mgg._require(logits.dim() == 2, "logits must be [T, G]")
    T, G = logits.shape
    dt, code = _act(logits, "logits"), _score_code(score)
    ld = _rows(logits, T, G, logits.dtype, "logits")
    S = _sequences(seq_ends)
    _mgg._require(ids.dim() == 2 and ids.shape[0] == T and ids.dtype == torch.int32,
                  "ids must be int32 [T, k]")
    k = ids.shape[1]
    _mgg._require(1 <= k <= min(G, 32), "k must be in [1, min(G, 32)]")
    _mgg._require(d_weights is not None or d_balance is not None,
                  "one of d_weights and d_balance must be given")
    if d_weights is not None:
        _mgg._require(d_weights.dtype == torch.float32 and d_weights.shape == (T, k),
                      "d_weights must be float32 [T, k]")
    if d_balance is not None:
        _mgg._require(d_balance.dtype == torch.float32 and d_balance.shape == (S,),
                      "d_balance must be float32 [S]")
        _mgg._require(counts is not None and tokens is not None,
                      "d_balance needs counts and tokens")
        _mgg._require(counts.dtype == torch.int32 and counts.shape == (S, G),
                      "counts must be int32 [S, G]")
        _mgg._require(tokens.dtype == torch.int32 and tokens.shape == (S,),
                      "tokens must be int32 [S]")
    else:
        counts = tokens = None
    lib = _mgg.load_library()
    _same_device(logits, ids, counts, tokens, d_weights, d_balance, seq_ends, d_logits)
    _mgg._contig(ids, counts, tokens, d_weights, d_balance)
    d_logits = _given(d_logits, (T, G), logits.dtype, "d_logits", logits)
    _run(lib.route_topk_backward, logits.device, dt, T, G, k, _ptr(logits), ld, code,
         int(bool(renormalize)), float(scale), S, _ptr(seq_ends), _ptr(ids), _ptr(counts),
         _ptr(tokens), _ptr(d_weights), _ptr(d_balance), _ptr(d_logits))
    return d_logits


def _param(params, H):
    """Element type of the parameter vectors that are given (one for all)."""
    dtype = None
    for p in params:
        if p is None:
            continue
        if p.shape != (H,) or not p.is_contiguous():
            raise ValueError(f"scale and norm weights must be contiguous and must be [{H}]")
        if dtype is not None and p.dtype != dtype:
            raise ValueError("scale, w_after and w_before must have one element type")
        if dtype is None:
            dtype, code = p.dtype, _act(p, "scale and norm weights")
    return MGG_ACT_F32 if dtype is None else code


def _block(x, y, w_after, gate, scale, w_before, alpha, beta, eps):
    """mgg_block of a call, checked; the tensors stay alive with the caller."""
    _mgg._require(x.dim() == 2, "x must be [T, H]")
    T, H = x.shape
    dt = _act(x, "x")
    ldx = _rows(x, T, H, x.dtype, "x")
    ldy = _rows(y, T, H, x.dtype, "y")
    kind, ld_gate = MGG_GATE_NONE, 0
    if gate is not None:
        if gate.dim() == 2:
            kind, ld_gate = MGG_GATE_ELEMENT, _rows(gate, T, H, x.dtype, "gate")
        else:
            if gate.shape != (T,) or gate.dtype != x.dtype:
                raise ValueError(f"gate must be {x.dtype} [T] or [T, H]")
            kind, ld_gate = MGG_GATE_TOKEN, gate.stride(0) if T > 1 else 1
            _mgg._require(ld_gate >= 1, "gate: values must not overlap")
    param = _param((scale, w_after, w_before), H)
    return MggBlock(dt, param, T, H, x.data_ptr(), ldx, y.data_ptr(), ldy, kind, _ptr(gate),
                    ld_gate, _ptr(scale), _ptr(w_after), _ptr(w_before), alpha, beta, eps)


def block_norm(x, w, eps=1e-6, u=None):
    """The norm before a block: u = x / sqrt(mean(x^2) + eps) * w over the rows of x[T, H]."""
    import torch
    _mgg._require(x.dim() == 2, "x must be [T, H]")
    T, H = x.shape
    dt, ldx, param = _act(x, "x"), _rows(x, T, H, x.dtype, "x"), _param((w,), H)
    lib = _mgg.load_library()
    _same_device(x, w, u)
    u = _given(u, (T, H), x.dtype, "u", x)
    _run(lib.block_norm, x.device, dt, param, T, H, _ptr(x), ldx, _ptr(w), float(eps), _ptr(u))
    return u


def block_norm_backward(x, w, d_u, d_x=None, eps=1e-6, workspace=None):
    """Gradients of block_norm: (d_x_in [T, H], d_w float32 [H]). d_x, when given, is the
    gradient that already reaches x past the block and is added."""
    import torch
    _mgg._require(x.dim() == 2, "x must be [T, H]")
    T, H = x.shape
    dt, ldx, param = _act(x, "x"), _rows(x, T, H, x.dtype, "x"), _param((w,), H)
    ld_du = _rows(d_u, T, H, x.dtype, "d_u")
    ld_dx = _rows(d_x, T, H, x.dtype, "d_x") if d_x is not None else H
    lib = _mgg.load_library()
    _same_device(x, w, d_u, d_x, workspace)
    d_in = x.new_empty((T, H), dtype=x.dtype)
    d_w = x.new_empty(H, dtype=torch.float32)
    size = lib.block_residual_norm_backward_workspace(T, H)
    workspace = _workspace(workspace, size, x)
    _run(lib.block_norm_backward, x.device, dt, param, T, H, _ptr(x), ldx, _ptr(w), float(eps),
         _ptr(d_x), ld_dx, _ptr(d_u), ld_du, _ptr(d_in), _ptr(d_w), _ptr(workspace), size)
    return d_in, d_w


def block_residual_norm(x, y, w_after=None, gate=None, scale=None, w_before=None, alpha=1.0,
                        beta=1.0, eps=1e-6, x_out=None, u=None):
    """The end of a block and the start of the next: with z = rms(y; w_after) (y without
    w_after) and g = sigmoid(gate) (gate [T] or [T, H]; 1 without),
        x_out = alpha * x + beta * scale * g * z,    u = rms(x_out; w_before),
    for x, y [T, H]. Returns (x_out, u); u is None without w_before."""
    import torch
    block = _block(x, y, w_after, gate, scale, w_before, alpha, beta, eps)
    T, H = x.shape
    _mgg._require(u is None or w_before is not None, "u and w_before go together")
    lib = _mgg.load_library()
    _same_device(x, y, w_after, gate, scale, w_before, x_out, u)
    x_out = _given(x_out, (T, H), x.dtype, "x_out", x)
    if w_before is not None:
        u = _given(u, (T, H), x.dtype, "u", x)
    _run(lib.block_residual_norm, x.device, ctypes.byref(block), _ptr(x_out), _ptr(u))
    return x_out, u


def block_residual_norm_backward(x_out, y, d_x=None, d_u=None, w_after=None, gate=None,
                                 scale=None, w_before=None, alpha=1.0, beta=1.0, eps=1e-6,
                                 workspace=None):
    """Gradients of block_residual_norm from its output stream x_out and its y: d_x is the
    gradient of x_out from the rest of the model, d_u that of u. Returns (d_x_in, d_y, d_gate,
    d_scale, d_w_after, d_w_before), None where the input was None; the last three are float32
    [H]."""
    import torch
    block = _block(x_out, y, w_after, gate, scale, w_before, alpha, beta, eps)
    T, H = x_out.shape
    _mgg._require((d_u is None) == (w_before is None), "d_u and w_before go together")
    _mgg._require(d_x is not None or d_u is not None, "one of d_x and d_u must be given")
    ld_dx = _rows(d_x, T, H, x_out.dtype, "d_x") if d_x is not None else H
    ld_du = _rows(d_u, T, H, x_out.dtype, "d_u") if d_u is not None else H
    lib = _mgg.load_library()
    _same_device(x_out, y, d_x, d_u, w_after, gate, scale, w_before, workspace)

    def like(t, shape, dtype):
        return None if t is None else x_out.new_empty(shape, dtype=dtype)

    d_in = x_out.new_empty((T, H), dtype=x_out.dtype)
    d_y = x_out.new_empty((T, H), dtype=x_out.dtype)
    d_gate = None if gate is None else like(gate, tuple(gate.shape), x_out.dtype)
    d_scale, d_w_after, d_w_before = (like(p, (H,), torch.float32)
                                      for p in (scale, w_after, w_before))
    size = lib.block_residual_norm_backward_workspace(T, H)
    workspace = _workspace(workspace, size, x_out)
    _run(lib.block_residual_norm_backward, x_out.device, ctypes.byref(block), _ptr(d_x), ld_dx,
         _ptr(d_u), ld_du, _ptr(d_in), _ptr(d_y), _ptr(d_gate), _ptr(d_scale), _ptr(d_w_after),
         _ptr(d_w_before), _ptr(workspace), size)
    return d_in, d_y, d_gate, d_scale, d_w_after, d_w_before


def grouped_newton_schulz(X, out=None, steps=5, coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7,
                          scale=1.0, out_dtype=None, workspace=None):
    """Orthogonalised update of each matrix of X[G, M, N] (bf16 or float32): X / (|X|_F + eps),
    then `steps` of X <- a X + (b A + c A A) X with A = X X^T, times `scale`. coeffs: one
    (a, b, c) for all steps, or one for each. `out` takes X's element type, or out_dtype."""
    import torch
    _mgg._require(X.dim() == 3, "X must be [G, M, N]")
    G, M, N = X.shape
    dt = _act(X, "X")
    steps = int(steps)
    _mgg._require(1 <= steps <= 32, "steps must be in [1, 32]")
    rows = list(coeffs)
    if rows and not hasattr(rows[0], "__len__"):
        rows = [rows] * steps
    _mgg._require(len(rows) == steps and all(len(r) == 3 for r in rows),
                  "coeffs must be (a, b, c), or one such triple for each step")
    flat = (ctypes.c_float * (3 * steps))(*(float(v) for r in rows for v in r))
    out_dtype = out.dtype if out is not None else (out_dtype or X.dtype)
    lib = _mgg.load_library()
    _same_device(X, out, workspace)
    _mgg._contig(X)
    out = _given(out, (G, M, N), out_dtype, "out", X)
    size = lib.grouped_newton_schulz_workspace(G, M, N)
    workspace = _workspace(workspace, size, X)
    _run(lib.grouped_newton_schulz, X.device, dt, _act(out, "out"), G, M, N, _ptr(X), _ptr(out),
         steps, flat, float(eps), float(scale), _ptr(workspace), size)
    return out
