"""Float64 definitions of the MoE layer for few tokens (include/mgg/few_tokens.h) and of the
dense products with bias, activation and residual and their gradients (include/mgg/linear.h).
Inputs are float64 arrays holding the element values (dequantized weights)."""

from __future__ import annotations

import math

import numpy as np

from .formats import decode_e2m1, decode_e4m3fn, decode_scale, unpack_fp4

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def sigmoid(v):
    with np.errstate(over="ignore"):
        return np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))),
                        np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))


def silu(v):
    return v * sigmoid(v)


def normal_cdf(v):
    return 0.5 * _erfc(-np.asarray(v) / math.sqrt(2.0))


# --------------------------------------------------------------------------- few tokens

def expert_weights(codes, scales, gran, fmt):
    """Values [G, N, K] of FP8 (uint8 [G, N, K]) or packed FP4 (uint8 [G, N, K/2], gran
    "block32") weights with their scales in the grouped products' layouts."""
    if gran == "block32":
        v = decode_e2m1(unpack_fp4(codes))
        s = decode_scale(scales, "ue8m0")                      # [G, K/128, N, 4]
        G, N, K = v.shape
        return v * np.repeat(s.transpose(0, 2, 1, 3).reshape(G, N, K // 32), 32, 2)
    v = decode_e4m3fn(codes)
    s = decode_scale(scales, fmt)
    N = v.shape[1]
    if gran == "channel":
        s = s.transpose(0, 2, 1)                               # [G, N, K/128]
    else:
        s = np.repeat(s, 128, 1)[:, :N]
    return v * np.repeat(s, 128, 2)


def moe_few_tokens(x, ids, weights, w13, w2, residual=None, roundings=None, held=2.0 ** -24):
    """out [T, H]; with `roundings` (u: relative size of a float32 rounding) also a bound on what
    float32 sums may be off by, counting one rounding for each term of a sum, the gated unit's
    own, and `held`: the relative error of silu(g) u between the products (2^-8
    as one bfloat16, 2^-24 as three)."""
    T, H = x.shape
    G, I = w13.shape[0], w13.shape[1] // 2
    out = np.zeros((T, H)) if residual is None else residual.copy()
    err, size = np.zeros((T, H)), np.abs(out)
    u = roundings or 0.0
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < G:
                continue
            z, zs = w13[e] @ x[t], np.abs(w13[e]) @ np.abs(x[t])
            g, up = z[:I], z[I:]
            h = silu(g) * up
            y, ys = w2[e] @ h, np.abs(w2[e]) @ np.abs(h)
            out[t] += weights[t, j] * y
            if roundings:
                dz = (H + 8) * u * zs
                dh = 1.1 * dz[:I] * np.abs(up) + np.abs(silu(g)) * dz[I:] \
                    + ((16 + 2 * np.abs(g)) * u + held) * np.abs(h)
                err[t] += abs(weights[t, j]) * (np.abs(w2[e]) @ dh + (I + 8) * u * ys)
                size[t] += np.abs(weights[t, j]) * ys
    return (out, err + (ids.shape[1] + 12) * u * size) if roundings else out


# --------------------------------------------------------------------------- linear

def func_of(func, z):
    """f(z); the gated unit halves the columns."""
    if func == "none":
        return z
    if func == "relu":
        return np.maximum(z, 0.0)
    if func == "gelu":
        return z * normal_cdf(z)
    if func == "silu":
        return silu(z)
    g, up = np.split(z, 2, 1)
    return silu(g) * up


def linear(x, w, bias=None, func="none", residual=None):
    """(out, z)."""
    z = x @ w.T
    if bias is not None:
        z = z + bias
    out = func_of(func, z)
    return (out if residual is None else out + residual), z


def func_grad(func, z, d):
    """Gradient of z from that of f(z)."""
    if func == "none":
        return d
    if func == "relu":
        return np.where(z > 0, d, 0.0)
    if func == "gelu":
        return d * (normal_cdf(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi))
    if func == "silu":
        q = sigmoid(z)
        return d * q * (1.0 + z * (1.0 - q))
    g, up = np.split(z, 2, 1)
    q = sigmoid(g)
    return np.concatenate([d * up * q * (1.0 + g * (1.0 - q)), d * g * q], 1)


def linear_grad(x, w, d_out, z=None, func="none"):
    """(d_x, d_w, d_bias, dz)."""
    dz = func_grad(func, z, d_out)
    return dz @ w, dz.T @ x, dz.sum(0), dz
