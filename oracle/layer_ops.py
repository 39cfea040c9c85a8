"""Float64 definitions of the operators around the grouped products (include/mgg/layer_ops.h):
routing with its balance loss, the norms around a block, and Newton-Schulz updates, each with
its gradient where it has one. Inputs are float64 arrays holding the element values."""

from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------------------ routing

def sequence_ranges(T, seq_ends):
    """[(start, end)] of each sequence: ends clamped to [0, T] and raised to the largest
    earlier end; one sequence of all rows without ends."""
    if seq_ends is None:
        return [(0, T)]
    out, start = [], 0
    for e in seq_ends:
        end = max(start, min(max(int(e), 0), T))
        out.append((start, end))
        start = end
    return out


def _log_scores(l, score):
    """log q and log p of each row; a row of -inf has no p (all -inf)."""
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        if score == "softmax":
            m = l.max(axis=1, keepdims=True)
            m = np.where(np.isneginf(m), 0.0, m)
            s = np.exp(l - m).sum(axis=1, keepdims=True)
            logp = np.where(s == 0, -np.inf, l - m - np.log(s))
            return logp, logp
        logq = np.where(l >= 0, -np.log1p(np.exp(-l)), l - np.log1p(np.exp(l)))
        logq = np.where(np.isneginf(l), -np.inf, logq)
        m = logq.max(axis=1, keepdims=True)
        m = np.where(np.isneginf(m), 0.0, m)
        s = np.exp(logq - m).sum(axis=1, keepdims=True)
        return logq, np.where(s == 0, -np.inf, logq - m - np.log(s))


def route(l, k, score="softmax", renormalize=True, scale=1.0, bias=None, seq_ends=None):
    """dict: ids, weights [T, k]; p [T, G]; counts [S, G], tokens [S], balance [S]."""
    T, G = l.shape
    logq, logp = _log_scores(l, score)
    p = np.exp(logp)
    key = l if bias is None else np.where(np.isneginf(l), -np.inf, np.exp(logq) + bias)
    key = np.where(np.isnan(key), -np.inf, key)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k].astype(np.int64)
    taken = np.take_along_axis(key, ids, 1) > -np.inf
    ranges = sequence_ranges(T, seq_ends)
    live = np.zeros(T, bool)
    for a, e in ranges:
        live[a:e] = True
    taken &= live[:, None]
    ql = np.where(taken, np.take_along_axis(logq, np.where(taken, ids, 0), 1), -np.inf)
    if renormalize:
        m = ql.max(axis=1, keepdims=True)
        w = np.exp(ql - np.where(np.isneginf(m), 0.0, m))
        total = w.sum(axis=1, keepdims=True)
        w = w / np.where(total == 0, 1.0, total)
    else:
        w = np.exp(ql)
    ids = np.where(taken, ids, -1)
    S = len(ranges)
    counts = np.zeros((S, G), np.int64)
    balance = np.zeros(S)
    for s, (a, e) in enumerate(ranges):
        chosen = ids[a:e].ravel()
        counts[s] = np.bincount(chosen[chosen >= 0], minlength=G)
        if e > a:
            f = G * counts[s] / (k * (e - a))
            balance[s] = float(np.sum(f * p[a:e].mean(axis=0)))
    return dict(ids=ids, weights=scale * w, p=p, counts=counts,
                tokens=np.array([e - a for a, e in ranges]), balance=balance)


def route_grad(l, ids, counts, tokens, d_weights=None, d_balance=None, score="softmax",
               renormalize=True, scale=1.0, seq_ends=None):
    """(d_logits, magnitude): the gradient, and the sum of the absolute values of the terms
    that it is the difference of."""
    T, G = l.shape
    k = ids.shape[1]
    logq, logp = _log_scores(l, score)
    q, p = np.exp(logq), np.exp(logp)
    not_q = np.ones_like(l) if score == "softmax" else np.where(
        l >= 0, np.exp(-np.abs(l)), 1.0) / (1.0 + np.exp(-np.abs(l)))
    d, mag = np.zeros((T, G)), np.zeros((T, G))
    for s, (a, e) in enumerate(sequence_ranges(T, seq_ends)):
        rows = slice(a, e)
        if e == a:
            continue
        if d_balance is not None:
            b = d_balance[s] * G * counts[s] / (k * float(tokens[s]) ** 2)
            mean = (p[rows] * b).sum(1, keepdims=True)
            d[rows] += p[rows] * (b - mean) * not_q[rows]
            mag[rows] += p[rows] * (np.abs(b) + (p[rows] * np.abs(b)).sum(1, keepdims=True)) \
                * not_q[rows]
        if d_weights is None:
            continue
        for t in range(a, e):
            js = [j for j in range(k) if 0 <= ids[t, j] < G]
            sel = [int(ids[t, j]) for j in js]
            if not sel:
                continue
            dw = d_weights[t, js]
            if renormalize:
                z = np.exp(logq[t, sel] - logq[t, sel].max())
                pi = z / z.sum()
                d[t, sel] += scale * pi * (dw - (pi * dw).sum()) * not_q[t, sel]
                mag[t, sel] += abs(scale) * pi * (np.abs(dw) + (pi * np.abs(dw)).sum()) \
                    * not_q[t, sel]
            elif score == "softmax":
                g, ga = np.zeros(G), np.zeros(G)
                g[sel], ga[sel] = scale * dw, np.abs(scale * dw)
                d[t] += p[t] * (g - (p[t] * g).sum())
                mag[t] += p[t] * (ga + (p[t] * ga).sum())
            else:
                d[t, sel] += scale * dw * q[t, sel] * not_q[t, sel]
                mag[t, sel] += np.abs(scale * dw) * q[t, sel] * not_q[t, sel]
    return d, mag


# -------------------------------------------------------------------- norms of a block

def _sigmoid(v):
    a = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, a) / (1.0 + a)


def _rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def _gate(gate):
    if gate is None:
        return 1.0
    return _sigmoid(gate if gate.ndim == 2 else gate[:, None])


def block_residual_norm(x, y=None, w_after=None, gate=None, scale=None, w_before=None,
                        alpha=1.0, beta=1.0, eps=1e-6):
    """dict: x_out, u and the magnitudes of the terms they are sums of."""
    if y is None:
        out, mag = x, np.abs(x)
    else:
        z = y if w_after is None else y * _rstd(y, eps) * w_after
        z = beta * (1.0 if scale is None else scale) * _gate(gate) * z
        out, mag = alpha * x + z, np.abs(alpha * x) + np.abs(z)
    r = dict(x_out=out, x_mag=mag)
    if w_before is not None:
        f = _rstd(out, eps) * w_before
        r.update(u=out * f, u_mag=mag * np.abs(f))
    return r


def block_residual_norm_grad(x, y=None, d_x=None, d_u=None, w_after=None, gate=None, scale=None,
                             w_before=None, alpha=1.0, beta=1.0, eps=1e-6):
    """{name: (gradient, magnitude)} for x (after the block), y, gate, scale, w_after and
    w_before; sums over rows or columns have the sums of the magnitudes."""
    D = np.zeros_like(x) if d_x is None else d_x
    mag = np.abs(D)
    out = {}
    if w_before is not None:
        r = _rstd(x, eps)
        xh, g = x * r, d_u * w_before
        D = D + r * (g - xh * (g * xh).mean(axis=1, keepdims=True))
        mag = mag + r * (np.abs(g) + np.abs(xh) * np.abs(g * xh).mean(axis=1, keepdims=True))
        out["w_before"] = ((d_u * xh).sum(0), np.abs(d_u * xh).sum(0))
    out["x"] = (alpha * D, abs(alpha) * mag)
    if y is None:
        return out
    ry = 1.0 if w_after is None else _rstd(y, eps)
    yh = y * ry
    wa = 1.0 if w_after is None else w_after
    sc = 1.0 if scale is None else scale
    gv = _gate(gate)
    e, em = beta * D * sc * wa * gv, np.abs(beta * sc * wa * gv) * mag
    if w_after is None:
        out["y"] = (e, em)
    else:
        out["y"] = (ry * (e - yh * (e * yh).mean(axis=1, keepdims=True)),
                    ry * (em + np.abs(yh) * np.abs(em * yh).mean(axis=1, keepdims=True)))
        out["w_after"] = ((beta * D * sc * gv * yh).sum(0),
                          np.abs(beta * mag * sc * gv * yh).sum(0))
    if scale is not None:
        out["scale"] = ((beta * D * gv * yh * wa).sum(0),
                        np.abs(beta * mag * gv * yh * wa).sum(0))
    if gate is not None:
        not_g = _gate(-gate)  # 1 - sigmoid, exact where the sigmoid is next to 1
        d, m = e * yh * not_g, em * np.abs(yh) * not_g
        out["gate"] = (d, m) if gate.ndim == 2 else (d.sum(1), m.sum(1))
    return out


# ---------------------------------------------------------------------- Newton-Schulz

def newton_schulz(X, coeffs, eps=1e-7, scale=1.0, dtype=np.float64):
    """Each matrix of X [G, M, N] after the steps in `coeffs` [(a, b, c)], in `dtype`
    arithmetic."""
    out = []
    for x in X:
        norm = np.sqrt((x.astype(np.float64) ** 2).sum()) + eps
        x = (x / norm).astype(dtype)
        tall = x.shape[0] > x.shape[1]
        x = x.T.copy() if tall else x
        for a, b, c in coeffs:
            a, b, c = dtype(a), dtype(b), dtype(c)
            A = x @ x.T
            x = a * x + (b * A + c * (A @ A)) @ x
        out.append(dtype(scale) * (x.T if tall else x))
    return np.stack(out)
