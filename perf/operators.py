"""What is measured of the operators that stand around the grouped products of an MoE layer
in training and serving, and their plain forms:

  route     top-k routing of tokens to experts with per-expert counts and a balance loss per
            sequence (forward), and the gradient of the logits (backward);
  norm      the norm before a block, and the norm after it fused with its gate, residual
            scale, residual sum and the next block's norm, forward and backward;
  ns        the orthogonalised update of every expert's weight gradient by Newton-Schulz
            products, all experts in one call.

`own` selects between the plain forms (elementary torch operations in 32 bits or more, rounded
once) and the entry points of moe_grouped_gemm_nt_amd.
"""

import math

import torch

own = False

EPS = 1e-6                             # of the norms
NS_EPS = 1e-7                          # added to the Frobenius norm
NS_COEFFS = (3.4445, -4.7750, 2.0315)  # the usual odd quintic, five steps of it
NS_STEPS = 5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of four requests, 288 experts: latency alone
        dict(name="route_decode", op="route", way="serve", T=4, G=288, k=8, S=1, dtype="bf16",
             score="softmax", renorm=True, bias=False, pad=0.0),
        # one training micro-batch of 16 packed sequences with a padded end, 288 experts
        dict(name="route_train", op="route", way="fwd", T=65536, G=288, k=8, S=16, dtype="f32",
             score="softmax", renorm=True, bias=False, pad=0.03),
        # sigmoid scores, selection by score plus a balancing bias; odd token count
        dict(name="route_sigmoid_bias", op="route", way="fwd", T=16381, G=288, k=6, S=1,
             dtype="bf16", score="sigmoid", renorm=True, bias=True, pad=0.0),
        # gradient of the logits for the training micro-batch
        dict(name="route_train_grad", op="route", way="bwd", T=65536, G=288, k=8, S=16,
             dtype="f32", score="softmax", renorm=True, bias=False, pad=0.03),
        # end of one block and start of the next for a single token
        dict(name="norm_decode", op="norm", way="fwd", T=1, H=7168, dtype="bf16", gate="token",
             scale=True, after=True, before=True),
        # the same for a training micro-batch, gated per token
        dict(name="norm_train", op="norm", way="fwd", T=16384, H=7168, dtype="bf16",
             gate="token", scale=True, after=True, before=True),
        # its gradients: activations, gate, residual scale and both norm weights
        dict(name="norm_train_grad", op="norm", way="bwd", T=16384, H=7168, dtype="bf16",
             gate="token", scale=True, after=True, before=True),
        # float32 activations of odd width, gated per element
        dict(name="norm_odd_grad", op="norm", way="bwd", T=4099, H=2047, dtype="f32",
             gate="element", scale=True, after=True, before=True),
        # eight small square experts: launch-bound
        dict(name="ns_small", op="ns", G=8, M=256, N=256, dtype="f32"),
        # the weight gradients of four 2048 x 2048 experts, as the K-grouped product writes them
        dict(name="ns_wgrad", op="ns", G=4, M=2048, N=2048, dtype="f32"),
        # six wide experts kept in bf16
        dict(name="ns_wide_bf16", op="ns", G=6, M=1536, N=4096, dtype="bf16"),
        # tall matrices of odd sizes
        dict(name="ns_tall_odd", op="ns", G=3, M=1999, N=501, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "norm", "norm", "ns"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "route":
        T, G = _log_int(rng, 1, 65536), _log_int(rng, 4, 288)
        way = rng.choice(["serve", "fwd", "bwd"])
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, way=way, T=T, G=G, k=rng.randint(1, min(8, G)),
                    S=1 if way == "serve" else rng.randint(1, 16), dtype=dtype, score=score,
                    renorm=rng.random() < 0.7, bias=score == "sigmoid" and rng.random() < 0.5,
                    pad=0.0 if way == "serve" else rng.choice([0.0, 0.1]))
    if op == "norm":
        H = rng.choice([256, 1536, 2048, 4096, 7168, _log_int(rng, 64, 7168)])
        T = _log_int(rng, 1, 16384 * 7168 // 2 // H if dtype == "f32" else 16384 * 7168 // H)
        before = rng.random() < 0.8
        return dict(op=op, way=rng.choice(["fwd", "bwd"]), T=min(T, 65536), H=H, dtype=dtype,
                    gate=rng.choice(["none", "token", "element"]), scale=rng.random() < 0.6,
                    after=rng.random() < 0.8 or not before, before=before)
    M, N = _log_int(rng, 32, 2048), _log_int(rng, 32, 2048)
    return dict(op=op, G=rng.randint(1, 4), M=M, N=N, dtype=dtype)


# ------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    if case["op"] == "route":
        T, G, k, S = (case[n] for n in ("T", "G", "k", "S"))
        # a router prefers some experts; its logits spread over a few units
        logits = (1.5 * normal(T, G) + 0.7 * normal(G)).to(dt)
        s = {"case": case, "logits": logits,
             "bias": 0.05 * normal(G) if case["bias"] else None, "seq_ends": None}
        if S > 1 or case["pad"] > 0:
            # ragged sequences, back to back; rows past the last end are padding
            cuts = torch.rand(S, device="cuda", generator=g) + 0.2
            ends = (cuts.cumsum(0) / cuts.sum() * (T * (1.0 - case["pad"]))).to(torch.int32)
            s["seq_ends"] = ends
        if case["way"] == "bwd":
            ids, _, counts, tokens, _ = _route_plain(case, logits, s["bias"], s["seq_ends"])
            s.update(ids=ids, counts=counts, tokens=tokens, d_weights=normal(T, k),
                     d_balance=0.01 * (1.0 + torch.rand(S, device="cuda", generator=g)))
        return s
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s = {"case": case, "x": normal(T, H).to(dt),
             "y": (0.5 * normal(T, H)).to(dt) if _has_block(case) else None,
             "gate": None, "scale": None, "w_after": None, "w_before": None}
        if case["gate"] == "token":
            s["gate"] = normal(T).to(dt)
        elif case["gate"] == "element":
            s["gate"] = normal(T, H).to(dt)
        if case["scale"]:
            s["scale"] = 0.3 + 0.05 * normal(H)
        if case["after"]:
            s["w_after"] = 1.0 + 0.1 * normal(H)
        if case["before"]:
            s["w_before"] = 1.0 + 0.1 * normal(H)
        if case["way"] == "bwd":
            s["d_x"] = normal(T, H).to(dt)
            s["d_u"] = normal(T, H).to(dt) if case["before"] else None
        return s
    G, M, N = case["G"], case["M"], case["N"]
    # a momentum of gradients: a few strong directions over noise, small in value
    r = 4
    low = torch.matmul(normal(G, M, r), normal(G, r, N))
    return {"case": case, "X": (1e-3 * (normal(G, M, N) + 0.5 * low)).to(dt)}


def _has_block(case):
    """Whether a block's output joins: without it the call is the norm before a block."""
    return case["after"] or case["gate"] != "none" or case["scale"]


# ------------------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if case["op"] == "route":
        return _route_own(state) if own else _route(state)
    if case["op"] == "norm":
        return _norm_own(state) if own else _norm(state)
    if own:
        import moe_grouped_gemm_nt_amd as mgg
        return mgg.grouped_newton_schulz(state["X"], coeffs=NS_COEFFS, steps=NS_STEPS, eps=NS_EPS)
    return _ns_plain(state["X"])


def _route_own(s):
    import moe_grouped_gemm_nt_amd as mgg
    c = s["case"]
    how = dict(score=c["score"], renormalize=c["renorm"])
    if c["way"] == "serve":
        return mgg.route_topk(s["logits"], c["k"], bias=s["bias"], balance=False, **how)
    if c["way"] == "fwd":
        return mgg.route_topk(s["logits"], c["k"], bias=s["bias"], seq_ends=s["seq_ends"], **how)
    return mgg.route_topk_backward(s["logits"], s["ids"], s["counts"], s["tokens"],
                                   d_weights=s["d_weights"], d_balance=s["d_balance"],
                                   seq_ends=s["seq_ends"], **how)


def _norm_own(s):
    import moe_grouped_gemm_nt_amd as mgg
    c = s["case"]
    if not _has_block(c):
        if c["way"] == "fwd":
            return mgg.block_norm(s["x"], s["w_before"], eps=EPS)
        return mgg.block_norm_backward(s["x"], s["w_before"], s["d_u"], d_x=s["d_x"], eps=EPS)
    how = dict(w_after=s["w_after"], gate=s["gate"], scale=s["scale"], w_before=s["w_before"],
               eps=EPS)
    if c["way"] == "fwd":
        return mgg.block_residual_norm(s["x"], s["y"], **how)
    return mgg.block_residual_norm_backward(s["x"], s["y"], d_x=s["d_x"], d_u=s["d_u"], **how)


# -------------------------------------------------------------------------- plain forms

def _segments(T, S, ends, device):
    """Sequence of each row (S for padding rows)."""
    if ends is None:
        return torch.zeros(T, dtype=torch.int64, device=device)
    rows = torch.arange(T, device=device)
    return (rows[:, None] >= ends[None, :]).sum(1)


def _softmax(l):
    e = (l - l.amax(1, keepdim=True)).exp()
    return e / e.sum(1, keepdim=True)


def _route_plain(c, logits, bias, ends):
    """ids, weights, counts, tokens and balance loss."""
    T, G, k, S = logits.shape[0], c["G"], c["k"], c["S"]
    l = logits.float()
    if c["score"] == "softmax":
        score = prob = _softmax(l)
        key = l  # the order of the logits is the order of their softmax
    else:
        score = 1.0 / (1.0 + (-l).exp())
        prob = score / score.sum(1, keepdim=True)
        # selection compares sums: in 64 bits, so that near ones fall the same way
        key = l if bias is None else 1.0 / (1.0 + (-l.double()).exp()) + bias.double()
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    if c["way"] == "serve":
        return ids.to(torch.int32), w
    seg = _segments(T, S, ends, l.device)
    live = seg < S
    ids = torch.where(live[:, None], ids, -1)
    w = torch.where(live[:, None], w, 0.0)
    member = seg[:, None] == torch.arange(S, device=l.device)[None, :]
    tokens = member.sum(0)
    slot = torch.where(live[:, None], seg[:, None] * G + ids, S * G).reshape(-1)
    counts = torch.zeros(S * G + 1, dtype=torch.int64, device=l.device)
    counts = counts.scatter_add_(0, slot, torch.ones_like(slot))[:-1].reshape(S, G)
    mean = torch.matmul(member.double().t().contiguous(), prob.double())  # long sums
    n = tokens.double().clamp(min=1.0)[:, None]
    balance = (G / k * (counts.double() / n) * (mean / n)).sum(1)
    return (ids.to(torch.int32), w, counts.to(torch.int32), tokens.to(torch.int32),
            balance.float())


def _route(s):
    c = s["case"]
    if c["way"] != "bwd":
        return _route_plain(c, s["logits"], s["bias"], s["seq_ends"])
    T, G, k, S = s["logits"].shape[0], c["G"], c["k"], c["S"]
    l, dw = s["logits"].float(), s["d_weights"]
    seg = _segments(T, S, s["seq_ends"], l.device)
    live = (seg < S)[:, None]
    at = s["ids"].long().clamp(min=0)
    n = s["tokens"].float().clamp(min=1.0)
    per_count = G / k * s["d_balance"] / (n * n)
    d_prob = (per_count[:, None] * s["counts"].float())[seg.clamp(max=S - 1)]
    if c["score"] == "softmax":
        score = prob = _softmax(l)
    else:
        score = 1.0 / (1.0 + (-l).exp())
        prob = score / score.sum(1, keepdim=True)
    chosen = score.gather(1, at)
    d_chosen = dw
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True)
        d_chosen = (dw - (dw * chosen / total).sum(1, keepdim=True)) / total
    d_score = torch.zeros_like(l).scatter_(1, at, d_chosen)
    if c["score"] == "softmax":
        d_score = d_score + d_prob
        d = prob * (d_score - (prob * d_score).sum(1, keepdim=True))
    else:
        mean = (prob * d_prob).sum(1, keepdim=True)
        d_score = d_score + (d_prob - mean) / score.sum(1, keepdim=True)
        d = d_score * score * (1.0 - score)
    return torch.where(live, d, 0.0).to(s["logits"].dtype)


def _rstd(v):
    return ((v * v).mean(1, keepdim=True) + EPS).rsqrt()


def _gate(g):
    return 1.0 if g is None else 1.0 / (1.0 + (-(g.float() if g.dim() == 2 else g.float()[:, None])).exp())


def _norm(s):
    c, dt = s["case"], s["x"].dtype
    x = s["x"].float()
    if not _has_block(c):
        rx = _rstd(x)
        if c["way"] == "fwd":
            return (x * rx * s["w_before"]).to(dt)
        du = s["d_u"].float()
        g, hat = du * s["w_before"], x * rx
        d = s["d_x"].float() + rx * (g - hat * (g * hat).mean(1, keepdim=True))
        return d.to(dt), (du * hat).sum(0)
    y = s["y"].float()
    gate = _gate(s["gate"])
    scale = 1.0 if s["scale"] is None else s["scale"]
    wa = 1.0 if s["w_after"] is None else s["w_after"]
    ry = _rstd(y) if s["w_after"] is not None else 1.0
    yhat = y * ry
    if c["way"] == "fwd":
        out = x + scale * gate * (yhat * wa)
        u = (out * _rstd(out) * s["w_before"]).to(dt) if c["before"] else None
        return out.to(dt), u
    # here x is the residual stream after the block
    d, d_before = s["d_x"].float(), None
    if c["before"]:
        du, rx = s["d_u"].float(), _rstd(x)
        g, hat = du * s["w_before"], x * rx
        d = d + rx * (g - hat * (g * hat).mean(1, keepdim=True))
        d_before = (du * hat).sum(0)
    d_gate = d_scale = d_after = None
    if s["gate"] is not None:
        d_gate = d * scale * (yhat * wa) * gate * (1.0 - gate)
        d_gate = (d_gate if s["gate"].dim() == 2 else d_gate.sum(1)).to(dt)
    if s["scale"] is not None:
        d_scale = (d * gate * (yhat * wa)).sum(0)
    d_yhat = d * scale * gate * wa
    d_y = d_yhat
    if s["w_after"] is not None:
        d_after = (d * scale * gate * yhat).sum(0)
        d_y = ry * (d_yhat - yhat * (d_yhat * yhat).mean(1, keepdim=True))
    return d.to(dt), d_y.to(dt), d_gate, d_scale, d_after, d_before


def _ns_plain(X):
    dt, (a, b, c) = X.dtype, NS_COEFFS
    x = X.float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / ((x * x).sum((1, 2), keepdim=True, dtype=torch.float64).sqrt() + NS_EPS).float()
    for _ in range(NS_STEPS):
        A = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * A + c * torch.bmm(A, A), x)
    if tall:
        x = x.transpose(1, 2).contiguous()
    return x.to(dt)


# ------------------------------------------------------------------------------ the work

def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "route":
        T, G, k, S = (case[n] for n in ("T", "G", "k", "S"))
        move = T * G * b + T * k * 8 + (4 * G if case["bias"] else 0)
        if case["way"] == "fwd":
            move += S * (G + 3) * 4
        if case["way"] == "bwd":
            move += T * G * b + S * (G + 3) * 4
        return {"bytes": move, "flops": 8 * T * G}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        gate = {"none": 0, "token": T, "element": T * H}[case["gate"]]
        vectors = H * 4 * (case["scale"] + case["after"] + case["before"])
        tensors = 1 + _has_block(case)                       # x and y
        if case["way"] == "fwd":
            tensors += _has_block(case) + case["before"]     # the new stream and its norm
            return {"bytes": tensors * T * H * b + gate * b + vectors, "flops": 12 * T * H}
        tensors += 1 + case["before"] + 1 + _has_block(case)  # both gradients in, both out
        return {"bytes": tensors * T * H * b + 2 * gate * b + 2 * vectors, "flops": 30 * T * H}
    G, M, N = case["G"], case["M"], case["N"]
    m, n = min(M, N), max(M, N)
    # per step: half of X X^T and of A A (both symmetric), and all of (bA + cAA) X
    return {"bytes": 2 * G * M * N * b,
            "flops": G * NS_STEPS * (m * m * n + m * m * m + 2 * m * m * n)}


# --------------------------------------------------- the definitions in 64 bits, for checks

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "norm": _exact_norm, "ns": _exact_ns}[case["op"]](case, s)


def _exact_route(c, s):
    l = s["logits"].double().requires_grad_(c["way"] == "bwd")
    T, G, k, S = l.shape[0], c["G"], c["k"], c["S"]
    if c["score"] == "softmax":
        score = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
        prob = score
    else:
        score = torch.special.expit(l)
        prob = torch.exp(torch.log(score) - torch.log(score.sum(1, keepdim=True)))
    if c["way"] == "bwd":
        ids = s["ids"].long()
    else:
        # place in the order: how many experts come before it (a lower index wins a tie)
        key = l if s["bias"] is None else score + s["bias"].double()
        left, ids = key.clone(), []
        for _ in range(k):
            top = left.amax(1, keepdim=True)
            first = torch.where(left == top, torch.arange(G, device=l.device), G).amin(1)
            ids.append(first)
            left.scatter_(1, first[:, None], -math.inf)
        ids = torch.stack(ids, 1)
    w = torch.gather(score, 1, ids.clamp(min=0))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    if c["way"] == "serve":
        return ids.to(torch.int32), w
    ends = [T] if s["seq_ends"] is None else s["seq_ends"].tolist()
    starts = [0] + ends[:-1]
    losses, counts, tokens = [], [], []
    for a, e in zip(starts, ends):
        chosen = ids[a:e].reshape(-1)
        n = e - a
        f = torch.bincount(chosen, minlength=G) if n else torch.zeros(G, dtype=torch.int64, device=l.device)
        counts.append(f)
        tokens.append(n)
        mean = prob[a:e].mean(0) if n else torch.zeros(G, dtype=torch.float64, device=l.device)
        losses.append(torch.dot(f.double() * (G / (k * max(n, 1))), mean))
    losses = torch.stack(losses)
    live = (torch.arange(T, device=l.device) < ends[-1])[:, None]
    if c["way"] == "bwd":
        total = (w * live * s["d_weights"].double()).sum() + (losses * s["d_balance"].double()).sum()
        return torch.autograd.grad(total, l)[0]
    return (torch.where(live, ids, -1).to(torch.int32), w * live,
            torch.stack(counts).to(torch.int32),
            torch.tensor(tokens, dtype=torch.int32, device=l.device), losses)


def _exact_rms(v, w):
    return v / torch.sqrt(v.pow(2).sum(1, keepdim=True) / v.shape[1] + EPS) * w


def _exact_norm(c, s):
    names = [n for n in ("x", "y", "gate", "scale", "w_after", "w_before") if s[n] is not None]
    v = dict.fromkeys(("y", "gate", "scale", "w_after", "w_before"))
    v.update({n: s[n].double().requires_grad_(c["way"] == "bwd") for n in names})

    def block():
        z = v["y"] if v["w_after"] is None else _exact_rms(v["y"], v["w_after"])
        if v["gate"] is not None:
            g = torch.special.expit(v["gate"])
            z = z * (g if g.dim() == 2 else g.unsqueeze(1))
        return z if v["scale"] is None else z * v["scale"]

    if c["way"] == "fwd":
        if not _has_block(c):
            return _exact_rms(v["x"], v["w_before"])
        out = v["x"] + block()
        return out, _exact_rms(out, v["w_before"]) if c["before"] else None
    # the stream's gradient first, then through the block at that gradient
    wanted = [v["x"]] + ([v["w_before"]] if c["before"] else [])
    total = (v["x"] * s["d_x"].double()).sum()
    if c["before"]:
        total = total + (_exact_rms(v["x"], v["w_before"]) * s["d_u"].double()).sum()
    got = torch.autograd.grad(total, wanted)
    d_before = got[1] if c["before"] else None
    if not _has_block(c):
        return got[0], d_before
    inner = [n for n in ("y", "gate", "scale", "w_after") if v[n] is not None]
    d = dict(zip(inner, torch.autograd.grad((block() * got[0]).sum(), [v[n] for n in inner])))
    return got[0], d["y"], d.get("gate"), d.get("scale"), d.get("w_after"), d_before


def _exact_ns(c, s):
    a, b, q = NS_COEFFS
    out = []
    for x in s["X"].double():
        x = x / (torch.linalg.vector_norm(x) + NS_EPS)
        small = x.shape[0] <= x.shape[1]
        eye = torch.eye(min(x.shape), dtype=torch.float64, device=x.device)
        for _ in range(NS_STEPS):
            xt = x.t().contiguous()
            gram = x @ xt if small else xt @ x
            poly = a * eye + gram @ (b * eye + q * gram)
            x = poly @ x if small else x @ poly
        out.append(x)
    return torch.stack(out)
