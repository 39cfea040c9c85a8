"""What is measured of the products of an MoE layer that the grouped ones leave out, and their
plain forms:

  few      a whole MoE layer (both products of the chosen experts, SwiGLU, the weighted sum over
           the experts, the residual) for the few tokens of a decoding step, over weights in the
           grouped products' layouts;
  linear   a dense product with bias, activation and residual in its epilogue (router, shared
           expert, projections), forward and backward.

`own` selects between the plain forms (elementary torch operations in 32 bits or more, rounded
once) and the entry points of moe_grouped_gemm_nt_amd.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of one request, 288 small experts: latency, 25 MB of weights
        dict(name="few_one_token", op="few", T=1, k=8, G=288, H=4096, I=256, weights="fp8",
             scales="ue8m0", gran="block128", out="bf16", residual=True, pad=0.0),
        # a step of 64 requests: most of the 288 experts are read for a row or two
        dict(name="few_batch", op="few", T=64, k=8, G=288, H=4096, I=256, weights="fp8",
             scales="ue8m0", gran="block128", out="bf16", residual=True, pad=0.0),
        # four requests, bf16 weights
        dict(name="few_bf16", op="few", T=4, k=4, G=32, H=2048, I=768, weights="bf16",
             scales="none", gran="none", out="bf16", residual=False, pad=0.0),
        # 32 requests over six wide experts in FP4: about ten rows each
        dict(name="few_fp4", op="few", T=32, k=2, G=6, H=4096, I=2048, weights="fp4",
             scales="ue8m0", gran="block32", out="bf16", residual=True, pad=0.0),
        # odd sizes, places left empty by the router, float32 sums for a later reduction
        dict(name="few_odd", op="few", T=13, k=3, G=12, H=2056, I=200, weights="bf16",
             scales="none", gran="none", out="f32", residual=False, pad=0.2),
        # the shared expert's down projection for one token, onto the residual stream
        dict(name="linear_token", op="linear", way="fwd", M=1, N=7168, K=2048, dtype="bf16",
             func="none", bias=False, residual=True, keep_z=False, out="bf16"),
        # its gate and up projections for a decoding batch
        dict(name="linear_batch", op="linear", way="fwd", M=48, N=4096, K=4096, dtype="bf16",
             func="swiglu", bias=False, residual=False, keep_z=False, out="bf16"),
        # the same for a training micro-batch, the pre-activation kept for the backward
        dict(name="linear_train", op="linear", way="fwd", M=8192, N=4096, K=4096, dtype="bf16",
             func="swiglu", bias=False, residual=False, keep_z=True, out="bf16"),
        # a wide projection onto the residual stream of a training micro-batch
        dict(name="linear_residual", op="linear", way="fwd", M=16384, N=7168, K=2048,
             dtype="bf16", func="none", bias=True, residual=True, keep_z=False, out="bf16"),
        # gradients of a biased layer with gelu: input, weight and bias
        dict(name="linear_grad", op="linear", way="bwd", M=8192, N=4096, K=4096, dtype="bf16",
             func="gelu", bias=True, residual=False, keep_z=True, out="bf16"),
        # the router's product, kept in float32
        dict(name="linear_router", op="linear", way="fwd", M=8192, N=288, K=4096, dtype="f32",
             func="none", bias=True, residual=False, keep_z=False, out="f32"),
        # gradients at odd sizes in float32
        dict(name="linear_odd_grad", op="linear", way="bwd", M=1999, N=777, K=501, dtype="f32",
             func="relu", bias=True, residual=False, keep_z=True, out="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    return _draw_few(rng) if rng.random() < 0.5 else _draw_linear(rng)


def _draw_few(rng):
    weights = rng.choice(["bf16", "fp8", "fp8", "fp4"])
    step = 8 if weights == "bf16" else 128
    gran = {"bf16": "none", "fp4": "block32"}.get(weights) or rng.choice(["block128", "channel"])
    scales = {"bf16": "none", "fp4": "ue8m0"}.get(weights) or rng.choice(["f32", "ue8m0"])
    G = _log_int(rng, 2, 288)
    k = rng.randint(1, min(8, G))
    H = step * _log_int(rng, 2 if step == 128 else 16, 7168 // step)
    most = 3 * 288 * 256 * 4096                       # weights of the largest listed case
    I = step * _log_int(rng, 1 if step == 128 else 8, max(1, min(2048, most // (3 * G * H)) // step))
    T = _log_int(rng, 1, max(1, min(128, 512 * 3 * 256 * 4096 // (k * 3 * I * H))))
    return dict(op="few", T=T, k=k, G=G, H=H, I=I, weights=weights, scales=scales, gran=gran,
                out=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.5,
                pad=rng.choice([0.0, 0.0, 0.2]))


def _draw_linear(rng):
    dtype, way = rng.choice(["bf16", "bf16", "f32"]), rng.choice(["fwd", "fwd", "bwd"])
    func = rng.choice(["none", "relu", "gelu", "silu", "swiglu"])
    N = rng.choice([256, 288, 1536, 2048, 4096, 7168, 2 * _log_int(rng, 8, 3584)])
    K = rng.choice([256, 512, 2048, 4096, 7168, _log_int(rng, 16, 7168)])
    most = (16384 * 7168 * 2048 if dtype == "bf16" else 2 ** 35) // (2 if way == "bwd" else 1)
    M = _log_int(rng, 1, max(1, min(16384, most // (N * K))))
    return dict(op="linear", way=way, M=M, N=N, K=K, dtype=dtype, func=func,
                bias=rng.random() < 0.5, residual=way == "fwd" and rng.random() < 0.5,
                keep_z=way == "bwd" or (func != "none" and rng.random() < 0.5),
                out="f32" if dtype == "f32" else rng.choice(["bf16", "bf16", "f32"])
                if way == "fwd" else "bf16")


# ------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    def uniform(*shape):
        return torch.rand(shape, device="cuda", generator=g)

    if case["op"] == "few":
        T, k, G, H, I = (case[n] for n in ("T", "k", "G", "H", "I"))
        # a router prefers some experts; its weights sum to one
        logits = 1.5 * normal(T, G) + 0.7 * normal(G)
        top, ids = logits.topk(k, 1)
        weights = top.softmax(1)
        if case["pad"] > 0:
            empty = uniform(T, k) < case["pad"]
            ids, weights = torch.where(empty, -1, ids), torch.where(empty, 0.0, weights)
        out = DTYPES[case["out"]]
        w13, s13 = _weights(case, G, 2 * I, H, normal, uniform)
        w2, s2 = _weights(case, G, H, I, normal, uniform)
        return {"case": case, "x": normal(T, H).bfloat16(), "ids": ids.to(torch.int32),
                "weights": weights, "w13": w13, "s13": s13, "w2": w2, "s2": s2,
                "residual": normal(T, H).to(out) if case["residual"] else None}
    M, N, K, dt = case["M"], case["N"], case["K"], DTYPES[case["dtype"]]
    cols = N // 2 if case["func"] == "swiglu" else N
    s = {"case": case, "x": normal(M, K).to(dt), "w": (K ** -0.5 * normal(N, K)).to(dt),
         "bias": 0.5 * normal(N) if case["bias"] else None,
         "residual": normal(M, cols).to(DTYPES[case["out"]]) if case["residual"] else None}
    if case["way"] == "bwd":
        s["z"] = normal(M, N).to(dt) if case["func"] != "none" else None
        s["d_out"] = normal(M, cols).to(dt)
    return s


def _weights(case, G, N, K, normal, uniform):
    """Expert weights of variance 1 / K and their scales, in the grouped products' layouts."""
    if case["weights"] == "bf16":
        return (K ** -0.5 * normal(G, N, K)).bfloat16(), None
    if case["weights"] == "fp8":
        codes = (100.0 * normal(G, N, K)).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
        w = codes.view(torch.uint8)
        shape = (G, -(-N // 128), K // 128) if case["gran"] == "block128" else (G, K // 128, N)
        size = K ** -0.5 / 100.0
    else:
        w = (256.0 * uniform(G, N, K // 2)).to(torch.uint8)
        shape, size = (G, K // 128, N, 4), K ** -0.5 / 2.9  # 2.9: rms of the sixteen codes
    s = size * torch.exp2(uniform(*shape) - 0.5)
    if case["scales"] == "ue8m0":
        s = (s.log2().round() + 127.0).to(torch.uint8)
    return w, s


# ------------------------------------------------------------------------------ one pass

def run(state):
    if state["case"]["op"] == "few":
        return _few_own(state) if own else _few(state)
    return _linear_own(state) if own else _linear(state)


def _few_own(s):
    import moe_grouped_gemm_nt_amd as mgg
    c = s["case"]
    return mgg.moe_few_tokens(s["x"], s["ids"], s["weights"], s["w13"], s["w2"], s["s13"], s["s2"],
                              sfb_gran=None if c["gran"] == "none" else c["gran"],
                              residual=s["residual"], out_dtype=DTYPES[c["out"]])


def _linear_own(s):
    import moe_grouped_gemm_nt_amd as mgg
    c = s["case"]
    if c["way"] == "fwd":
        return mgg.linear_act(s["x"], s["w"], s["bias"], func=c["func"], residual=s["residual"],
                              keep_z=c["keep_z"], out_dtype=DTYPES[c["out"]])
    return mgg.linear_act_backward(s["x"], s["w"], s["d_out"], s["z"], func=c["func"],
                                   need_bias=c["bias"])


# -------------------------------------------------------------------------- plain forms

def _values(case, w, s):
    """Float32 values of weights [.., N, K]."""
    if case["weights"] == "bf16":
        return w.float()
    s = torch.exp2(s.float() - 127.0) if case["scales"] == "ue8m0" else s
    if case["weights"] == "fp4":
        code = torch.arange(256, device=w.device)  # the two values of each byte
        pairs = torch.tensor(E2M1, device=w.device)[torch.stack([code & 15, code >> 4], 1)]
        v = pairs[w.int()]
        P, N = w.shape[0], w.shape[1]
        s = s.permute(0, 2, 1, 3).reshape(P, N, -1, 1)
        return (v.reshape(P, N, s.shape[2], 32) * s).reshape(P, N, -1)
    v = w.view(torch.float8_e4m3fn).float()
    P, N, K = v.shape
    if case["gran"] == "channel":
        s = s.transpose(1, 2)
    else:
        s = s.repeat_interleave(128, 1)[:, :N]
    return (v.reshape(P, N, K // 128, 128) * s[..., None]).reshape(P, N, K)


def _few(s):
    c, x = s["case"], s["x"].float()
    (T, H), k, I = x.shape, c["k"], c["I"]
    at = s["ids"].long().clamp(min=0).reshape(-1)
    w13 = _values(c, s["w13"][at], None if s["s13"] is None else s["s13"][at])
    z = torch.matmul(w13, x.repeat_interleave(k, 0)[..., None])[..., 0]
    h = z[:, :I] / (1.0 + (-z[:, :I]).exp()) * z[:, I:]
    w2 = _values(c, s["w2"][at], None if s["s2"] is None else s["s2"][at])
    y = torch.matmul(w2, h[..., None]).view(T, k, H)
    y = torch.where((s["ids"] >= 0)[..., None], y * s["weights"][..., None], 0.0).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[c["out"]])


def _sigmoid(v):
    return 1.0 / (1.0 + (-v).exp())


def _normal_cdf(v):
    return 0.5 * torch.erfc(v * -math.sqrt(0.5))


def _linear(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    func, x, w = c["func"], s["x"].float(), s["w"].float()
    if c["way"] == "bwd":
        d = s["d_out"].float()
        if func != "none":
            z = s["z"].float()
        if func == "relu":
            d = torch.where(z > 0, d, 0.0)
        elif func == "gelu":
            d = d * (_normal_cdf(z) + z * (-0.5 * z * z).exp() / math.sqrt(2.0 * math.pi))
        elif func == "silu":
            q = _sigmoid(z)
            d = d * (q * (1.0 + z * (1.0 - q)))
        elif func == "swiglu":
            a, u = z.chunk(2, 1)
            q = _sigmoid(a)
            d = torch.cat([d * u * (q * (1.0 + a * (1.0 - q))), d * (a * q)], 1)
        d_w = torch.matmul(d.t(), x)
        return (torch.matmul(d, w).to(dt), d_w.to(dt),
                d.sum(0, dtype=torch.float64).float() if c["bias"] else None)
    z = torch.matmul(x, w.t())
    if s["bias"] is not None:
        z = z + s["bias"]
    y = z
    if func == "relu":
        y = torch.where(z > 0, z, 0.0)
    elif func == "gelu":
        y = z * _normal_cdf(z)
    elif func == "silu":
        y = z * _sigmoid(z)
    elif func == "swiglu":
        a, u = z.chunk(2, 1)
        y = a * _sigmoid(a) * u
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(DTYPES[c["out"]])
    return (y, z.to(dt)) if c["keep_z"] else y


# ------------------------------------------------------------------------------ the work

def work(case):
    if case["op"] == "few":
        T, k, G, H, I = (case[n] for n in ("T", "k", "G", "H", "I"))
        experts = G * (1.0 - (1.0 - k / G) ** T)      # the different ones among the chosen
        elements = 3 * H * I
        weight = {"bf16": 2.0, "fp8": 1.0, "fp4": 0.5 + 1.0 / 32.0}[case["weights"]] * elements
        out = {"bf16": 2, "f32": 4}[case["out"]]
        return {"bytes": int(experts * weight) + T * H * (2 + out * (1 + case["residual"])) + T * k * 8,
                "flops": 2 * T * k * elements}
    M, N, K = case["M"], case["N"], case["K"]
    b, out = (2 if case[n] == "bf16" else 4 for n in ("dtype", "out"))
    cols = N // 2 if case["func"] == "swiglu" else N
    if case["way"] == "fwd":
        move = (M * K + N * K) * b + M * cols * out * (1 + case["residual"])
        move += M * N * b * case["keep_z"] + 4 * N * case["bias"]
        return {"bytes": move, "flops": 2 * M * N * K}
    move = 2 * (M * K + N * K) * b + M * cols * b + 4 * N * case["bias"]
    move += M * N * b * (case["func"] != "none")
    return {"bytes": move, "flops": 4 * M * N * K}


# --------------------------------------------------- the definitions in 64 bits, for checks

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_few(case, s) if case["op"] == "few" else _exact_linear(case, s)


def _exact_weights(c, w, s):
    """Float64 values of one expert's weights [N, K]."""
    if c["weights"] == "bf16":
        return w.double()
    K = w.shape[1] * (2 if c["weights"] == "fp4" else 1)
    s = s.double() if c["scales"] == "f32" else torch.pow(2.0, s.double() - 127.0)
    k = torch.arange(K, device=w.device)
    n = torch.arange(w.shape[0], device=w.device)
    if c["weights"] == "fp4":
        code = (w[:, k // 2].long() >> (4 * (k % 2))) & 15
        low, exponent = (code & 1).double(), (code >> 1) & 3
        size = torch.where(exponent == 0, 0.5 * low,
                           (1.0 + 0.5 * low) * torch.pow(2.0, exponent.double() - 1.0))
        value = torch.where(code >= 8, -size, size)
        return value * s[k // 128][:, n].permute(1, 0, 2).gather(
            2, ((k % 128) // 32).expand(len(n), K)[..., None])[..., 0]
    value = w.view(torch.float8_e4m3fn).double()
    if c["gran"] == "channel":
        return value * s[k // 128].t()
    return value * s[n // 128][:, k // 128]


def _exact_few(c, s):
    x, ids = s["x"].double(), s["ids"].tolist()
    out = torch.zeros_like(x) if s["residual"] is None else s["residual"].double()
    places = {}
    for t, row in enumerate(ids):
        for j, e in enumerate(row):
            if 0 <= e < c["G"]:
                places.setdefault(e, []).append((t, j))
    for e, at in places.items():
        t, j = (torch.tensor(v, device=x.device) for v in zip(*at))
        z = x[t] @ _exact_weights(c, s["w13"][e], None if s["s13"] is None else s["s13"][e]).t()
        a, u = z.split(c["I"], 1)
        h = a * torch.special.expit(a) * u
        y = h @ _exact_weights(c, s["w2"][e], None if s["s2"] is None else s["s2"][e]).t()
        out.index_add_(0, t, y * s["weights"][t, j].double()[:, None])
    return out


def _exact_func(func, z):
    if func == "none":
        return z
    if func == "relu":
        return z.clamp(min=0.0)
    if func == "gelu":
        return torch.nn.functional.gelu(z)
    if func == "silu":
        return z * torch.special.expit(z)
    a, u = z.split(z.shape[1] // 2, 1)
    return a * torch.special.expit(a) * u


def _exact_linear(c, s):
    x, w = s["x"].double(), s["w"].double()
    if c["way"] == "bwd":
        d = s["d_out"].double()
        if c["func"] != "none":
            z = s["z"].double().requires_grad_()
            d = torch.autograd.grad(_exact_func(c["func"], z), z, d)[0]
        return d @ w, d.t() @ x, d.sum(0) if c["bias"] else None
    z = x @ w.t()
    if s["bias"] is not None:
        z = z + s["bias"].double()
    y = _exact_func(c["func"], z)
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return (y, z) if c["keep_z"] else y
