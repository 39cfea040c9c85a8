"""The norms around a block on the GPU against the float64 definitions.

Tolerances count float32 roundings, u = 2^-24, relative to the sum of the absolute values of an
output's terms (`mag` of the definitions). A row's sum has at most 64 addends a thread, six
halvings of a wave and 16 waves: under 96 roundings of a sum of terms that are themselves
rounded twice; a norm's factor and the products add about 20. One sum enters a forward
value, two a backward one: C = 128 and 256. A parameter's gradient adds the rows of a group one
after another: one more rounding for each, at most T. bf16 outputs add half a step, 2^-8."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg
from oracle import layer_ops as ref
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
EPS = 1e-5


def make(T, H, dtype, gate=None, scale=True, after=True, before=True, param=torch.float32,
         seed=0):
    g = torch.Generator().manual_seed(seed + 13 * H + T)

    def n(*shape, mul=1.0, add=0.0, dt=dtype):
        return (add + mul * torch.randn(shape, generator=g)).to(dt)

    return dict(x=n(T, H), y=n(T, H, mul=0.5),
                gate=None if gate is None else n(*((T,) if gate == "token" else (T, H))),
                scale=n(H, mul=0.1, add=0.3, dt=param) if scale else None,
                w_after=n(H, mul=0.1, add=1.0, dt=param) if after else None,
                w_before=n(H, mul=0.1, add=1.0, dt=param) if before else None,
                d_x=n(T, H), d_u=n(T, H) if before else None)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def dev(t):
    return None if t is None else t.to(DEV)


def close(got, want, mag, c, name):
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else U
    off = np.abs(f64(got) - want)
    bound = c * U * mag + half * np.abs(want) + 1e-37
    assert np.isfinite(f64(got)).all(), name
    assert (off <= bound).all(), (name, (off / bound).max())


def params(s, **kw):
    return dict(w_after=s["w_after"], gate=s["gate"], scale=s["scale"], w_before=s["w_before"],
                eps=EPS, **kw)


def check(s, alpha=1.0, beta=1.0, use_dx=True):
    kw = params(s, alpha=alpha, beta=beta)
    on = {k: dev(v) if torch.is_tensor(v) else v for k, v in kw.items()}
    ref_kw = {k: f64(v) if torch.is_tensor(v) else v for k, v in kw.items()}
    x, y = dev(s["x"]), dev(s["y"])
    out, u = mgg.block_residual_norm(x, y, **on)
    r = ref.block_residual_norm(f64(s["x"]), f64(s["y"]), **ref_kw)
    close(out, r["x_out"], r["x_mag"], 128, "x_out")
    assert (u is None) == (s["w_before"] is None)
    if u is not None:
        close(u, r["u"], r["u_mag"], 128, "u")
    dx = s["d_x"] if use_dx else None
    got = mgg.block_residual_norm_backward(out, y, dev(dx), dev(s["d_u"]), **on)
    want = ref.block_residual_norm_grad(f64(out), f64(s["y"]), f64(dx), f64(s["d_u"]), **ref_kw)
    T = s["x"].shape[0]
    names = ("x", "y", "gate", "scale", "w_after", "w_before")
    for name, g in zip(names, got):
        assert (g is None) == (name not in want), name
        if g is not None:
            c = 256 + (T if name in names[3:] else 0)
            close(g, *want[name], c, name)
    return (out, u) + got


WIDTHS = [1, 7, 8, 64, 255, 256, 511, 1024, 2047, 2048, 4096, 7168, 8192, 8200, 16384, 16391, 32768]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_widths(H, dtype):
    say(f"block norm width {H} {dtype}")
    for T, gate in ((1, "token"), (13, "element"), (3, None)):
        check(make(T, H, dtype, gate, param=torch.float32))


@pytest.mark.parametrize("gate", [None, "token", "element"])
@pytest.mark.parametrize("scale", [True, False])
@pytest.mark.parametrize("after", [True, False])
@pytest.mark.parametrize("before", [True, False])
def test_parts(gate, scale, after, before):
    say(f"block norm parts {gate} {scale} {after} {before}")
    for dtype, param, H in ((torch.bfloat16, torch.bfloat16, 776), (torch.float32, torch.float32, 301),
                            (torch.bfloat16, torch.float32, 2500)):
        s = make(37, H, dtype, gate, scale, after, before, param)
        check(s, alpha=0.75, beta=-1.5)
        if before:
            check(s, use_dx=False)


@pytest.mark.parametrize("T", [0, 2, 70, 1025, 5000])
def test_row_counts(T):
    say(f"block norm rows {T}")
    for H in (96, 2304):
        check(make(T, H, torch.float32, "token"))


@pytest.mark.parametrize("H", [5, 640, 7168, 20000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_alone(H, dtype):
    say(f"block norm alone {H} {dtype}")
    for T in (0, 1, 29):
        s = make(T, H, dtype)
        x, w = dev(s["x"]), dev(s["w_before"])
        u = mgg.block_norm(x, w, eps=EPS)
        r = ref.block_residual_norm(f64(s["x"]), w_before=f64(s["w_before"]), eps=EPS)
        close(u, r["u"], r["u_mag"], 128, "u")
        for dx in (s["d_x"], None):
            d, dw = mgg.block_norm_backward(x, w, dev(s["d_u"]), dev(dx), eps=EPS)
            want = ref.block_residual_norm_grad(f64(s["x"]), None, f64(dx), f64(s["d_u"]),
                                                w_before=f64(s["w_before"]), eps=EPS)
            close(d, *want["x"], 256, "x")
            close(dw, *want["w_before"], 256 + T, "w")


def test_rows_of_zeros_and_extremes():
    """Zero rows (eps alone under the root), tiny and large values, saturated gates."""
    say("block norm extremes")
    for dtype in (torch.bfloat16, torch.float32):
        for gate in ("token", "element"):
            s = make(12, 300, dtype, gate)
            s["y"][0] = 0
            s["x"][1] = 0
            s["y"][1] = 0
            s["y"][2] *= 1e-12
            s["x"][3] *= 1e12
            s["gate"][4] = 60.0
            s["gate"][5] = -60.0
            s["gate"][6] = -1000.0
            s["gate"][7] = 1000.0
            check(s)


def test_nan_stays_in_its_row():
    say("block norm nan")
    s = make(9, 520, torch.float32, "token")
    x, y = dev(s["x"]), dev(s["y"])
    kw = {k: dev(v) if torch.is_tensor(v) else v for k, v in params(s).items()}
    a = mgg.block_residual_norm(x, y, **kw)
    y2 = y.clone()
    y2[4, 100] = float("nan")
    b = mgg.block_residual_norm(x, y2, **kw)
    keep = [t for t in range(9) if t != 4]
    for p, q in zip(a, b):
        assert torch.equal(p[keep], q[keep]) and torch.isnan(q[4]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,start,pad", [(64, 1, 2), (300, 3, 0), (2048, 1, 6), (2600, 5, 1)])
def test_strided_and_shifted_rows(dtype, H, start, pad):
    say(f"block norm strided {dtype} {H} {start}")
    T = 11
    s = make(T, H, dtype, "element")
    on = {}
    for n in ("x", "y", "gate", "d_x", "d_u"):
        wide = torch.full((T, start + H + pad), float("nan"), dtype=dtype, device=DEV)
        wide[:, start:start + H] = dev(s[n])
        on[n] = wide[:, start:start + H]
    kw = {k: dev(s[k]) for k in ("scale", "w_after", "w_before")}
    a = mgg.block_residual_norm(on["x"], on["y"], gate=on["gate"], eps=EPS, **kw)
    b = mgg.block_residual_norm(dev(s["x"]), dev(s["y"]), gate=dev(s["gate"]), eps=EPS, **kw)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a = mgg.block_residual_norm_backward(on["x"], on["y"], on["d_x"], on["d_u"], gate=on["gate"],
                                         eps=EPS, **kw)
    b = mgg.block_residual_norm_backward(dev(s["x"]), dev(s["y"]), dev(s["d_x"]), dev(s["d_u"]),
                                         gate=dev(s["gate"]), eps=EPS, **kw)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    # a token gate taken from a column of a wider tensor
    g = torch.randn((T, 7), generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    a = mgg.block_residual_norm(on["x"], on["y"], gate=g[:, 3], eps=EPS, **kw)
    b = mgg.block_residual_norm(on["x"], on["y"], gate=g[:, 3].contiguous(), eps=EPS, **kw)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_writes_stay_in_bounds():
    """Outputs inside larger buffers: the bytes around them keep their contents."""
    T, H = 5, 1001
    for dtype in (torch.bfloat16, torch.float32):
        say(f"block norm bounds {dtype}")
        s = make(T, H, dtype, "token")
        kw = {k: dev(v) if torch.is_tensor(v) else v for k, v in params(s).items()}
        bufs = [torch.full((T * H + 64,), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
        outs = [b[32:32 + T * H].view(T, H) for b in bufs]
        mgg.block_residual_norm(dev(s["x"]), dev(s["y"]), x_out=outs[0], u=outs[1], **kw)
        torch.cuda.synchronize()
        want = mgg.block_residual_norm(dev(s["x"]), dev(s["y"]), **kw)
        for b, o, w in zip(bufs, outs, want):
            assert torch.equal(o, w)
            assert (b[:32] == 7).all() and (b[32 + T * H:] == 7).all()


def test_gradient_against_differences():
    s = make(6, 40, torch.float32, "element")
    kw = params(s)
    x, y = f64(s["x"]), f64(s["y"])
    kn = {k: f64(v) if torch.is_tensor(v) else v for k, v in kw.items()}
    out = ref.block_residual_norm(x, y, **kn)["x_out"]
    got = mgg.block_residual_norm_backward(
        torch.from_numpy(out).float().to(DEV), dev(s["y"]), dev(s["d_x"]), dev(s["d_u"]),
        **{k: dev(v) if torch.is_tensor(v) else v for k, v in kw.items()})

    def loss(x_, y_, k_):
        r = ref.block_residual_norm(x_, y_, **k_)
        return (r["x_out"] * f64(s["d_x"])).sum() + (r["u"] * f64(s["d_u"])).sum()

    h = 1e-6
    for name, g in zip(("x", "y", "gate", "scale", "w_after", "w_before"), got):
        say(f"block norm differences {name}")
        at = {"x": x, "y": y}.get(name, kn.get(name))
        v = np.random.default_rng(3).normal(size=at.shape)

        def moved(sign):
            k2, x2, y2 = dict(kn), x, y
            if name == "x":
                x2 = x + sign * h * v
            elif name == "y":
                y2 = y + sign * h * v
            else:
                k2[name] = at + sign * h * v
            return loss(x2, y2, k2)

        num = (moved(1) - moved(-1)) / (2 * h)
        d = f64(g) * v
        # the rounding of x_out to float32 and C roundings of the terms
        assert abs(d.sum() - num) <= 1e-7 + 512 * U * np.abs(d).sum(), name


def test_results_repeat_and_workspaces_may_hold_anything():
    T, H = 2100, 520
    s = make(T, H, torch.bfloat16, "token")
    kw = {k: dev(v) if torch.is_tensor(v) else v for k, v in params(s).items()}
    size = mgg.load_library().block_residual_norm_backward_workspace(T, H)
    args = [dev(s[n]) for n in ("x", "y", "d_x", "d_u")]
    say("block norm repeat")
    first = mgg.block_residual_norm_backward(*args, **kw)
    for fill in (0, 255):
        ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        again = mgg.block_residual_norm_backward(*args, workspace=ws, **kw)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_graph_replays_follow_inputs():
    T, H = 260, 2304
    s = make(T, H, torch.bfloat16, "token")
    kw = {k: dev(v) if torch.is_tensor(v) else v for k, v in params(s).items()}
    x, y, dx, du = (dev(s[n]) for n in ("x", "y", "d_x", "d_u"))

    def step():
        out, u = mgg.block_residual_norm(x, y, **kw)
        return (out, u) + mgg.block_residual_norm_backward(out, y, dx, du, **kw)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        say(f"block norm replay {i}")
        n = make(T, H, torch.bfloat16, "token", seed=100 + i)
        x.copy_(n["x"]), y.copy_(n["y"]), du.copy_(n["d_u"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_offsets_beyond_32_bits():
    """Rows that start past 2^32 elements, in every tensor of both directions."""
    H = 4096
    T = (1 << 32) // H + 100
    say(f"block norm {T} rows")
    s = make(100, H, torch.bfloat16, None, scale=False, after=True, before=True)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    y = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    x[-100:], y[-100:] = dev(s["x"]), dev(s["y"])
    kw = {k: dev(v) if torch.is_tensor(v) else v for k, v in params(s).items()}
    small = mgg.block_residual_norm(dev(s["x"]), dev(s["y"]), **kw)
    big = mgg.block_residual_norm(x, y, **kw)
    assert all(torch.equal(a, b[-100:]) for a, b in zip(small, big))
    assert not big[0][:-100].any()
    d = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    d[-100:] = dev(s["d_x"])
    g = mgg.block_residual_norm_backward(x, y, d, d, **kw)
    gs = mgg.block_residual_norm_backward(dev(s["x"]), dev(s["y"]), dev(s["d_x"]), dev(s["d_x"]), **kw)
    assert torch.equal(g[0][-100:], gs[0]) and torch.equal(g[1][-100:], gs[1])
    assert not g[0][:-100].any() and not g[1][:-100].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [64, 250, 256, 1000, 2048, 4100, 7168, 8192])
def test_many_rows(H, dtype):
    """Enough rows for workgroups that walk several and keep the parameters in LDS."""
    say(f"block norm many rows {H} {dtype}")
    T = 40000 if H <= 256 else 9001 if H <= 2048 else 2100
    for gate in ("token", "element"):
        s = make(T, H, dtype, gate)
        out = check(s, alpha=1.25)
        # each row is its own: a few of them alone give the same bits
        kw = {k: dev(v) if torch.is_tensor(v) else v for k, v in params(s, alpha=1.25).items()}
        rows = slice(T - 3, T)
        kw["gate"] = kw["gate"][rows]
        few = mgg.block_residual_norm(dev(s["x"])[rows], dev(s["y"])[rows], **kw)
        for a, b in zip(few, out):
            assert (a.double() - b[rows].double()).abs().max() <= \
                2.0 ** -7 * b[rows].double().abs().max()


def test_two_streams():
    say("block norm streams")
    ss = [make(3000, 1024, torch.bfloat16, "token"), make(700, 7168, torch.bfloat16, "element")]
    kws = [{k: dev(v) if torch.is_tensor(v) else v for k, v in params(s).items()} for s in ss]
    ins = [[dev(s[n]) for n in ("x", "y", "d_x", "d_u")] for s in ss]
    want = [mgg.block_residual_norm_backward(*i, **k) for i, k in zip(ins, kws)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(mgg.block_residual_norm_backward(*ins[i], **kws[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i in range(2) for o in got[i] for a, b in zip(o, want[i]))
