"""Dense products with their epilogue, and their gradients, on the GPU against float64.

Tolerances, u = 2^-24: a float32 sum of K products is off by at most (K + 8) u of the sum of the
products' absolute values (one rounding for each addition); a function passes that on with its
largest slope (1.13 for gelu, 1.1 for silu) and adds up to 16 + 2 |z| roundings of its own value;
bias and residual add one each. A bf16 output adds half a step, 2^-8 of the value. Backward: dz has
the function's roundings, and half a step of its type where it is rounded (f32: none); products as
above."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg
from oracle import products as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
FUNCS = ["none", "relu", "gelu", "silu", "swiglu"]


def make(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(shape, generator=g)).to(dtype).to(DEV)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def half_step(dtype):
    return 2.0 ** -8 if dtype == BF else U


def close(got, want, err):
    off = np.abs(f64(got) - want)
    assert np.isfinite(off).all()
    assert (off <= err + 1e-37).all(), (off / (err + 1e-37)).max()


def check_forward(x, w, bias=None, func="none", residual=None, out_dtype=None, **kw):
    out, z = mgg.linear_act(x, w, bias, func, residual, keep_z=True, out_dtype=out_dtype, **kw)
    assert torch.equal(mgg.linear_act(x, w, bias, func, residual, out_dtype=out_dtype), out)
    X, W, B, R = f64(x), f64(w), f64(bias), f64(residual)
    want, zw = ref.linear(X, W, B, func, R)
    K = X.shape[1]
    ez = (K + 8) * U * (np.abs(X) @ np.abs(W).T) + U * np.abs(zw)
    if B is not None:
        ez = ez + U * np.abs(B)
    close(z, zw, ez + half_step(x.dtype) * np.abs(zw))
    if func == "swiglu":
        (g, u), (eg, eu) = np.split(zw, 2, 1), np.split(ez, 2, 1)
        h = np.abs(ref.silu(g))
        e = 1.1 * eg * np.abs(u) + h * eu + (16 + 2 * np.abs(g)) * U * h * np.abs(u)
    else:
        e = 1.13 * ez + (16 + 2 * np.abs(zw)) * U * np.abs(ref.func_of(func, zw))
    if R is not None:
        e = e + U * np.abs(R)
    close(out, want, e + half_step(out.dtype) * np.abs(want))
    return out, z


def check_backward(x, w, d_out, z=None, func="none", dw_dtype=None, **kw):
    dx, dw, db = mgg.linear_act_backward(x, w, d_out, z, func, need_bias=True, dw_dtype=dw_dtype,
                                         **kw)
    X, W, D, Z = f64(x), f64(w), f64(d_out), f64(z)
    wx, ww, wb, dz = ref.linear_grad(X, W, D, Z, func)
    M, N = dz.shape
    # slopes are sums of two terms: roundings count against the sizes of both
    if func == "none":
        size = np.abs(dz)
    elif func == "swiglu":
        g, u = np.split(np.abs(Z), 2, 1)
        size = np.concatenate([np.abs(D) * u * (1 + g), np.abs(D) * g], 1)
    else:
        size = np.abs(D) * (1 + np.abs(Z))
    z2 = 0 if Z is None else np.abs(Z) ** 2
    ez = (16 + 2 * z2) * U * size * (func != "none")
    held = func != "none" or d_out.dtype != x.dtype
    er = ez + (half_step(x.dtype) * (np.abs(dz) + ez) if held else 0)
    close(db, wb, ez.sum(0) + (M + 8) * U * (np.abs(dz) + ez).sum(0))
    a = np.abs(dz) + er
    close(dx, wx, er @ np.abs(W) + (N + 8) * U * (a @ np.abs(W)) + half_step(dx.dtype) * np.abs(wx))
    close(dw, ww, er.T @ np.abs(X) + (M + 8) * U * (a.T @ np.abs(X)) +
          half_step(dw.dtype) * np.abs(ww))
    return dx, dw, db


SIZES = [(1, 2, 1), (1, 288, 512), (2, 30, 7), (16, 64, 96), (17, 34, 65), (33, 16, 1000),
         (64, 100, 300), (65, 128, 64), (66, 130, 127), (128, 128, 128), (130, 258, 200),
         (257, 62, 1001), (300, 1000, 72), (513, 520, 264)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward_sizes(dtype, M, N, K):
    print(dtype, M, N, K, flush=True)
    x, w = make((M, K), dtype, 1), make((N, K), dtype, 2, K ** -0.5)
    check_forward(x, w, make((N,), F32, 3), "gelu", make((M, N), dtype, 4))
    check_forward(x, w, None, "swiglu")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(130, 258, 2056), (300, 70, 5000), (90, 40, 3333), (70, 3000, 640)])
def test_long_sums(dtype, M, N, K):
    """Few tiles and a long axis, which is cut into parts: of x w^T, and, with the sides exchanged,
    of dz w and dz^T x."""
    print(dtype, M, N, K, flush=True)
    x, w = make((M, K), dtype, 90), make((N, K), dtype, 91, K ** -0.5)
    check_forward(x, w, make((N,), F32, 92), "silu", make((M, N), F32, 93), F32)
    check_forward(x, w, None, "swiglu")
    for m, n, k in ((M, K, N), (K, M, N)):
        x, w = make((m, k), dtype, 94), make((n, k), dtype, 95)
        check_backward(x, w, make((m, n), dtype, 96), make((m, n), dtype, 97), "relu")


@pytest.mark.parametrize("M,N,K", [(4100, 4104, 72), (4352, 4096, 64), (4200, 4360, 136)])
def test_large_tiles(M, N, K):
    """As many rows and columns as fill the GPU with the largest tiles, with and without some left
    over; outputs in pieces and not. Against float64 on the GPU."""
    print(M, N, K, flush=True)
    x, w, b = make((M, K), BF, 100), make((N, K), BF, 101, K ** -0.5), make((N,), BF, 102)
    X, W = x.double(), w.double()
    z = X @ W.t() + b.double()
    err = (K + 10) * U * (X.abs() @ W.abs().t() + b.double().abs())
    for func, cols in (("none", N), ("swiglu", N // 2), ("gelu", N)):
        for out, ld in ((BF, cols), (F32, cols), (BF, cols + 1)):
            r = make((M, ld), out, 103)[:, :cols]
            got, gz = mgg.linear_act(x, w, b, func, r, keep_z=True, out_dtype=out)
            if func == "swiglu":
                g, u = z.chunk(2, 1)
                eg, eu = err.chunk(2, 1)
                h = g * torch.sigmoid(g)
                want, e = h * u, 1.1 * eg * u.abs() + h.abs() * eu + (16 + 2 * g.abs()) * U * (h * u).abs()
            else:
                want = z if func == "none" else torch.nn.functional.gelu(z)
                e = 1.13 * err + (16 + 2 * z.abs()) * U * want.abs()
            want = want + r.double()
            e = e + U * r.double().abs() + half_step(out) * want.abs()
            assert ((got.double() - want).abs() <= e).all()
            assert ((gz.double() - z).abs() <= err + half_step(BF) * z.abs()).all()
    # the same sizes as the sides of the gradients: dz [k, m] gives d_w [m, n], dz [m, k] d_x [m, n]
    for rows, d, other, turned in ((K, make((K, M), BF, 104), make((K, N), BF, 105), True),
                                   (M, make((M, K), BF, 106), make((K, N), BF, 107), False)):
        if turned:
            got = mgg.linear_act_backward(other, make((M, N), BF, 108), d, need_x=False)[1]
            a, c = d.double().t(), other.double()
        else:
            got = mgg.linear_act_backward(make((M, N), BF, 109), other, d, need_w=False)[0]
            a, c = d.double(), other.double()
        want = a @ c
        e = (K + 8) * U * (a.abs() @ c.abs()) + half_step(BF) * want.abs()
        assert ((got.double() - want).abs() <= e).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("func", FUNCS)
@pytest.mark.parametrize("M", [20, 150])
def test_forward_functions(dtype, func, M):
    N, K = 84, 136
    x, w = make((M, K), dtype, 5, 2.0), make((N, K), dtype, 6, 2 * K ** -0.5)
    C = N // 2 if func == "swiglu" else N
    for out in (BF, F32):
        for bias in (None, BF, F32):
            b = None if bias is None else make((N,), bias, 7)
            check_forward(x, w, b, func, make((M, C), out, 8) if bias == F32 else None, out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_backward_sizes(dtype, M, N, K):
    print(dtype, M, N, K, flush=True)
    x, w = make((M, K), dtype, 9), make((N, K), dtype, 10)
    check_backward(x, w, make((M, N), dtype, 11))
    check_backward(x, w, make((M, N // 2), dtype, 12), make((M, N), dtype, 13), "swiglu")
    check_backward(x, w, make((M, N), dtype, 14), make((M, N), dtype, 15), "silu", dw_dtype=F32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("func", FUNCS)
def test_backward_functions(dtype, func):
    M, N, K = 90, 84, 72
    C = N // 2 if func == "swiglu" else N
    x, w = make((M, K), dtype, 16), make((N, K), dtype, 17)
    z = None if func == "none" else make((M, N), dtype, 18, 3.0)
    for d in (BF, F32):
        check_backward(x, w, make((M, C), d, 19), z, func)


@pytest.mark.parametrize("func", FUNCS)
def test_gradients_against_differences(func):
    """The slope of sum(out * d) along a random direction of x, w and bias, float32."""
    M, N, K = 70, 48, 56
    C = N // 2 if func == "swiglu" else N
    x, w, b = make((M, K), F32, 20), make((N, K), F32, 21, K ** -0.5), make((N,), F32, 22)
    d = make((M, C), F32, 23)
    _, z = mgg.linear_act(x, w, b, func, keep_z=True)
    grads = mgg.linear_act_backward(x, w, d, None if func == "none" else z, func, need_bias=True)
    for i, t in enumerate((x, w, b)):
        v = make(t.shape, F32, 24 + i)
        sides = []
        for h in (1e-2, -1e-2):
            p = [x, w, b]
            p[i] = t + h * v
            sides.append((mgg.linear_act(*p, func).double() * d.double()).sum().item())
        slope = (sides[0] - sides[1]) / 2e-2
        want = (grads[i].double() * v.double()).sum().item()
        size = (grads[i].double() * v.double()).norm().item()
        # The third derivative: h^2 against sums of thousands of terms. Relu has none, but a kink:
        # where z passes 0 within the step, |z| <= h |s| with s the slope of z, the difference
        # quotient is (z + h |s|) / 2h |s| of s where the gradient has 0 or 1 of it; the two are
        # furthest apart at z = 0, by |s| / 2.
        kink = 0.0
        if func == "relu":
            s = v @ w.T if i == 0 else x @ v.T if i == 1 else v.expand(M, N)
            kink = (torch.where(z.abs() <= 1e-2 * s.abs(), s * d, 0.0).abs().sum() / 2).item()
        assert abs(slope - want) <= 2e-2 * size + 1e-2 + kink, (slope, want, size, kink)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M", [9, 140])
@pytest.mark.parametrize("offset,extra", [(0, 8), (1, 0), (1, 3), (4, 9)])
def test_strides(dtype, M, offset, extra):
    """Operands anywhere in wider tensors, NaN between the rows: bits of contiguous ones."""
    N, K = 72, 104

    def wide(t):
        R, C = t.shape
        buf = torch.full((offset + R * (C + extra),), float("nan"), dtype=t.dtype, device=DEV)
        view = buf[offset:].view(R, C + extra)[:, :C]
        view.copy_(t)
        return view
    x, w = make((M, K), dtype, 30), make((N, K), dtype, 31)
    r, d = make((M, N), dtype, 32), make((M, N), dtype, 33)
    a = mgg.linear_act(x, w, None, "silu", r, keep_z=True)
    b = mgg.linear_act(wide(x), wide(w), None, "silu", wide(r), keep_z=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for func, z in (("silu", a[1]), ("none", None)):
        g = mgg.linear_act_backward(x, w, d, z, func, need_bias=True)
        h = mgg.linear_act_backward(wide(x), wide(w), wide(d), None if z is None else wide(z), func,
                                    need_bias=True)
        assert all(torch.equal(p, q) for p, q in zip(g, h))


def test_empty_batches():
    w = make((6, 8), F32, 40)
    x, d, z = w[:0], w.new_empty((0, 6)), w.new_empty((0, 6))
    out, z2 = mgg.linear_act(x, w, func="relu", keep_z=True)
    assert out.shape == z2.shape == (0, 6)
    dx, dw, db = mgg.linear_act_backward(x, w, d, z, "relu", need_bias=True)
    assert dx.shape == (0, 8) and not dw.any() and not db.any() and dw.shape == (6, 8)


@pytest.mark.parametrize("M", [12, 200])
def test_only_what_is_needed(M):
    x, w, d = make((M, 40), BF, 41), make((56, 40), BF, 42), make((M, 56), BF, 43)
    z = make((M, 56), BF, 44)
    whole = mgg.linear_act_backward(x, w, d, z, "gelu", need_bias=True)
    for i in range(3):
        need = [j == i for j in range(3)]
        part = mgg.linear_act_backward(x, w, d, z, "gelu", *need)
        assert torch.equal(part[i], whole[i])
        assert all(part[j] is None for j in range(3) if j != i)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(20, 72, 100), (150, 136, 203)])
def test_isolation(dtype, M, N, K):
    """A NaN or infinity in a row stays in what depends on it; guard rows around an output stay;
    a workspace's old contents have no effect."""
    x, w = make((M, K), dtype, 50), make((N, K), dtype, 51)
    room = torch.full((M + 2, N), 7.0, dtype=dtype, device=DEV)
    a = mgg.linear_act(x, w)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(mgg.linear_act(x, w, out=room[1:-1], workspace=ws), a)
    assert (room[0] == 7).all() and (room[-1] == 7).all()
    bx, bw = x.clone(), w.clone()
    bx[3, K - 1], bw[N - 2, 0] = float("nan"), float("inf")
    b = mgg.linear_act(bx, bw)
    rows, cols = [m for m in range(M) if m != 3], [n for n in range(N) if n != N - 2]
    assert torch.equal(b[rows][:, cols], a[rows][:, cols]) and b[3].isnan().all()
    assert not b[rows, N - 2].isfinite().any()
    d = make((M, N), dtype, 52)
    g = mgg.linear_act_backward(x, w, d, a, "relu", need_bias=True, workspace=ws)
    bd = d.clone()
    bd[5, 7] = float("nan")
    ba = a.clone()
    ba[5, 7] = 1.0
    h = mgg.linear_act_backward(x, w, bd, ba, "relu", need_bias=True)
    rows, cols = [m for m in range(M) if m != 5], [n for n in range(N) if n != 7]
    assert torch.equal(h[0][rows], g[0][rows]) and h[0][5].isnan().all()
    assert torch.equal(h[1][cols], g[1][cols]) and h[1][7].isnan().all()
    assert torch.equal(h[2][cols], g[2][cols]) and h[2][7].isnan()


def test_function_ends():
    """Arguments far out: no NaN from an exponential, infinities where they belong."""
    x = torch.tensor([[-1e30], [-1e4], [-30.0], [0.0], [30.0], [1e4], [1e30]], device=DEV)
    w = torch.ones((1, 1), device=DEV)
    for func in ("gelu", "silu"):
        out, z = mgg.linear_act(x, w, func=func, keep_z=True)
        assert torch.equal(z, x)
        assert out[:2, 0].tolist() == [0.0, 0.0] and out[3:, 0].tolist() == [0.0, 30.0, 1e4, out[6, 0]]
        d, _, _ = mgg.linear_act_backward(x, w, torch.ones_like(x), z, func)
        assert d[0, 0] == 0 and d[1, 0] == 0 and d[3, 0] == 0.5 and d[5, 0] == 1 and d[6, 0] == 1


def test_bitwise_repeats_and_graph_replays():
    """Equal bits from call to call; forward and backward in one graph, replayed with new values
    among eager calls."""
    M, N, K = 200, 264, 136
    x, w, b = make((M, K), BF, 60), make((N, K), BF, 61), make((N,), F32, 62)
    d = make((M, N), BF, 63)

    def step():
        out, z = mgg.linear_act(x, w, b, "gelu", d, keep_z=True)
        return (out, z, *mgg.linear_act_backward(x, w, d, z, "gelu", need_bias=True))
    first = step()
    for _ in range(10):
        assert all(torch.equal(p, q) for p, q in zip(step(), first))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = step()
    for seed in range(4):
        x.copy_(make((M, K), BF, 70 + seed))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(step(), captured))


def test_streams():
    x, w = make((300, 512), BF, 80), make((256, 512), BF, 81)
    few = x[:8]
    want = mgg.linear_act(x, w), mgg.linear_act(few, w)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(mgg.linear_act(x if i == 0 else few, w))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])
