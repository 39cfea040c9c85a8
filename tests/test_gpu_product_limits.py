"""Products whose operands or outputs pass 2^32 bytes, and the widest and longest sides: rows and
columns sampled from all over against float64 on the GPU.

Tolerances: (K + 8) roundings u = 2^-24 of the sum of the products' absolute values, and half a step
2^-8 of bf16 results; the MoE layer's as in oracle.products with its h held in bf16."""

import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF = torch.bfloat16


def rand(*shape, seed=0, dtype=BF):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, device=DEV, generator=g, dtype=dtype)


def close(got, a, b, K):
    """got against a b^T in float64."""
    a, b = a.double(), b.double()
    want = a @ b.T
    err = (K + 8) * U * (a.abs() @ b.abs().T) + 2.0 ** -8 * want.abs()
    assert ((got.double() - want).abs() <= err).all()


def spread(n, count=40):
    return torch.linspace(0, n - 1, count).long().to(DEV)


def test_output_beyond_4_gib():
    M, N, K = 70001, 32776, 16
    x, w = rand(M, K, seed=1), rand(N, K, seed=2)
    out, z = mgg.linear_act(x, w, func="relu", keep_z=True)
    m, n = spread(M), spread(N)
    close(z[m][:, n], x[m], w[n], K)
    assert torch.equal(out[m], z[m].clamp(min=0))
    del z
    # the same through the gradients: d_x = dz w with dz [N, K] and w [K, ...]
    got = mgg.linear_act_backward(rand(M, N - 8, seed=3), w[:K, :].new_zeros((K, N - 8)), x,
                                  need_w=False)[0]
    assert got.shape == (M, N - 8) and not got[m].any()


@pytest.mark.parametrize("M", [5, 200])
@pytest.mark.parametrize("func", ["none", "swiglu"])
def test_weights_beyond_4_gib(M, func):
    N, K = 270000, 8200
    x, w = rand(M, K, seed=4), rand(N, K, seed=5)
    out = mgg.linear_act(x, w, func=func, out_dtype=torch.float32)
    n = spread(out.shape[1])
    z = (x.double() @ w[n].double().T)
    err = (K + 8) * U * (x.double().abs() @ w[n].double().abs().T)
    if func == "swiglu":
        up = w[n + N // 2].double()
        u = x.double() @ up.T
        eu = (K + 8) * U * (x.double().abs() @ up.abs().T)
        h = z * torch.sigmoid(z)
        err = 1.1 * err * u.abs() + h.abs() * eu + (16 + 2 * z.abs()) * U * (h * u).abs()
        z = h * u
    assert ((out[:, n].double() - z).abs() <= err + 1e-30).all()


def test_long_sum_beyond_4_gib():
    """d_w over 600001 rows: both operands are walked along more than 4 GiB."""
    M, N, K = 600001, 72, 4104
    x, d = rand(M, K, seed=6), rand(M, N, seed=7)
    w = rand(N, K, seed=8)
    _, dw, db = mgg.linear_act_backward(x, w, d, need_x=False, need_bias=True,
                                        dw_dtype=torch.float32)
    k = spread(K, 24)
    a, b = d.double().T.contiguous(), x[:, k].double()
    # (K + 8) roundings of a sum of 600001 terms are no bound worth having: the tiles add 16 at a time
    # and join parts of the axis, so a term meets at most M / 16 roundings
    err = (M / 16 + 300) * U * (a.abs() @ b.abs())
    assert ((dw[:, k].double() - a @ b).abs() <= err).all()
    assert ((db.double() - d.double().sum(0)).abs() <= (M / 512 + 300) * U * d.double().abs().sum(0)).all()


def test_widest_rows():
    """K = 2^20, and rows that lie further apart than the tiles read (they are packed)."""
    K = 1 << 20
    x, w = rand(70, K, seed=9), rand(34, K, seed=10)
    close(mgg.linear_act(x, w), x, w, K)
    close(mgg.linear_act(x[:3], w), x[:3], w, K)
    wide = rand(200, (1 << 20) + 64, seed=11)[:, :96]
    w = rand(40, 96, seed=12)
    close(mgg.linear_act(wide, w), wide, w, 96)


@pytest.mark.parametrize("T", [3, 40])
def test_experts_beyond_4_gib(T):
    G, H, I, k = 300, 4096, 2048, 2
    g = torch.Generator(device=DEV).manual_seed(13)

    def codes(*shape):
        return (100 * torch.randn(shape, device=DEV, generator=g, dtype=BF)).clamp(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8)
    w13, w2 = codes(G, 2 * I, H), codes(G, H, I)
    s13 = torch.full((G, 2 * I // 128, H // 128), 118, dtype=torch.uint8, device=DEV)  # 2^-9
    s2 = torch.full((G, H // 128, I // 128), 117, dtype=torch.uint8, device=DEV)
    s13 -= torch.randint(0, 3, s13.shape, dtype=torch.uint8, device=DEV, generator=g)
    x = rand(T, H, seed=14) / 64
    ids = torch.tensor([[G - 1, 0], [G - 2, G - 1], [255, 128]], dtype=torch.int32,
                       device=DEV).repeat(T // 3 + 1, 1)[:T].contiguous()
    wt = torch.rand((T, k), device=DEV, generator=g)
    got = mgg.moe_few_tokens(x, ids, wt, w13, w2, s13, s2, out_dtype=torch.float32)
    want, err = torch.zeros((T, H), device=DEV, dtype=torch.float64), 0.0
    for e in ids.unique().tolist():
        def values(w, s):
            s = torch.exp2(s[e].double() - 127).repeat_interleave(128, 0).repeat_interleave(128, 1)
            return w[e].view(torch.float8_e4m3fn).double() * s
        a, b = values(w13, s13), values(w2, s2)
        z, zs = x.double() @ a.T, x.double().abs() @ a.abs().T
        gate, up = z[:, :I], z[:, I:]
        h = gate * torch.sigmoid(gate) * up
        dz = (H + 8) * U * zs
        dh = 1.1 * dz[:, :I] * up.abs() + gate.abs() * dz[:, I:] + (17 + 2 * gate.abs()) * U * h.abs()
        ww = (wt.double() * (ids == e)).sum(1, keepdim=True)
        want += ww * (h @ b.T)
        err = err + ww * (dh @ b.abs().T + (I + 24) * U * (h.abs() @ b.abs().T))
    assert ((got.double() - want).abs() <= err).all()
