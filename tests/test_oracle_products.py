"""Pins of the float64 definitions in oracle/products.py: torch's own float64 operations and
autograd, finite differences, closed forms (CPU)."""

import numpy as np
import pytest
import torch

import oracle
from moe_grouped_gemm_nt_amd import synth
from oracle import products as ref

FUNCS = ["none", "relu", "gelu", "silu", "swiglu"]


def torch_func(func, z):
    if func == "swiglu":
        a, b = z.chunk(2, 1)
        return torch.nn.functional.silu(a) * b
    return {"none": lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
            "silu": torch.nn.functional.silu}[func](z)


@pytest.mark.parametrize("func", FUNCS)
def test_linear_and_gradients_against_torch(func):
    g = np.random.default_rng(1)
    M, N, K = 7, 10, 5
    x, w, b = g.normal(size=(M, K)), g.normal(size=(N, K)), g.normal(size=N)
    C = N // 2 if func == "swiglu" else N
    r, d = g.normal(size=(M, C)), g.normal(size=(M, C))
    out, z = ref.linear(x, w, b, func, r)
    t = [torch.from_numpy(v).requires_grad_() for v in (x, w, b, r)]
    y = torch_func(func, t[0] @ t[1].T + t[2]) + t[3]
    np.testing.assert_allclose(out, y.detach().numpy(), rtol=1e-13, atol=1e-14)
    y.backward(torch.from_numpy(d))
    dx, dw, db, _ = ref.linear_grad(x, w, d, z, func)
    for got, want in zip((dx, dw, db, d), t):
        np.testing.assert_allclose(got, want.grad.numpy(), rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("func", FUNCS[1:])
def test_func_grad_against_differences(func):
    z = np.linspace(-6.0, 6.0, 24).reshape(3, 8) + 0.013
    d = np.random.default_rng(2).normal(size=(3, 4 if func == "swiglu" else 8))
    got, h = ref.func_grad(func, z, d), 1e-6
    for i in np.ndindex(z.shape):
        up, down = z.copy(), z.copy()
        up[i] += h
        down[i] -= h
        want = ((ref.func_of(func, up) - ref.func_of(func, down)) / (2 * h) * d).sum()
        assert got[i] == pytest.approx(want, rel=1e-7, abs=1e-9)


def test_function_values():
    z = np.array([[-np.inf, -40.0, 0.0, 40.0, np.inf]])
    assert ref.func_of("relu", z)[0].tolist() == [0.0, 0.0, 0.0, 40.0, np.inf]
    np.testing.assert_allclose(ref.func_of("gelu", z[:, 1:4])[0], [-1.4666e-348, 0.0, 40.0], atol=0)
    assert ref.func_of("silu", z[:, 3:])[0].tolist() == [40.0, np.inf]
    assert ref.normal_cdf(np.array([0.0]))[0] == 0.5


def test_few_tokens_against_torch():
    g = np.random.default_rng(3)
    T, k, G, H, I = 5, 3, 4, 6, 3
    x, w13, w2 = g.normal(size=(T, H)), g.normal(size=(G, 2 * I, H)), g.normal(size=(G, H, I))
    ids = np.array([[0, 1, 2], [3, 3, -1], [-1, -1, -1], [4, 2, -7], [1, 0, 3]])
    wt, res = g.normal(size=(T, k)), g.normal(size=(T, H))
    wt[ids < 0] = np.nan  # nothing that stands at an empty place has an effect
    got = ref.moe_few_tokens(x, ids, wt, w13, w2, res)
    for t in range(T):
        want = torch.from_numpy(res[t]).clone()
        for j in range(k):
            e = ids[t, j]
            if 0 <= e < G:
                z = torch.from_numpy(w13[e]) @ torch.from_numpy(x[t])
                h = torch.nn.functional.silu(z[:I]) * z[I:]
                want += wt[t, j] * (torch.from_numpy(w2[e]) @ h)
        np.testing.assert_allclose(got[t], want.numpy(), rtol=1e-12, atol=1e-13)
    assert (got[2] == res[2]).all()
    both, err = ref.moe_few_tokens(x, ids, wt, w13, w2, res, roundings=2.0 ** -24)
    assert (both == got).all() and (err[[0, 1, 3, 4]] > 0).all() and (err < 1e-3).all()


@pytest.mark.parametrize("gran,fmt", [("block128", "f32"), ("block128", "ue8m0"),
                                      ("channel", "f32"), ("channel", "ue8m0"),
                                      ("block32", "ue8m0")])
def test_expert_weights_are_the_grouped_products(gran, fmt):
    """The same weights as oracle.grouped_gemm_masked reads: its product with unit vectors."""
    kind = "fp8_fp4" if gran == "block32" else "fp8"
    p = synth.make_masked(kind, 2, 8, 136, 256, [8, 8], seed=4, sf_fmt=fmt, sfb_gran=gran)
    A = np.zeros((2, 8, 256), np.uint8)
    A[:, np.arange(8), np.arange(8) * 31] = 0x38  # 1.0 in E4M3
    one = np.full((2, 2, 8), 127, np.uint8) if fmt == "ue8m0" else np.ones((2, 2, 8), np.float32)
    got, _ = oracle.grouped_gemm_masked(kind, A, p.B.numpy(), [8, 8], one, p.SFB.numpy(), gran, fmt)
    w = ref.expert_weights(p.B.numpy(), p.SFB.numpy(), gran, fmt)
    np.testing.assert_array_equal(got, w[:, :, np.arange(8) * 31].transpose(0, 2, 1))
