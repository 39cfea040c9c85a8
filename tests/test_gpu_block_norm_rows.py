"""The norms around a block over many rows, where workgroups walk several rows each and keep the
parameters in LDS: every form of the kernels, and sums over rows that miss no row.

Tolerances are those of test_gpu_block_norm.py, C = 128 roundings for a forward value and 256 for
a gradient, but for the parameters' gradients: at least 256 row groups deal the rows among them, so
a thread adds at most T / 256 rows (two, where that is more) in float32, a workgroup its eight groups
at most, and the rest is added in float64. So C = 256 + T / 256 + 8 there, and a reference that
lacks two rows, the least that a workgroup takes, has to fail it."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg
from oracle import layer_ops as ref
from parity_util import say
from test_gpu_block_norm import EPS, U, close, dev, f64, make, params

pytestmark = pytest.mark.gpu
SUMS = ("scale", "w_after", "w_before")


def sum_roundings(T):
    return 256 + max(2, -(-T // 256)) + 8


def within(got, want, mag, c):
    return np.abs(f64(got) - want) <= c * U * mag + U * np.abs(want) + 1e-37


def check_sums(got, grads, missing, T):
    """Parameter gradients against the reference, and against one without some rows."""
    c = sum_roundings(T)
    for name, g in got.items():
        want, mag = grads[name]
        assert g.dtype == torch.float32 and within(g, want, mag, c).all(), name
        lacking, mag = missing[name]
        assert not within(g, lacking, mag, c).all(), name


def run(s, alpha=1.0, beta=1.0):
    kw = params(s, alpha=alpha, beta=beta)
    on = {k: dev(v) if torch.is_tensor(v) else v for k, v in kw.items()}
    ref_kw = {k: f64(v) if torch.is_tensor(v) else v for k, v in kw.items()}
    T = s["x"].shape[0]
    out, u = mgg.block_residual_norm(dev(s["x"]), dev(s["y"]), **on)
    r = ref.block_residual_norm(f64(s["x"]), f64(s["y"]), **ref_kw)
    close(out, r["x_out"], r["x_mag"], 128, "x_out")
    if u is not None:
        close(u, r["u"], r["u_mag"], 128, "u")
    # a few rows alone, by workgroups that take one row each
    few = slice(T - 3, T)
    on_few = dict(on, gate=None if on["gate"] is None else on["gate"][few])
    for a, b in zip(mgg.block_residual_norm(dev(s["x"])[few], dev(s["y"])[few], **on_few),
                    ("x_out", "u")):
        if a is not None:
            close(a, r[b][few], r[b[0] + "_mag"][few], 128, b)
    got = dict(zip(("x", "y", "gate") + SUMS,
                   mgg.block_residual_norm_backward(out, dev(s["y"]), dev(s["d_x"]),
                                                    dev(s["d_u"]), **on)))
    args = [f64(out), f64(s["y"]), f64(s["d_x"]), f64(s["d_u"])]
    want = ref.block_residual_norm_grad(*args, **ref_kw)
    for name in ("x", "y", "gate"):
        if got[name] is not None:
            close(got[name], *want[name], 256, name)
    gone = np.zeros(T, bool)
    gone[[T // 5, T // 2]] = True
    keep = [None if a is None else a[~gone] for a in args]
    kw_keep = dict(ref_kw)
    if kw_keep["gate"] is not None:
        kw_keep["gate"] = kw_keep["gate"][~gone]
    missing = ref.block_residual_norm_grad(*keep, **kw_keep)
    check_sums({n: got[n] for n in SUMS if got[n] is not None}, want, missing, T)


# a half wave, a wave with one and with two pieces a thread, and whole workgroups to a row
SHAPES = [(33000, 64), (33000, 250), (17000, 500), (17000, 1000), (5000, 2048), (2100, 7168)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_rows(T, H, dtype):
    say(f"block norm rows {T} {H} {dtype}")
    run(make(T, H, dtype, "token", param=torch.float32), alpha=1.25)


@pytest.mark.parametrize("T,H,dtype", [(33000, 200, torch.float32), (17000, 777, torch.bfloat16),
                                       (17000, 512, torch.float32), (2100, 5001, torch.bfloat16)])
def test_many_rows_gated_per_element(T, H, dtype):
    say(f"block norm rows, element gates {T} {H} {dtype}")
    run(make(T, H, dtype, "element", param=torch.bfloat16), alpha=1.25)


@pytest.mark.parametrize("scale,after,before,gate", [
    (False, True, True, "token"), (True, False, True, "element"), (True, True, False, None),
    (False, False, True, "element"), (False, True, False, "token"), (True, False, False, None),
    (False, False, True, None)])
def test_many_rows_with_parts(scale, after, before, gate):
    for T, H, dtype in ((4200, 2048, torch.bfloat16), (2100, 3001, torch.float32)):
        say(f"block norm rows with {scale} {after} {before} {gate} {dtype}")
        run(make(T, H, dtype, gate, scale, after, before, dtype), alpha=0.75, beta=-1.5)


@pytest.mark.parametrize("T,H", [(33000, 256), (17000, 1000), (4200, 2047), (2100, 7168)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_alone(T, H, dtype):
    say(f"block norm alone {T} {H} {dtype}")
    s = make(T, H, dtype)
    x, w = dev(s["x"]), dev(s["w_before"])
    u = mgg.block_norm(x, w, eps=EPS)
    wn = f64(s["w_before"])
    r = ref.block_residual_norm(f64(s["x"]), w_before=wn, eps=EPS)
    close(u, r["u"], r["u_mag"], 128, "u")
    gone = np.zeros(T, bool)
    gone[[T // 5, T // 2]] = True
    for dx in (s["d_x"], None):
        d, dw = mgg.block_norm_backward(x, w, dev(s["d_u"]), dev(dx), eps=EPS)
        args = [f64(s["x"]), None, f64(dx), f64(s["d_u"])]
        want = ref.block_residual_norm_grad(*args, w_before=wn, eps=EPS)
        close(d, *want["x"], 256, "x")
        missing = ref.block_residual_norm_grad(*(None if a is None else a[~gone] for a in args),
                                               w_before=wn, eps=EPS)
        check_sums({"w_before": dw}, want, missing, T)
