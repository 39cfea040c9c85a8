"""Newton-Schulz updates on the GPU against the float64 definition.

The products are to be of float32 grade. What that allows is measured by the same steps in
plain float32 arithmetic on the CPU: the result may be four times as far from the float64 one
as those are, plus the most that one rounding to 22 bits of each factor of a step's polynomial
commits, 2^-22 (|a| + |b| + |c|), added over the steps. bf16 outputs add half a step, 2^-8, of
each value. Distances are Frobenius norms relative to the result's."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg
from oracle import layer_ops as ref
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
USUAL = (3.4445, -4.7750, 2.0315)


def momenta(G, M, N, dtype, seed=0, rank=0):
    g = torch.Generator().manual_seed(seed + 31 * M + N)
    x = torch.randn((G, M, N), generator=g)
    if rank:
        x = x + 2.0 * torch.randn((G, M, rank), generator=g) @ torch.randn((G, rank, N), generator=g)
    return (1e-3 * x).to(dtype)


def check(X, coeffs=USUAL, steps=5, out_dtype=None, scale=1.0, eps=1e-7):
    rows = [coeffs] * steps if not hasattr(coeffs[0], "__len__") else coeffs
    out = mgg.grouped_newton_schulz(X.to(DEV), steps=steps, coeffs=coeffs, scale=scale, eps=eps,
                                    out_dtype=out_dtype)
    torch.cuda.synchronize()
    x = X.double().numpy()
    f32 = [np.float32(v) for r in rows for v in r]
    rows = [tuple(float(v) for v in f32[3 * i:3 * i + 3]) for i in range(len(rows))]
    want = ref.newton_schulz(x, rows, eps, scale)
    plain = ref.newton_schulz(x, rows, eps, scale, np.float32)
    got = out.double().cpu().numpy()
    for g in range(X.shape[0]):
        size = np.linalg.norm(want[g])
        if size == 0:
            assert not got[g].any()
            continue
        allowed = 4 * np.linalg.norm(plain[g] - want[g]) / size
        allowed += sum(2.0 ** -22 * sum(abs(v) for v in r) for r in rows)
        if out.dtype == torch.bfloat16:
            allowed += 2.0 ** -8
        off = np.linalg.norm(got[g] - want[g]) / size
        assert off <= allowed, (g, off, allowed)
    return out


SIZES = [(1, 1, 1), (2, 1, 9), (2, 9, 1), (3, 2, 3), (2, 31, 17), (1, 64, 64), (2, 127, 128),
         (2, 129, 64), (1, 128, 300), (1, 300, 129), (3, 257, 200), (1, 512, 512), (2, 100, 1000),
         (1, 1000, 130), (1, 640, 385)]


@pytest.mark.parametrize("G,M,N", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sizes(G, M, N, dtype):
    say(f"ns {G} {M} {N} {dtype}")
    check(momenta(G, M, N, dtype))
    check(momenta(G, M, N, dtype, rank=2))


# Few tiles and a long K: the sums of X X^T are cut into parts, the last of them shorter or not.
@pytest.mark.parametrize("G,M,N", [(1, 64, 4099), (1, 5000, 60), (3, 230, 1878), (7, 200, 1500),
                                   (1, 449, 3000), (2, 2300, 380)])
def test_long_sums(G, M, N):
    say(f"ns long sums {G} {M} {N}")
    X = momenta(G, M, N, torch.float32)
    out = check(X)
    assert torch.equal(out, mgg.grouped_newton_schulz(X.to(DEV)))
    check(momenta(G, M, N, torch.bfloat16, rank=3))


@pytest.mark.parametrize("steps", [1, 2, 7])
def test_steps_and_coefficients(steps):
    say(f"ns steps {steps}")
    X = momenta(2, 140, 90, torch.float32)
    check(X, steps=steps)
    check(X, steps=steps, coeffs=[(2.0 - 0.01 * i, -1.5, 0.5) for i in range(steps)], scale=-3.0)
    check(X, steps=steps, coeffs=(1.5, -0.5, 0.0), eps=1e-2)


def test_mixed_types():
    say("ns types")
    check(momenta(2, 70, 150, torch.float32), out_dtype=torch.bfloat16)
    check(momenta(2, 150, 70, torch.bfloat16), out_dtype=torch.float32)


def test_orthogonal_result():
    """A convergent cubic iteration ends at the polar factor: rows orthonormal."""
    say("ns orthogonal")
    X = torch.eye(96)[None] + 0.05 * torch.randn((1, 96, 96), generator=torch.Generator().manual_seed(0))
    out = mgg.grouped_newton_schulz(X.to(DEV), steps=20, coeffs=(1.5, -0.5, 0.0)).double().cpu()[0]
    # twenty steps converge quadratically; each leaves 22-bit roundings of 96 products a row
    assert (out @ out.t() - torch.eye(96).double()).abs().max() < 96 * 2.0 ** -22


def test_spread_of_singular_values():
    """Singular values down to 1e-4 of the largest, which five steps raise several hundred
    times: errors of 16-bit size would show."""
    say("ns spread")
    g = torch.Generator().manual_seed(2)
    u, _ = torch.linalg.qr(torch.randn((200, 200), generator=g, dtype=torch.float64))
    v, _ = torch.linalg.qr(torch.randn((260, 200), generator=g, dtype=torch.float64))
    s = torch.logspace(0, -4, 200, dtype=torch.float64)
    check(((u * s) @ v.t()).float()[None])


def test_zero_and_nan_matrices_leave_others_alone():
    say("ns zero and nan")
    X = momenta(4, 60, 80, torch.float32)
    alone = mgg.grouped_newton_schulz(X.to(DEV))
    X[1] = 0
    X[2, 3, 4] = float("nan")
    out = mgg.grouped_newton_schulz(X.to(DEV))
    assert torch.equal(out[0], alone[0]) and torch.equal(out[3], alone[3])
    assert not out[1].any() and torch.isnan(out[2]).all()
    X[2, 3, 4] = float("inf")
    out = mgg.grouped_newton_schulz(X.to(DEV))
    assert torch.equal(out[3], alone[3]) and torch.isnan(out[2]).all()


def test_magnitudes():
    """The result does not depend on the matrix's size, from tiny to where squares overflow
    float32."""
    say("ns magnitudes")
    X = momenta(1, 50, 70, torch.float32)
    for mul in (1e-20, 1e5, 1e25, 1e33):
        check(X * mul, eps=1e-30)


def test_transpose_and_repeat():
    say("ns transpose, repeat")
    X = momenta(2, 150, 210, torch.float32).to(DEV)
    a = mgg.grouped_newton_schulz(X)
    b = mgg.grouped_newton_schulz(X.transpose(1, 2).contiguous()).transpose(1, 2)
    # the same products in the same order but for the sum of squares
    assert (a - b).norm() <= 2.0 ** -20 * a.norm()
    size = mgg.load_library().grouped_newton_schulz_workspace(2, 150, 210)
    for fill in (0, 255, 60):
        ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(a, mgg.grouped_newton_schulz(X, workspace=ws))
    assert torch.equal(a[1:], mgg.grouped_newton_schulz(X[1:].contiguous()))


def test_writes_stay_in_bounds():
    for M, N in ((33, 130), (130, 33)):
        for dt in (torch.float32, torch.bfloat16):
            say(f"ns bounds {M} {N} {dt}")
            X = momenta(2, M, N, torch.float32).to(DEV)
            buf = torch.full((2 * M * N + 66,), 7.0, dtype=dt, device=DEV)
            out = buf[33:33 + 2 * M * N].view(2, M, N)
            mgg.grouped_newton_schulz(X, out=out)
            torch.cuda.synchronize()
            assert torch.equal(out, mgg.grouped_newton_schulz(X, out_dtype=dt))
            assert (buf[:33] == 7).all() and (buf[33 + 2 * M * N:] == 7).all()


def test_graph_replays_follow_inputs():
    X = momenta(3, 130, 260, torch.float32).to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mgg.grouped_newton_schulz(X)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mgg.grouped_newton_schulz(X)
    for i in range(4):
        say(f"ns replay {i}")
        X.copy_(momenta(3, 130, 260, torch.float32, seed=i + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mgg.grouped_newton_schulz(X))


def test_update_of_a_weight_gradient():
    """The K-grouped product's gradients, experts without tokens among them, straight into
    the update."""
    from moe_grouped_gemm_nt_amd import synth
    say("ns after kgrouped")
    p = synth.make_kgrouped("bf16", [64, 0, 128], 128, 256, seed=3, device=DEV)
    D = torch.empty((3, 128, 256), device=DEV)
    mgg.grouped_gemm_kgrouped(p.A, p.B, D, p.ks, 128, 256, accumulate=False)
    out = check(D.cpu())
    assert not out[1].any()


def test_large_wide():
    """A larger matrix against float64 on the GPU, relative to float32 products there."""
    say("ns large")
    X = momenta(2, 1024, 1536, torch.float32).to(DEV)

    def steps(dtype):
        x = X.double() / (X.double().pow(2).sum((1, 2), keepdim=True).sqrt() + 1e-7)
        x = x.to(dtype)
        a, b, c = (float(np.float32(v)) for v in USUAL)
        for _ in range(5):
            A = torch.stack([m @ m.t().contiguous() for m in x])
            B = torch.stack([b * m + c * (m @ m) for m in A])
            x = torch.stack([a * m + B[i] @ m for i, m in enumerate(x)])
        return x.double()

    want, plain = steps(torch.float64), steps(torch.float32)
    out = mgg.grouped_newton_schulz(X).double()
    allowed = 4 * (plain - want).norm() / want.norm() + 5 * 2.0 ** -22 * 10.251
    assert (out - want).norm() / want.norm() <= allowed


# One shape for every way that a product is dealt: 128-tiles of the symmetric products with the
# last of them quartered and one full round of 256-tiles; 256-tiles with their last round
# quartered; 256-tiles of the symmetric products; sides that are no multiple of any tile.
@pytest.mark.parametrize("G,M,N,dtype", [(4, 2048, 2048, torch.float32),
                                         (6, 1536, 4096, torch.bfloat16),
                                         (7, 2048, 2050, torch.float32),
                                         (5, 3001, 1025, torch.float32)])
def test_large_shapes(G, M, N, dtype):
    say(f"ns large {G} {M} {N} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(M)
    X = (1e-3 * torch.randn((G, M, N), device=DEV, generator=g)).to(dtype)
    a, b, c = (float(np.float32(v)) for v in USUAL)

    def steps(m, to):
        x = (m.double() / (m.double().norm() + 1e-7)).to(to)
        x = x.t().contiguous() if M > N else x
        for _ in range(5):
            A = x @ x.t().contiguous()
            x = a * x + (b * A + c * (A @ A)) @ x
        return (x.t() if M > N else x).double()

    out = mgg.grouped_newton_schulz(X)
    for i in range(G):
        want, plain = steps(X[i], torch.float64), steps(X[i], torch.float32)
        allowed = 4 * (plain - want).norm() / want.norm() + 5 * 2.0 ** -22 * 10.251
        if dtype == torch.bfloat16:
            allowed += 2.0 ** -8
        assert (out[i].double() - want).norm() / want.norm() <= allowed, i
    # captured and replayed, the same bits
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = mgg.grouped_newton_schulz(X)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, out)
        assert torch.equal(mgg.grouped_newton_schulz(X), out)


def test_two_streams():
    """Calls on two streams at once, each with its own workspace, give the same bits."""
    say("ns streams")
    X, Y = momenta(3, 300, 400, torch.float32).to(DEV), momenta(2, 500, 200, torch.bfloat16).to(DEV)
    want = mgg.grouped_newton_schulz(X), mgg.grouped_newton_schulz(Y)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (s, t) in enumerate(zip(streams, (X, Y))):
            with torch.cuda.stream(s):
                got[i].append(mgg.grouped_newton_schulz(t))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for outs, w in zip(got, want) for o in outs)
