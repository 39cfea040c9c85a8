"""Newton-Schulz updates of matrices that are small next to eps, and steps that shrink them: the
products stay of float32 grade whatever the size of X on its way.

Tolerances are those of test_gpu_newton_schulz.py: four times what plain float32 steps are off by,
and one rounding to 22 bits of each factor of a step's polynomial. Steps with b = c = 0 only
multiply; there a step rounds X and P to 22 bits and drops the product of their lower halves,
each at most 2^-22 of the result, and the division by the norm and the last store add two
roundings to 24 bits."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg
from parity_util import say
from test_gpu_newton_schulz import check, momenta

pytestmark = pytest.mark.gpu
DEV = "cuda"


def of_norm(X, norm):
    """Every matrix of X scaled to this Frobenius norm."""
    n = X.double().pow(2).sum((1, 2), keepdim=True).sqrt()
    return (X.double() / n * norm).float()


# 64-tiles, a cut sum, both orientations, 128-tiles and 256-tiles
@pytest.mark.parametrize("G,M,N", [(2, 50, 70), (1, 300, 129), (1, 512, 512), (1, 64, 4099),
                                   (5, 640, 896)])
@pytest.mark.parametrize("norm", [1e-7, 1e-9, 1e-11, 1e-12, 1e-14, 1e-20, 1e-30])
def test_norms_below_eps(G, M, N, norm):
    say(f"ns norm {norm} {G} {M} {N}")
    check(of_norm(momenta(G, M, N, torch.float32), norm))


@pytest.mark.parametrize("eps", [1.0, 1e6, 1e20])
def test_large_eps(eps):
    say(f"ns eps {eps}")
    check(momenta(2, 130, 200, torch.float32, rank=2), eps=eps)
    check(momenta(2, 200, 130, torch.bfloat16), eps=eps, out_dtype=torch.float32)


def test_every_matrix_has_its_own_size():
    say("ns sizes in one call")
    X = momenta(6, 90, 140, torch.float32)
    for i, norm in enumerate((1.0, 1e-9, 0.0, 1e-13, 1e-25, 1e-7)):
        X[i:i + 1] = of_norm(X[i:i + 1], norm)
    out = check(X)
    for i in range(6):
        assert torch.equal(out[i:i + 1], mgg.grouped_newton_schulz(X[i:i + 1].to(DEV))), i
    X[3, 5, 6] = float("nan")
    again = mgg.grouped_newton_schulz(X.to(DEV))
    assert torch.isnan(again[3]).all()
    for i in (0, 1, 2, 4, 5):
        assert torch.equal(again[i], out[i]), i


@pytest.mark.parametrize("factors", [[0.03] * 5, [0.5] * 30, [1e-3, 1e-4, 1e-3], [1e-6, 3.0, 3.0],
                                     [1e-8, 1e-8, 3.9, 3.9, 0.1]])
def test_steps_that_shrink(factors):
    say(f"ns shrinking {factors[:3]}")
    X = momenta(2, 100, 70, torch.float32)
    out = mgg.grouped_newton_schulz(X.to(DEV), steps=len(factors),
                                    coeffs=[(f, 0.0, 0.0) for f in factors])
    x = X.double().numpy()
    total = float(np.prod([np.float64(np.float32(f)) for f in factors]))
    got = out.double().cpu().numpy()
    for g in range(2):
        want = x[g] / (np.linalg.norm(x[g]) + 1e-7) * total
        allowed = 3 * len(factors) * 2.0 ** -22 + 2 * 2.0 ** -24
        assert np.linalg.norm(got[g] - want) <= allowed * np.linalg.norm(want)


@pytest.mark.parametrize("norm", [1e-3, 1e-8, 1e-10, 1e-13])
def test_steps_without_a_linear_term(norm):
    """X' = b X X^T X: here A and P are small with X. Two products of two factors, each rounded
    to 22 bits and without its lower halves' product: six times 2^-22 a step, of norms that the
    singular values' spread makes up to four times the result's."""
    say(f"ns cubic alone {norm}")
    X = of_norm(momenta(2, 80, 110, torch.float32), norm)
    for steps in (1, 2):
        got = mgg.grouped_newton_schulz(X.to(DEV), steps=steps, coeffs=(0.0, 1.2, 0.0))
        got = got.double().cpu().numpy()
        for g in range(2):
            x = X[g].double().numpy()
            x = x / (np.linalg.norm(x) + 1e-7)
            for _ in range(steps):
                x = float(np.float32(1.2)) * x @ x.T @ x
            least = 2.0 ** -126 * x.size ** 0.5  # of values below float32's range
            assert np.linalg.norm(got[g] - x) <= 4 * 6 * 3 ** (steps - 1) * 2.0 ** -22 \
                * np.linalg.norm(x) + least


def test_matrices_beyond_32_bits():
    """More than 2^32 elements in one call: the last matrices, some of them far below eps, against
    the same in a call of their own (other tiles, so other orders of the sums: each is within the
    bound of float32 products in five steps, five times 2^-22 (|a| + |b| + |c|) twice over)."""
    G, N, last = 1050, 2048, 3
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB")
    say(f"ns {G} {N} {N}")
    X = torch.zeros((G, N, N), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    X[-last:] = (1e-3 * torch.randn((last, N, N), device=DEV, generator=g)).to(torch.bfloat16)
    X[-2] *= 2.0 ** -40
    X[0] = X[-1]
    out = mgg.grouped_newton_schulz(X)
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[-1])
    for part in out[1:-last].split(64):
        assert not part.any()
    got, own = out[-last:].double(), mgg.grouped_newton_schulz(X[-last:].contiguous()).double()
    for i in range(last):
        allowed = 2 * 5 * 2.0 ** -22 * 10.251 + 2.0 ** -8  # and half a bf16 step of each
        assert (got[i] - own[i]).norm() <= allowed * own[i].norm() and own[i].norm() > 0
    del X, out, part
    torch.cuda.empty_cache()
