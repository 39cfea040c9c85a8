"""The smallest eps of the norms around a block: a normal float32. With a subnormal one the square
of 1 / sqrt(eps) is infinite, and a row of zeros got NaN gradients, an infinity times zero (CPU)."""

import ctypes

import numpy as np
import pytest

import moe_grouped_gemm_nt_amd as mgg
from moe_grouped_gemm_nt_amd.layer_ops import MggBlock

P = 1 << 20  # never dereferenced: every call below fails host validation or has no rows
LEAST = float(np.finfo(np.float32).tiny)


def calls(eps, T):
    lib = mgg.load_library()
    b = MggBlock(0, 1, T, 8, P, 8, P, 8, 0, None, 0, None, P, P, 1.0, 1.0, eps)
    yield lib.block_residual_norm(ctypes.byref(b), P, P, None)
    yield lib.block_norm(0, 1, T, 8, P, 8, P, eps, P, None)
    if T:
        big = 1 << 40
        yield lib.block_residual_norm_backward(ctypes.byref(b), P, 8, P, 8, P, P, None, None, P, P,
                                               P, big, None)
        yield lib.block_norm_backward(0, 1, T, 8, P, 8, P, eps, P, 8, P, 8, P, P, P, big, None)


@pytest.mark.parametrize("eps", [LEAST / 2, 1e-40, 1e-45, 0.0, -1e-6, float("inf"), float("nan")])
def test_refused(eps):
    for status in calls(eps, 4):
        assert status == 1 and b"eps" in mgg.load_library().mgg_last_error()


@pytest.mark.parametrize("eps", [LEAST, 1e-12, 1e-5, 1.0])
def test_accepted(eps):
    assert list(calls(eps, 0)) == [0, 0]


def test_square_of_the_largest_factor_is_finite():
    r = np.float32(1) / np.sqrt(np.float32(LEAST))
    assert np.isfinite(r * r)
    with np.errstate(over="ignore"):
        r = np.float32(1) / np.sqrt(np.float32(1e-40))
        assert np.isinf(r * r)
