"""Calls without rows (a rank that got no tokens): a tensor of no elements has address 0, so
pointers that would be refused elsewhere are in order here, and nothing is launched (CPU)."""

import ctypes

import pytest

import moe_grouped_gemm_nt_amd as mgg
from moe_grouped_gemm_nt_amd.layer_ops import MggBlock

P, NUL = 1 << 20, None  # never dereferenced: there are no rows


@pytest.fixture(scope="module")
def lib():
    return mgg.load_library()


@pytest.mark.parametrize("G,k", [(16, 4), (288, 8)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("S,ends,counts,tokens,d_balance", [
    (1, NUL, NUL, NUL, NUL),  # d_weights alone, which has no elements
    (1, NUL, P, P, P), (3, P, P, P, P)])
def test_route_backward(lib, G, k, score, S, ends, counts, tokens, d_balance):
    status = lib.route_topk_backward(1, 0, G, k, NUL, G, score, 1, 1.0, S, ends, NUL, counts,
                                     tokens, NUL, d_balance, NUL, None)
    assert status == 0, lib.mgg_last_error()


def test_route_forward_without_counts(lib):
    status = lib.route_topk(1, 0, 16, 4, NUL, 16, NUL, 0, 1, 1.0, 1, NUL, NUL, NUL, NUL, NUL, NUL,
                            NUL, 0, None)
    assert status == 0, lib.mgg_last_error()


def test_block_forward(lib):
    b = MggBlock(0, 1, 0, 8, NUL, 8, NUL, 8, 1, NUL, 1, NUL, P, P, 1.0, 1.0, 1e-6)
    assert lib.block_residual_norm(ctypes.byref(b), NUL, NUL, None) == 0, lib.mgg_last_error()


def test_block_norm_forward(lib):
    assert lib.block_norm(0, 1, 0, 8, NUL, 8, P, 1e-6, NUL, None) == 0, lib.mgg_last_error()


def test_rows_without_gradients_stay_refused(lib):
    assert lib.route_topk_backward(1, 1, 16, 4, P, 16, 0, 1, 1.0, 1, NUL, P, NUL, NUL, NUL, NUL, P,
                                   None) == 1
    assert b"one of" in lib.mgg_last_error()
    # what has elements without rows is still asked for
    assert lib.route_topk_backward(1, 0, 16, 4, NUL, 16, 0, 1, 1.0, 1, NUL, NUL, NUL, NUL, NUL, P,
                                   NUL, None) == 1
    assert b"counts" in lib.mgg_last_error()
