"""Calls at the edges of the layer operators' ranges on the GPU."""

import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_batch_without_rows(dtype):
    """Every entry point that takes rows, forward and backward, with each gradient alone."""
    say(f"no rows {dtype}")
    l = torch.empty((0, 12), dtype=dtype, device=DEV)
    ids, w, counts, tokens, loss = mgg.route_topk(l, 3)
    assert not counts.any() and not tokens.any() and not loss.any()
    one = torch.ones(1, device=DEV)
    for dw, db in ((w, None), (None, one), (w, one)):
        assert mgg.route_topk_backward(l, ids, counts, tokens, dw, db).shape == (0, 12)
    x, p = torch.empty((0, 40), dtype=dtype, device=DEV), torch.ones(40, device=DEV)
    assert mgg.block_norm(x, p).shape == (0, 40)
    for dx in (x, None):
        d, dp = mgg.block_norm_backward(x, p, x, d_x=dx)
        assert d.shape == (0, 40) and not dp.any()
    for gate in (None, torch.empty(0, dtype=dtype, device=DEV), x):
        assert mgg.block_residual_norm(x, x, gate=gate)[0].shape == (0, 40)
        got = mgg.block_residual_norm_backward(x, x, d_x=x, gate=gate)
        assert got[0].shape == got[1].shape == (0, 40) and got[3:] == (None, None, None)
        got = mgg.block_residual_norm_backward(x, x, d_u=x, gate=gate, scale=p, w_after=p,
                                               w_before=p)
        assert not any(g.any() for g in got[3:])
