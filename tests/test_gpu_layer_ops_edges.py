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


def test_more_wide_rows_than_a_grid_has_threads_for():
    """2^22 rows of more than 8192 columns: a workgroup of 1024 threads for each row would be
    2^32 threads, which a launch does not hold (it took what was left past them, and seventy times
    as long). Right, and in no more than four times the time of a fourth of the rows, twice over
    for what else uses the memory meanwhile."""
    H, most = 8200, (1 << 22) + 3
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB")
    x = torch.zeros((most, H), dtype=torch.bfloat16, device=DEV)
    u = torch.empty((most, H), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(0)
    some = torch.tensor([0, 1, 5000, (1 << 20) - 1, 1 << 20, (1 << 22) - 1, 1 << 22, most - 1])
    rows = torch.randn((len(some), H), generator=g).to(torch.bfloat16).to(DEV)
    x[some.to(DEV)] = rows
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(DEV)

    def timed(T):
        mgg.block_norm(x[:T], w, u=u[:T])
        start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        mgg.block_norm(x[:T], w, u=u[:T])
        stop.record()
        torch.cuda.synchronize()
        return start.elapsed_time(stop)

    say(f"block norm {1 << 20} rows of {H}")
    fourth = timed(1 << 20)
    for T in (most, 1 << 22):
        say(f"block norm {T} rows of {H}")
        u.fill_(7.0)
        assert timed(T) <= 2 * 4 * fourth
        at = some[some < T].to(DEV)
        assert torch.equal(u[at], mgg.block_norm(rows[:len(at)], w))
        # all others are rows of zeros
        u[at] = 0
        for part in u[:T].split(1 << 19):
            assert not part.any()
        assert (u[T:] == 7).all()
    del x, u, part
    torch.cuda.empty_cache()
