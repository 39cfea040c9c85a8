"""The binding's refusals of arguments that go together, reached before any device is asked for
(CPU, and the same beside a GPU)."""

import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg

X, W = torch.zeros(4, 8), torch.ones(8)


@pytest.mark.parametrize("call", [
    lambda: mgg.block_residual_norm(X, X, u=X),
    lambda: mgg.block_residual_norm(X, X, w_after=W, u=X),
    lambda: mgg.block_residual_norm_backward(X, X, d_x=X, d_u=X),
    lambda: mgg.block_residual_norm_backward(X, X, d_x=X, w_before=W),
])
def test_u_and_its_weight(call):
    with pytest.raises(ValueError, match="go together"):
        call()
