"""Experts that a bias forces into the choice although their scores are many orders below the
row's best: the weights are shares of the chosen scores, whatever their size, and the gradient
goes through those shares. Tolerances are those of test_gpu_route.py."""

import pytest
import torch

from parity_util import say
from test_gpu_route import check_backward, check_forward, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [-20.0, -60.0, -80.0, -86.0, -88.0, -100.0, -900.0, -3e38])
@pytest.mark.parametrize("G,k", [(24, 4), (288, 8), (320, 17), (500, 6), (900, 32)])
def test_forced_choice(G, k, at, dtype):
    say(f"route forced {G} {k} {at} {dtype}")
    l = logits_of(37, G, dtype, G + k, 1.0)
    b = torch.zeros(G)
    forced = [(5 * j + 3) % G for j in range(k)]
    b[forced] = 1e3
    rows = slice(0, 30)
    for i, e in enumerate(forced):
        l[rows, e] = at + (1.5 * i if at > -1e3 else 0.0)
    l[20, :] = at               # a row without any other
    l[21, forced[0]] = 2.0      # one of them next to the row's best
    for renorm in (True, False):
        fwd = check_forward(l, k, ends=[10, 37], bias=b, score="sigmoid", renorm=renorm, scale=2.5)
        assert sorted(fwd[0][0].tolist()) == sorted(forced)
        if renorm:
            total = fwd[1].double().sum(1)
            assert (total - 2.5).abs().max() < 1e-5
        check_backward(l, k, ends=[10, 37], score="sigmoid", renorm=renorm, scale=2.5, fwd=fwd)
