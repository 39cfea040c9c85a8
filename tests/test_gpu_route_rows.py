"""Routing of a training batch: more rows than one pass of all workgroups, ragged sequences with
padded ends, counts and losses and both gradients. Tolerances
are those of test_gpu_route.py (a lane adds at most cdiv(T, 512) / 4 rows of a workgroup, 36 at
most here, of the 128 roundings that its sums over rows are given)."""

import pytest
import torch

from parity_util import say
from test_gpu_route import check_backward, check_forward, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [65535, 65536, 70001])
@pytest.mark.parametrize("G,k,dtype,score", [(40, 4, torch.float32, "softmax"),
                                             (33, 3, torch.bfloat16, "sigmoid")])
def test_training_batch(T, G, k, dtype, score):
    cuts = torch.randint(0, T - 900, (15,), generator=torch.Generator().manual_seed(T + G))
    ends = sorted(cuts.tolist()) + [T - 700]
    say(f"route batch {T} {G} {dtype} {score}")
    l = logits_of(T, G, dtype, T)
    fwd = check_forward(l, k, ends=ends, score=score)
    check_backward(l, k, ends=ends, score=score, fwd=fwd)
    if score == "sigmoid":
        b = 0.2 * torch.randn(G, generator=torch.Generator().manual_seed(1))
        check_forward(l, k, ends=ends, score=score, bias=b)


def test_training_batch_of_many_experts():
    T, G = 65537, 288
    say(f"route batch {T} {G}")
    l = logits_of(T, G, torch.float32, 3)
    ends = [1, 20000, 20000, 41001, 65000]
    fwd = check_forward(l, 8, ends=ends)
    check_backward(l, 8, ends=ends, fwd=fwd)


@pytest.mark.parametrize("G", [1, 2, 15, 31, 32, 33, 48, 63, 95, 96, 97, 127, 159, 161, 191, 193,
                               223, 224, 225, 257, 287, 289, 319])
def test_every_slot_count(G):
    """Expert counts on both sides of every number of slots that a lane holds."""
    say(f"route slots {G}")
    for dtype, score in ((torch.float32, "softmax"), (torch.bfloat16, "sigmoid")):
        l = logits_of(45, G, dtype, 7 * G)
        for k in {1, min(G, 8)}:
            fwd = check_forward(l, k, ends=[17, 40], score=score)
            check_backward(l, k, ends=[17, 40], score=score, fwd=fwd)
        b = 0.2 * torch.randn(G, generator=torch.Generator().manual_seed(G))
        check_forward(l, min(G, 6), score="sigmoid", bias=b)
