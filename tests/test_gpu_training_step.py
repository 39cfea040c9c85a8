"""The MoE training step of examples/moe_training_step.py on the GPU: forward values and every
gradient against the same step written with torch's float32 operations and autograd, routing
held fixed.

The step rounds its activations to bf16 (half a step is 2^-8 of a value) at each of about a
dozen places between an output and the inputs, independent errors that add in squares, and the
reference does not round there: relative errors (2-norm) stay below sqrt(12) 2^-8 = 0.0135."""

import os
import sys

import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg
from parity_util import say

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import moe_training_step as example  # noqa: E402

pytestmark = pytest.mark.gpu
BOUND = 0.0135


def rel(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


def reference(p, x, seq_ends, ids, counts, d_x, d_u):
    """The step in float32 with autograd, for the given choice of experts."""
    q = {k: v.float().requires_grad_() for k, v in p.items()}
    x = x.float().requires_grad_()
    T, k = ids.shape
    I = p["w2"].shape[2]
    G = p["router"].shape[0]

    def rms(v, w):
        return v * torch.rsqrt(v.pow(2).mean(1, keepdim=True) + example.EPS) * w

    u = rms(x, q["w_before"])
    prob = torch.softmax(u @ q["router"].t(), 1)
    live = (ids >= 0)
    at = ids.long().clamp(min=0)
    chosen = prob.gather(1, at) * live
    weights = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-30)
    y = torch.zeros_like(x)
    for e in range(G):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        h = u[t] @ q["w13"][e].t()
        a, b = h.split(I, 1)
        y = y.index_add(0, t, weights[t, j][:, None] * ((torch.nn.functional.silu(a) * b)
                                                        @ q["w2"][e].t()))
    gate = torch.sigmoid(u @ q["gate"])[:, None]
    out = x + q["scale"] * gate * rms(y, q["w_after"])
    u_next = rms(out, q["w_next"])
    total = (out * d_x.float()).sum() + (u_next * d_u.float()).sum()
    start = 0
    losses = []
    for s, end in enumerate(seq_ends.tolist()):
        n = end - start
        losses.append((G * counts[s].float() / (k * n) * prob[start:end].mean(0)).sum())
        start = end
    (total + example.BALANCE * torch.stack(losses).sum()).backward()
    return out, u_next, torch.stack(losses), dict({n: v.grad for n, v in q.items()}, x=x.grad)


@pytest.mark.parametrize("T,H,I,G,k,ends", [(96, 256, 128, 8, 2, [40, 96]),
                                            (130, 320, 64, 5, 3, [130]),
                                            (64, 128, 128, 16, 1, [10, 50])])
def test_step_against_float32(T, H, I, G, k, ends):
    say(f"training step {T} {H} {I} {G} {k}")
    p = example.make_params(H, I, G, seed=T)
    g = torch.Generator(device="cuda").manual_seed(7)
    x, d_x, d_u = (torch.randn((T, H), device="cuda", generator=g).bfloat16() for _ in range(3))
    seq_ends = torch.tensor(ends, dtype=torch.int32, device="cuda")
    if ends[-1] < T:  # padding rows take no part in the block's products or losses
        d_x[ends[-1]:] = 0
        d_u[ends[-1]:] = 0
    r = example.step(p, x, seq_ends, k, d_x, d_u)
    torch.cuda.synchronize()
    out, u_next, losses, grads = reference(p, x, seq_ends, r["ids"], r["counts"], d_x, d_u)
    n = ends[-1]
    assert rel(r["x_out"][:n], out[:n]) < BOUND and rel(r["u_next"][:n], u_next[:n]) < BOUND
    assert rel(r["balance"], losses) < BOUND
    assert set(r["grads"]) == set(grads)
    for name, want in grads.items():
        got = r["grads"][name]
        got, want = (got[:n], want[:n]) if name == "x" else (got, want)
        assert rel(got, want) < BOUND, (name, rel(got, want))
    # experts without tokens have a zero gradient and stay where they are
    idle = r["counts"].sum(0) == 0
    assert torch.equal(r["new"]["w2"][idle], p["w2"][idle])
    for d, o in zip((r["grads"]["w13"], r["grads"]["w2"]), r["updates"]):
        assert torch.equal(mgg.grouped_newton_schulz(d), o) and not o[idle].any()
