"""The operators as a model runs them, one after the other.

Serving: a decoding step of an MoE layer - norm, router product, routing, shared expert, the chosen
experts, and the next layer's norm - against float64 arithmetic that takes over each operator's
rounded inputs from the GPU, so that every operator's own error is bounded (1e-2 of the output's
size in bf16: three half steps of 2^-8 at most meet in one operator), and the whole captured in a
graph and replayed for new tokens.
Training: a shared expert forward and backward, against float64 autograd of the same layer; bf16
operands are rounded at each of its three products, 2^-8 each, in norm."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg
from moe_grouped_gemm_nt_amd import synth
from oracle import layer_ops, products

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, I, G, K = 512, 256, 24, 4


def rel(got, want):
    got = got.double().cpu().numpy()
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def weights(seed):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, std):
        return (std * torch.randn(shape, generator=g)).bfloat16().to(DEV)
    w13, s13 = synth._weights("fp8", G, 2 * I, H, g, "cpu", "ue8m0", "block128", std=H ** -0.5)
    w2, s2 = synth._weights("fp8", G, H, I, g, "cpu", "ue8m0", "block128", std=I ** -0.5)
    p = dict(norm=1 + n(H, std=0.1).float(), next=1 + n(H, std=0.1).float(),
             router=n(G, H, std=H ** -0.5), shared13=n(2 * I, H, std=H ** -0.5),
             shared2=n(H, I, std=I ** -0.5), bias=n(G, std=0.1).float())
    p.update({k: v.to(DEV) for k, v in dict(w13=w13, s13=s13, w2=w2, s2=s2).items()})
    return p


def decode(p, x):
    u = mgg.block_norm(x, p["norm"])
    logits = mgg.linear_act(u, p["router"], p["bias"], out_dtype=torch.float32)
    ids, w = mgg.route_topk(logits, K, balance=False)
    hidden = mgg.linear_act(u, p["shared13"], func="swiglu")
    shared = mgg.linear_act(hidden, p["shared2"])
    y = mgg.moe_few_tokens(u, ids, w, p["w13"], p["w2"], p["s13"], p["s2"], residual=shared)
    x_out, u_next = mgg.block_residual_norm(x, y, w_before=p["next"])
    return dict(u=u, logits=logits, ids=ids, w=w, hidden=hidden, shared=shared, y=y, x_out=x_out,
                u_next=u_next)


@pytest.mark.parametrize("T", [1, 7, 80])
def test_decoding_step(T):
    p = weights(1)
    x = torch.randn((T, H), generator=torch.Generator().manual_seed(T)).bfloat16().to(DEV)
    r = decode(p, x)
    f = {k: v.double().cpu().numpy() for k, v in {**p, **r, "x": x}.items()
         if v.dtype != torch.uint8}
    assert rel(r["logits"], products.linear(f["u"], f["router"], f["bias"])[0]) < 1e-5
    ref = layer_ops.route(f["logits"], K)
    assert (r["ids"].cpu().numpy() == ref["ids"]).all()
    assert rel(r["hidden"], products.linear(f["u"], f["shared13"], None, "swiglu")[0]) < 1e-2
    assert rel(r["shared"], products.linear(f["hidden"], f["shared2"])[0]) < 1e-2
    w13 = products.expert_weights(p["w13"].cpu().numpy(), p["s13"].cpu().numpy(), "block128", "ue8m0")
    w2 = products.expert_weights(p["w2"].cpu().numpy(), p["s2"].cpu().numpy(), "block128", "ue8m0")
    y = products.moe_few_tokens(f["u"], ref["ids"], f["w"], w13, w2, f["shared"])
    assert rel(r["y"], y) < 1e-2
    end = layer_ops.block_residual_norm(f["x"], f["y"], w_before=f["next"])
    assert rel(r["x_out"], end["x_out"]) < 1e-2 and rel(r["u_next"], end["u"]) < 1e-2


def test_decoding_step_replayed():
    p = weights(2)
    x = torch.randn((5, H), device=DEV).bfloat16()
    decode(p, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = decode(p, x)
    for _ in range(4):
        x.copy_(torch.randn((5, H), device=DEV).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        eager = decode(p, x)
        assert all(torch.equal(captured[k], eager[k]) for k in eager)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [33, 300])
def test_shared_expert_training(dtype, T):
    g = torch.Generator().manual_seed(3)

    def n(*shape, std=1.0):
        return (std * torch.randn(shape, generator=g)).to(dtype).to(DEV)
    x, res, d = n(T, H), n(T, H), n(T, H)
    w13, w2, b13 = n(2 * I, H, std=H ** -0.5), n(H, I, std=I ** -0.5), n(2 * I, std=0.3).float()
    h, z = mgg.linear_act(x, w13, b13, "swiglu", keep_z=True)
    y = mgg.linear_act(h, w2, residual=res)
    d_h, d_w2, _ = mgg.linear_act_backward(h, w2, d)
    d_x, d_w13, d_b13 = mgg.linear_act_backward(x, w13, d_h, z, "swiglu", need_bias=True)
    leaf = [t.double().cpu().requires_grad_() for t in (x, w13, b13, w2, res)]
    a, u = (leaf[0] @ leaf[1].T + leaf[2]).chunk(2, 1)
    want = (torch.nn.functional.silu(a) * u) @ leaf[3].T + leaf[4]
    want.backward(d.double().cpu())
    tol = 1e-5 if dtype == torch.float32 else 3 * 2.0 ** -8
    assert rel(y, want.detach().numpy()) < tol
    for got, t in zip((d_x, d_w13, d_b13, d_w2, d), leaf):
        assert rel(got, t.grad.numpy()) < tol
