"""One training step of an MoE block on one MI355X, from the kernels of this library: the norm
before the block, the router with its balance loss, the experts' grouped products, the end of
the block with its gate and residual scale, all gradients, and the orthogonalised update of the
experts' weights from their K-grouped gradients.

    python examples/moe_training_step.py [--tokens 4096 --hidden 2048 --inner 512 --experts 32 --topk 4]

What torch does here is what a model keeps in its own hands: gathering rows into expert order,
the gated activation, and the router's and gate's small dense products. Routing never visits
the host.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_grouped_gemm_nt_amd as mgg  # noqa: E402

EPS = 1e-6
BALANCE = 0.01  # weight of the balance loss


def make_params(H, I, G, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)

    def n(*shape, std=1.0, mean=0.0):
        return mean + std * torch.randn(shape, device=device, generator=g)

    return dict(
        w_before=n(H, std=0.1, mean=1.0), w_after=n(H, std=0.1, mean=1.0),
        w_next=n(H, std=0.1, mean=1.0), scale=n(H, std=0.05, mean=0.3),
        router=n(G, H, std=H ** -0.5), gate=n(H, std=H ** -0.5),
        w13=n(G, 2 * I, H, std=H ** -0.5).bfloat16(), w2=n(G, H, I, std=I ** -0.5).bfloat16())


class Dispatch:
    """Rows in expert order: row r of the experts' side is token token[r]'s choice, expert e owns
    the rows up to ends[e]; place[t, j] is the row of token t's j-th choice. Built on the device
    from ids and counts (ids of -1, padding tokens, go behind all experts)."""

    def __init__(self, ids, counts):
        T, k = ids.shape
        G = counts.shape[1]
        expert = torch.where(ids < 0, G, ids).reshape(-1)
        order = expert.sort(stable=True).indices
        self.token = order // k
        self.place = torch.empty_like(order).scatter_(
            0, order, torch.arange(T * k, device=ids.device)).view(T, k)
        self.counts = counts.sum(0)
        self.ends = self.counts.cumsum(0).to(torch.int32)
        # the K-grouped product packs each expert's tokens to a multiple of 8
        padded = (self.counts + 7) // 8 * 8
        self.k_ends = padded.cumsum(0).to(torch.int32)
        self.k_total = (T * k + 7) // 8 * 8 + 8 * G
        e = expert[order].clamp(max=G - 1)
        start = self.k_ends.long() - padded
        within = torch.arange(T * k, device=ids.device) - (self.ends.long() - self.counts)[e]
        self.live = expert[order] < G
        self.k_start, self.k_len, self.k_at = start[e], padded[e], within

    def pack(self, rows):
        """[R, M] rows of all experts -> the K-grouped operand: for each expert [M][k_e]."""
        M = rows.shape[1]
        flat = rows.new_zeros(M * self.k_total + 1)
        at = (M * self.k_start + self.k_at)[:, None] + \
            self.k_len[:, None] * torch.arange(M, device=rows.device)[None, :]
        flat[torch.where(self.live[:, None], at, M * self.k_total).reshape(-1)] = rows.reshape(-1)
        return flat[:-1]


def experts(rows, weights, ends):
    """rows [R, K] in expert order times each expert's weights [N, K], transposed."""
    out = rows.new_zeros((rows.shape[0], weights.shape[1]))
    return mgg.grouped_gemm_contiguous_psum(rows, weights, out, ends)


def weight_gradient(d, out_rows, in_rows, M, N):
    D = torch.empty((d.ends.numel(), M, N), device=in_rows.device)
    return mgg.grouped_gemm_kgrouped(d.pack(out_rows), d.pack(in_rows), D, d.k_ends, M, N,
                                     accumulate=False, psum=True)


def step(p, x, seq_ends, topk, d_x, d_u, lr=0.02):
    """Forward, backward for the gradients d_x of the new stream and d_u of the next block's
    input, and the update. Returns everything that a caller might look at."""
    T, H = x.shape
    G, I = p["router"].shape[0], p["w2"].shape[2]

    # ---- forward
    u = mgg.block_norm(x, p["w_before"], EPS)
    logits = u.float() @ p["router"].t()
    ids, weights, counts, tokens, balance = mgg.route_topk(logits, topk, seq_ends=seq_ends)
    d = Dispatch(ids, counts)
    rows = u[d.token]
    h = experts(rows, p["w13"], d.ends)
    a, b = h.float().split(I, 1)
    sig = torch.sigmoid(a)
    act = (a * sig * b).bfloat16()
    out_rows = experts(act, p["w2"], d.ends)
    y = (weights[..., None] * out_rows[d.place].float()).sum(1).bfloat16()
    gate = (u.float() @ p["gate"]).bfloat16()
    x_out, u_next = mgg.block_residual_norm(x, y, w_after=p["w_after"], gate=gate,
                                            scale=p["scale"], w_before=p["w_next"], eps=EPS)

    # ---- backward
    d_in, d_y, d_gate, d_scale, d_w_after, d_w_next = mgg.block_residual_norm_backward(
        x_out, y, d_x, d_u, w_after=p["w_after"], gate=gate, scale=p["scale"],
        w_before=p["w_next"], eps=EPS)
    d_weights = (out_rows[d.place].float() * d_y.float()[:, None]).sum(2)
    row_weight = torch.zeros_like(d.token, dtype=torch.float32).scatter_(
        0, d.place.reshape(-1), weights.reshape(-1))
    d_out_rows = (row_weight[:, None] * d_y[d.token].float()).bfloat16()
    d_w2 = weight_gradient(d, d_out_rows, act, H, I)
    d_act = experts(d_out_rows, p["w2"].transpose(1, 2).contiguous(), d.ends).float()
    d_h = torch.cat([d_act * b * sig * (1 + a * (1 - sig)), d_act * a * sig], 1).bfloat16()
    d_w13 = weight_gradient(d, d_h, rows, 2 * I, H)
    d_rows = experts(d_h, p["w13"].transpose(1, 2).contiguous(), d.ends)
    d_logits = mgg.route_topk_backward(
        logits, ids, counts, tokens, d_weights, torch.full_like(balance, BALANCE),
        seq_ends=seq_ends)
    d_router = d_logits.t() @ u.float()
    d_u_in = (d_rows[d.place].float().sum(1) + d_logits @ p["router"]
              + d_gate.float()[:, None] * p["gate"]).bfloat16()
    d_gate_w = d_gate.float() @ u.float()
    d_x_in, d_w_before = mgg.block_norm_backward(x, p["w_before"], d_u_in, d_in, EPS)

    # ---- the experts' weights move along their orthogonalised gradients
    o13, o2 = mgg.grouped_newton_schulz(d_w13), mgg.grouped_newton_schulz(d_w2)
    new = dict(p, w13=(p["w13"].float() - lr * o13).bfloat16(),
               w2=(p["w2"].float() - lr * o2).bfloat16())
    return dict(x_out=x_out, u_next=u_next, ids=ids, weights=weights, counts=counts,
                balance=balance, new=new, updates=(o13, o2), grads=dict(
                    x=d_x_in, w_before=d_w_before, w_after=d_w_after, w_next=d_w_next,
                    scale=d_scale, router=d_router, gate=d_gate_w, w13=d_w13, w2=d_w2))


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inner", 512), ("experts", 32),
                        ("topk", 4), ("sequences", 4), ("steps", 5)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    p = make_params(a.hidden, a.inner, a.experts)
    g = torch.Generator(device="cuda").manual_seed(1)

    def draw():
        return torch.randn((a.tokens, a.hidden), device="cuda", generator=g).bfloat16()

    x, d_x, d_u = draw(), draw() * 1e-3, draw() * 1e-3
    ends = (torch.arange(1, a.sequences + 1, device="cuda") * a.tokens // a.sequences).int()
    for i in range(a.steps):
        start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        r = step(p, x, ends, a.topk, d_x, d_u)
        stop.record()
        torch.cuda.synchronize()
        c = r["counts"].sum(0)
        print(f"step {i}: {start.elapsed_time(stop):.2f} ms, balance loss "
              f"{r['balance'].mean().item():.4f}, tokens per expert {c.min().item()}.."
              f"{c.max().item()}, |d_x| {r['grads']['x'].float().norm().item():.4e}", flush=True)
        p = r["new"]


if __name__ == "__main__":
    main()
