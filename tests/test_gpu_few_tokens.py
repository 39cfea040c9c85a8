"""The MoE layer for few tokens on the GPU against its float64 definition.

Tolerances: oracle.products.moe_few_tokens counts, with u = 2^-24, one rounding for each term of a
float32 sum, those of the gated unit, and of what stands between the products the half step 2^-8 of
one bfloat16 (bf16 outputs, as between the grouped products) or the 2^-24 of three (float32
outputs); a bf16 output adds half a step of its own, 2^-8 of the value."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg
from moe_grouped_gemm_nt_amd import synth
from oracle import products as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24

FORMS = ["bf16", "fp8/block128/f32", "fp8/block128/ue8m0", "fp8/channel/f32", "fp8/channel/ue8m0",
         "fp4/block32/ue8m0"]


class Layer:
    """Expert weights of a form, on the CPU, on the GPU and in float64."""

    def __init__(self, form, G, H, I, seed):
        self.G, self.H, self.I = G, H, I
        kind, self.gran, fmt = (form.split("/") + [None, None])[:3]
        gen = torch.Generator().manual_seed(seed)
        self.kw, self.f64, self.w = {}, {}, {}
        for name, N, K in (("13", 2 * I, H), ("2", H, I)):
            codes, s = synth._weights("fp8_fp4" if kind == "fp4" else kind, G, N, K, gen, "cpu", fmt,
                                      self.gran, std=K ** -0.5)
            v = codes.double().numpy() if kind == "bf16" else \
                ref.expert_weights(codes.numpy(), s.numpy(), self.gran, fmt)
            self.f64[name], self.w[name] = v, codes.to(DEV)
            self.kw["s" + name] = None if s is None else s.to(DEV)
        if self.gran:
            self.kw["sfb_gran"] = self.gran

    def __call__(self, x, ids, weights, **kw):
        return mgg.moe_few_tokens(x, ids, weights, self.w["13"], self.w["2"], **self.kw, **kw)

    def check(self, x, ids, weights, got, residual=None):
        want, err = ref.moe_few_tokens(
            x.double().cpu().numpy(), ids.cpu().numpy(), weights.double().cpu().numpy(),
            self.f64["13"], self.f64["2"],
            None if residual is None else residual.double().cpu().numpy(), roundings=U,
            held=2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24)
        if got.dtype == torch.bfloat16:
            err = err + 2.0 ** -8 * np.abs(want)
        off = np.abs(got.double().cpu().numpy() - want)
        assert (off <= err + 1e-37).all(), (off / (err + 1e-37)).max()


def tokens(T, k, G, H, seed, empty=0.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=gen).bfloat16()
    ids = torch.rand((T, G), generator=gen).argsort(1)[:, :k].to(torch.int32) if k <= G else \
        torch.randint(0, G, (T, k), generator=gen, dtype=torch.int32)
    weights = torch.rand((T, k), generator=gen)
    gone = torch.rand((T, k), generator=gen) < empty
    return x.to(DEV), torch.where(gone, -1, ids).to(DEV), weights.to(DEV)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,k,G,H,I", [
    (1, 1, 1, 128, 128), (1, 8, 40, 512, 256), (3, 2, 5, 640, 128), (17, 2, 3, 256, 384),
    (40, 3, 4, 384, 128), (70, 2, 2, 128, 256)])
def test_forms(form, T, k, G, H, I):
    print(form, T, k, G, H, I, flush=True)
    layer = Layer(form, G, H, I, T + 1)
    x, ids, w = tokens(T, k, G, H, T)
    res = torch.randn((T, H), device=DEV).bfloat16()
    layer.check(x, ids, w, layer(x, ids, w, residual=res), res)
    layer.check(x, ids, w, layer(x, ids, w, out_dtype=torch.float32))


@pytest.mark.parametrize("T,k,G,H,I", [
    (1, 2, 3, 8, 8), (2, 1, 2, 24, 40), (5, 3, 9, 200, 72), (33, 2, 7, 1000, 8), (64, 4, 9, 72, 136),
    (65, 1, 1, 136, 24), (128, 2, 6, 64, 72), (31, 32, 5, 64, 16), (128, 32, 4096, 8, 8),
    (100, 8, 900, 40, 16), (3, 2, 4, 8208, 16), (1, 1, 2, 65536, 8),
    (5, 2, 3, 16, 65536)])
def test_odd_sizes(T, k, G, H, I):
    """Widths off the blocks of K and of the workgroups; places that the router left empty; more
    tokens of one expert than are held at once; as many places and experts as are allowed."""
    print(T, k, G, H, I, flush=True)
    layer = Layer("bf16", G, H, I, T)
    x, ids, w = tokens(T, k, G, H, 3 * T, empty=0.3)
    res = torch.randn((T, H), device=DEV)
    got = layer(x, ids, w, residual=res, out_dtype=torch.float32)
    layer.check(x, ids, w, got, res)


@pytest.mark.parametrize("form", ["bf16", "fp8/block128/f32", "fp4/block32/ue8m0"])
def test_all_tokens_to_one_expert(form):
    layer = Layer(form, 9, 256, 128, 5)
    x, ids, w = tokens(120, 3, 9, 256, 6)
    ids[:, 1:] = -1
    ids[:, 0] = 7
    layer.check(x, ids, w, layer(x, ids, w, out_dtype=torch.float32))


@pytest.mark.parametrize("T,k,G", [(6, 4, 3), (6, 4, 300), (40, 5, 2)])
def test_same_expert_twice(T, k, G):
    """An expert that a token names more than once counts with the sum of its weights."""
    layer = Layer("bf16", G, 64, 32, 8)
    x, ids, w = tokens(T, k, G, 64, 9)
    ids[:, 1] = ids[:, 0]
    ids[T // 2:] = ids[T // 2:, :1]
    layer.check(x, ids, w, layer(x, ids, w, out_dtype=torch.float32))


def test_ids_outside_and_empty_batches():
    layer = Layer("bf16", 4, 64, 32, 10)
    x, ids, w = tokens(7, 3, 4, 64, 11)
    ids[0] = torch.tensor([-1, 4, -2 ** 31])
    ids[1] = torch.tensor([2 ** 31 - 1, 3, -5])
    w[0] = float("nan")  # whatever stands at an empty place has no effect
    w[1, 0] = float("inf")
    res = torch.randn((7, 64), device=DEV).bfloat16()
    got = layer(x, ids, w, residual=res)
    assert torch.equal(got[0], res[0])
    layer.check(x, ids, torch.where((ids < 0) | (ids > 3), 0.0, w), got, res)
    none = layer(x, torch.full_like(ids, -1), w)
    assert not none.any()
    assert layer(x[:0], ids[:0], w[:0]).shape == (0, 64)


@pytest.mark.parametrize("offset,ld", [(0, 300), (1, 301), (3, 263)])
def test_strides(offset, ld):
    """Rows of x and of the residual anywhere in wider tensors, what lies between them NaN."""
    T, H = 20, 256
    layer = Layer("fp8/channel/f32", 5, H, 128, 12)
    x, ids, w = tokens(T, 2, 5, H, 13)
    res = torch.randn((T, H), device=DEV).bfloat16()

    def wide(t):
        buf = torch.full((offset + T * ld,), float("nan"), dtype=t.dtype, device=DEV)
        view = buf[offset:].view(T, ld)[:, :H]
        view.copy_(t)
        return view
    a = layer(x, ids, w, residual=res)
    assert torch.equal(layer(wide(x), ids, w, residual=wide(res)), a)


@pytest.mark.parametrize("form", ["bf16", "fp8/block128/ue8m0", "fp4/block32/ue8m0"])
def test_isolation(form):
    """Experts that nobody names, other tokens and old workspaces have no effect; an infinity or
    NaN in a token stays in its row."""
    T, k, G, H, I = 12, 2, 9, 256, 128
    layer = Layer(form, G, H, I, 14)
    x, ids, w = tokens(T, k, 4, H, 15)
    size = mgg.load_library().moe_few_tokens_workspace(T, k, G, I)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    a = layer(x, ids, w)
    layer.w["13"].view(torch.uint8)[4:] = 0x7F
    layer.w["2"].view(torch.uint8)[4:] = 0x7F
    if layer.kw["s13"] is not None:
        layer.kw["s13"].view(torch.uint8)[4:] = 255
        layer.kw["s2"].view(torch.uint8)[4:] = 255
    room = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device=DEV)
    assert torch.equal(layer(x, ids, w, workspace=ws, out=room[1:-1]), a)
    assert (room[0] == 7).all() and (room[-1] == 7).all()
    bad = x.clone()
    bad[3, 5], bad[8, 200] = float("nan"), float("inf")
    b = layer(bad, ids, w)
    rest = [t for t in range(T) if t not in (3, 8)]
    assert torch.equal(b[rest], a[rest]) and b[3].isnan().all() and not b[8].isfinite().all()


def test_large_values():
    """silu far out on both sides; h beyond bfloat16 stays infinite, not NaN."""
    layer = Layer("bf16", 2, 64, 16, 16)
    x, ids, w = tokens(4, 1, 2, 64, 17)
    x *= 1000.0
    layer.check(x, ids, w, layer(x, ids, w, out_dtype=torch.float32))
    layer.w["13"].fill_(1.0)
    layer.w["2"].fill_(1.0)
    x.fill_(1e18)
    got = layer(x, ids, w.abs() + 0.5, out_dtype=torch.float32)
    assert (got == float("inf")).all()
    x.fill_(-1e18)  # silu is 0 there
    assert (layer(x, ids, w, out_dtype=torch.float32) == 0).all()


def test_bitwise_repeats_and_graph_replays():
    """Equal bits from call to call; a graph reads the ids of its replay; two graphs that share a
    workspace, replayed in turn."""
    T, k, G, H, I = 9, 2, 40, 512, 256
    layer = Layer("fp8/block128/f32", G, H, I, 18)
    x, ids, w = tokens(T, k, G, H, 19)
    ws = torch.empty(mgg.load_library().moe_few_tokens_workspace(T, k, G, I), dtype=torch.uint8,
                     device=DEV)
    first = layer(x, ids, w)
    for _ in range(20):
        assert torch.equal(layer(x, ids, w, workspace=ws), first)
    outs = [torch.empty_like(first) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    xs = [x, x.flip(0).contiguous()]
    with torch.cuda.stream(side):
        for graph, out, xi in zip(graphs, outs, xs):
            with torch.cuda.graph(graph, stream=side):
                layer(xi, ids, w, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for seed in range(4):
        _, new, nw = tokens(T, k, G, H, 100 + seed, empty=0.2)
        ids.copy_(new)
        w.copy_(nw)
        for graph, out, xi in zip(graphs, outs, xs):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, layer(xi, ids, w))


def test_streams():
    """Calls on two streams at once, each with a workspace of its own."""
    layer = Layer("bf16", 6, 1024, 512, 20)
    inputs = [tokens(30, 2, 6, 1024, 21 + i) for i in range(2)]
    want = [layer(*i) for i in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(*inputs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_refusals_on_the_gpu():
    layer = Layer("bf16", 4, 64, 32, 22)
    x, ids, w = tokens(3, 2, 4, 64, 23)
    with pytest.raises(ValueError, match="same GPU"):
        layer(x, ids.cpu(), w)
    with pytest.raises(ValueError, match="workspace"):
        layer(x, ids, w, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="out must be"):
        layer(x, ids, w, out=torch.empty((4, 64), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError, match="residual must be"):
        layer(x, ids, w, residual=torch.empty((3, 64), device=DEV))
    with pytest.raises(mgg.MggError, match="T must be"):
        layer(*tokens(129, 1, 4, 64, 24))
