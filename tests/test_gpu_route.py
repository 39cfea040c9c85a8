"""Routing with its balance loss on the GPU against the float64 definitions.

Tolerances count float32 roundings, u = 2^-24. A logit's distance from the row's maximum is
rounded once, which e^x turns into that many relative u; the exponential, a division and the
final products add about ten, and a sum over the row one for each addend that a lane adds (at
most 64) and one for each halving of the lanes (six). So a probability or weight is within
C = 2 * range + 96 roundings, with `range` the largest distance met. Gradients are differences:
the same C, relative to the sum of the absolute values of their terms. bf16 gradients add half
a step, 2^-8 of the value."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg
from oracle import layer_ops as ref
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def logits_of(T, G, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn((T, G), generator=g)).to(dtype)


def roundings(l):
    fin = l[np.isfinite(l) & (np.abs(l) < 1e3)]
    return 2 * (fin.max() - fin.min() if fin.size else 0.0) + 96


def check_forward(l, k, ends=None, bias=None, score="softmax", renorm=True, scale=1.0,
                  got=None):
    T, G = l.shape
    ends_t = None if ends is None else torch.tensor(ends, dtype=torch.int32, device=DEV)
    bias_t = None if bias is None else bias.to(DEV)
    kw = dict(bias=bias_t, seq_ends=ends_t, score=score, renormalize=renorm, scale=scale)
    lg = l.to(DEV)
    ids, w, counts, tokens, bal = got or mgg.route_topk(lg, k, **kw)
    torch.cuda.synchronize()
    r = ref.route(l.double().numpy(), k, score, renorm, scale,
                  None if bias is None else bias.double().numpy(), ends)
    assert (ids.cpu().numpy() == r["ids"]).all()
    assert (counts.cpu().numpy() == r["counts"]).all()
    assert (tokens.cpu().numpy() == r["tokens"]).all()
    c = roundings(l.double().numpy())
    np.testing.assert_allclose(w.cpu().numpy(), r["weights"], rtol=c * U, atol=1e-37)
    # the sum over rows adds one rounding for each of the few rows that a lane adds up
    np.testing.assert_allclose(bal.cpu().numpy(), r["balance"], rtol=(c + 128) * U, atol=1e-37)
    if got is None:
        i2, w2 = mgg.route_topk(lg, k, balance=False, **kw)
        assert torch.equal(i2, ids) and torch.equal(w2, w)
    return ids, w, counts, tokens, bal


def check_backward(l, k, ends=None, score="softmax", renorm=True, scale=1.0, use=("w", "b"),
                   seed=0, fwd=None):
    T, G = l.shape
    S = 1 if ends is None else len(ends)
    g = torch.Generator().manual_seed(seed + 77)
    dw = torch.randn((T, k), generator=g) if "w" in use else None
    db = torch.randn(S, generator=g) if "b" in use else None
    ends_t = None if ends is None else torch.tensor(ends, dtype=torch.int32, device=DEV)
    lg = l.to(DEV)
    ids, _, counts, tokens, _ = fwd or mgg.route_topk(lg, k, seq_ends=ends_t, score=score,
                                                      renormalize=renorm, scale=scale)
    d = mgg.route_topk_backward(lg, ids, counts, tokens,
                                None if dw is None else dw.to(DEV),
                                None if db is None else db.to(DEV), seq_ends=ends_t, score=score,
                                renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    ln = l.double().numpy()
    want, mag = ref.route_grad(ln, ids.cpu().numpy(), counts.cpu().numpy(), tokens.cpu().numpy(),
                               None if dw is None else dw.double().numpy(),
                               None if db is None else db.double().numpy(), score, renorm, scale,
                               ends)
    half = 2.0 ** -8 if l.dtype == torch.bfloat16 else 0.0
    off = np.abs(d.double().cpu().numpy() - want)
    assert (off <= 2 * roundings(ln) * U * mag + half * np.abs(want) + 1e-37).all(), \
        (off / (mag + 1e-300)).max()
    return d


SHAPES = [(1, 1, 1), (3, 5, 5), (17, 8, 2), (70, 64, 8), (33, 65, 3), (129, 128, 6),
          (50, 255, 8), (200, 288, 8), (31, 320, 4), (40, 321, 8), (20, 512, 32), (21, 1000, 16),
          (9, 2048, 8), (6, 4096, 32)]


@pytest.mark.parametrize("T,G,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_shapes(T, G, k, dtype, score):
    say(f"route {T} {G} {k} {dtype} {score}")
    l = logits_of(T, G, dtype, T + G)
    for renorm in (True, False):
        check_forward(l, k, score=score, renorm=renorm, scale=2.5)
        check_backward(l, k, score=score, renorm=renorm, scale=2.5, seed=G)


@pytest.mark.parametrize("G,k", [(16, 4), (288, 6), (700, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bias(G, k, dtype):
    say(f"route bias {G} {k} {dtype}")
    l = logits_of(60, G, dtype, G)
    b = 0.3 * torch.randn(G, generator=torch.Generator().manual_seed(5))
    fwd = check_forward(l, k, bias=b, score="sigmoid", ends=[20, 60])
    check_backward(l, k, ends=[20, 60], score="sigmoid", fwd=fwd)
    b[3], b[5] = float("-inf"), float("nan")
    ids = check_forward(l, k, bias=b, score="sigmoid")[0]
    assert not ((ids == 3) | (ids == 5)).any()


ENDS = [[40], [0, 0, 100], [100, 100, 100], [1, 2, 3, 50], [60, 30, 90], [-5, 200], [0],
        [17, 17, 16, 64, 65, 100], list(range(1, 101))]


@pytest.mark.parametrize("ends", ENDS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sequences(ends, score):
    say(f"route ends {ends[:6]} {score}")
    l = logits_of(100, 24, torch.float32, 3)
    check_forward(l, 3, ends=ends, score=score)
    for use in (("w", "b"), ("w",), ("b",)):
        check_backward(l, 3, ends=ends, score=score, use=use)


def test_many_rows_and_sequences():
    """More rows than one pass of the workgroups, with sequences that end inside chunks, at
    their borders, and several in one chunk."""
    T = 20000
    cuts = torch.randint(0, T + 1, (300,), generator=torch.Generator().manual_seed(1))
    ends = sorted(cuts.tolist()) + [T - 3]
    for dtype, G, k in [(torch.float32, 40, 4), (torch.bfloat16, 288, 8)]:
        say(f"route rows {T} {G}")
        l = logits_of(T, G, dtype, 9)
        check_forward(l, k, ends=ends)
        check_backward(l, k, ends=ends)


def test_sequence_counts_beyond_a_workgroup():
    ends = sorted(torch.randint(0, 900, (1500,), generator=torch.Generator().manual_seed(2)).tolist())
    say("route 1500 sequences")
    l = logits_of(1000, 12, torch.float32, 4)
    check_forward(l, 2, ends=ends)
    check_backward(l, 2, ends=ends)


def test_no_rows():
    say("route no rows")
    l = torch.zeros(0, 12)
    for ends in (None, [0], [0, 3]):
        ids, w, counts, tokens, bal = check_forward(l, 2, ends=ends)
        assert ids.shape == (0, 2) and not counts.any() and not bal.any()
    lg = l.to(DEV)
    d = mgg.route_topk_backward(lg, ids, counts, tokens, w, torch.ones(2, device=DEV),
                                seq_ends=torch.tensor([0, 3], dtype=torch.int32, device=DEV))
    assert d.shape == (0, 12)


def test_masked_and_equal_logits():
    """Unavailable experts, rows without any, rows of the lowest value, equal logits."""
    inf = float("inf")
    low32, low16 = torch.finfo(torch.float32).min, torch.finfo(torch.bfloat16).min
    for dtype, low in ((torch.float32, low32), (torch.bfloat16, low16)):
        l = logits_of(40, 37, dtype, 8)
        l[0] = -inf
        l[1, :] = -inf
        l[1, 36] = 0.5
        l[2, 5:] = -inf
        l[3] = low
        l[4, 1:] = low
        l[5] = 2.0
        l[6, 10:20] = 9.0
        l[7] = -200.0
        l[8] = torch.linspace(-150, -90, 37).to(dtype)
        l[9, ::2] = 0.0
        l[9, 1::2] = -0.0
        l[10] = 100.0
        for score in ("softmax", "sigmoid"):
            say(f"route masked {dtype} {score}")
            for renorm in (True, False):
                fwd = check_forward(l, 6, score=score, renorm=renorm, ends=[20, 40])
                check_backward(l, 6, score=score, renorm=renorm, ends=[20, 40], fwd=fwd)
            assert fwd[0][0].tolist() == [-1] * 6 and fwd[0][1].tolist() == [36] + [-1] * 5
            assert fwd[0][5].tolist() == list(range(6)) == fwd[0][9].tolist()
            assert fwd[0][6].tolist() == list(range(10, 16))


def test_nan_and_infinite_logits():
    """A NaN is never taken, stays in its own row, and shows in its sequence's loss only."""
    l = logits_of(20, 30, torch.float32, 6)
    clean = mgg.route_topk(l.to(DEV), 4, seq_ends=torch.tensor([10, 20], dtype=torch.int32, device=DEV))
    l[3, 7] = float("nan")
    say("route nan")
    for score in ("softmax", "sigmoid"):
        ids, w, counts, tokens, bal = mgg.route_topk(
            l.to(DEV), 4, score=score,
            seq_ends=torch.tensor([10, 20], dtype=torch.int32, device=DEV))
        assert not (ids[3] == 7).any() and torch.isnan(bal).tolist() == [True, False]
        assert ids[3].tolist() == ref.route(l.double().numpy(), 4, score)["ids"][3].tolist()
        if score == "softmax":
            keep = [t for t in range(20) if t != 3]
            assert torch.equal(w[keep], clean[1][keep]) and torch.equal(ids[keep], clean[0][keep])
            assert bal[1] == clean[4][1]
    l[3, 7] = float("inf")
    ids, w = mgg.route_topk(l.to(DEV), 4, balance=False)
    assert ids[3, 0] == 7 and torch.isnan(w[3]).all() and torch.isfinite(w[4:]).all()
    ids, w = mgg.route_topk(l.to(DEV), 4, balance=False, score="sigmoid", renormalize=False)
    assert ids[3, 0] == 7 and w[3, 0] == 1.0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("start,pad", [(0, 3), (1, 2), (3, 5)])
def test_strided_and_shifted_rows(dtype, start, pad):
    say(f"route strided {dtype} {start} {pad}")
    G = 50
    wide = logits_of(33, start + G + pad, dtype, 12)
    l = wide[:, start:start + G]
    view = wide.to(DEV)[:, start:start + G]
    check_forward(l.contiguous(), 5, got=mgg.route_topk(view, 5))
    a = mgg.route_topk(view, 5)
    dw = torch.randn((33, 5), generator=torch.Generator().manual_seed(1)).to(DEV)
    d1 = mgg.route_topk_backward(view, a[0], d_weights=dw)
    d2 = mgg.route_topk_backward(view.contiguous(), a[0], d_weights=dw)
    assert torch.equal(d1, d2)


def test_gradient_against_differences():
    """The losses that the GPU computes, moved along random directions in float64 steps of
    the definition, change as the GPU's gradient says."""
    l = logits_of(64, 48, torch.float32, 21, 1.0)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            say(f"route differences {score} {renorm}")
            ids, w, counts, tokens, bal = mgg.route_topk(l.to(DEV), 4, score=score,
                                                         renormalize=renorm)
            dw = torch.randn((64, 4), generator=torch.Generator().manual_seed(2))
            db = torch.tensor([3.0])
            d = mgg.route_topk_backward(l.to(DEV), ids, counts, tokens, dw.to(DEV), db.to(DEV),
                                        score=score, renormalize=renorm).cpu().double().numpy()

            def loss(v):
                r = ref.route(v, 4, score, renorm)
                same = (r["ids"] == ids.cpu().numpy()).all(1)
                assert same.all()
                return (r["weights"] * dw.double().numpy()).sum() + 3.0 * r["balance"].sum()

            base = l.double().numpy()
            for seed in range(4):
                v = np.random.default_rng(seed).normal(size=base.shape)
                h = 1e-6
                num = (loss(base + h * v) - loss(base - h * v)) / (2 * h)
                # the difference's own error is about 1e-16 / h of the loss; the gradient's
                # C roundings of each of its terms
                assert abs((d * v).sum() - num) <= 1e-8 + 128 * U * np.abs(d * v).sum()


def test_results_repeat_and_workspaces_may_hold_anything():
    l = logits_of(3000, 96, torch.float32, 30).to(DEV)
    ends = torch.tensor([100, 1500, 2900], dtype=torch.int32, device=DEV)
    size = mgg.load_library().route_topk_workspace(3000, 96, 3)
    say("route repeat")
    first = mgg.route_topk(l, 6, seq_ends=ends)
    for fill in (0, 255, 127):
        ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        again = mgg.route_topk(l, 6, seq_ends=ends, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_graph_replays_follow_inputs():
    T, G, k = 700, 72, 5
    l = logits_of(T, G, torch.bfloat16, 40).to(DEV)
    ends = torch.tensor([300, 650], dtype=torch.int32, device=DEV)
    dw = torch.ones((T, k), device=DEV)
    db = torch.ones(2, device=DEV)

    def step():
        out = mgg.route_topk(l, k, seq_ends=ends)
        return out + (mgg.route_topk_backward(l, out[0], out[2], out[3], dw, db, seq_ends=ends),)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        say(f"route replay {i}")
        l.copy_(logits_of(T, G, torch.bfloat16, 50 + i))
        ends.copy_(torch.tensor([100 * i, 700 - 20 * i], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_offsets_beyond_32_bits():
    """Rows whose logits start past 2^32 elements."""
    G = 288
    T = (1 << 32) // G + 200
    say(f"route {T} rows")
    l = torch.zeros((T, G), dtype=torch.bfloat16, device=DEV)
    tail = logits_of(100, G, torch.bfloat16, 60)
    l[-100:] = tail.to(DEV)
    ids, w = mgg.route_topk(l, 4, balance=False)
    torch.cuda.synchronize()
    r = ref.route(tail.double().numpy(), 4)
    assert (ids[-100:].cpu().numpy() == r["ids"]).all()
    np.testing.assert_allclose(w[-100:].cpu().numpy(), r["weights"], rtol=200 * U)
    dw = torch.zeros((T, 4), device=DEV)
    dw[-100:, 0] = 1.0
    d = mgg.route_topk_backward(l, ids, d_weights=dw)
    torch.cuda.synchronize()
    dwn = dw[-100:].double().cpu().numpy()
    want, mag = ref.route_grad(tail.double().numpy(), r["ids"], None, None, dwn)
    off = np.abs(d[-100:].double().cpu().numpy() - want)
    assert (off <= 256 * U * mag + 2.0 ** -8 * np.abs(want)).all()
    assert not d[:-100].any()


def test_two_streams():
    """Calls on two streams at once give the same bits as one after the other."""
    say("route streams")
    ls = [logits_of(5000, 288, torch.float32, 70).to(DEV), logits_of(3000, 40, torch.bfloat16, 71).to(DEV)]
    want = [mgg.route_topk(l, 8) for l in ls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(mgg.route_topk(ls[i], 8))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i in range(2) for o in got[i] for a, b in zip(o, want[i]))


@pytest.mark.parametrize("G", [16, 60, 64, 100, 128, 160, 192, 250, 256, 272, 288, 300, 320])
def test_crowded_candidates(G):
    """Rows whose candidates do not fit the ranking (few distinct values) next to rows whose
    candidates do: each row's result is the definition's, and the same beside other rows."""
    say(f"route crowded {G}")
    l = logits_of(64, G, torch.float32, 80 + G)
    l[::3] = torch.round(l[::3])
    l[1::3] = torch.where(l[1::3] > 0, 1.0, l[1::3])
    for k in (1, min(G, 8), min(G, 17), min(G, 32)):
        ids, w = check_forward(l, k)[:2]
        for t in (0, 1, 2, 31, 63):
            i1, w1 = mgg.route_topk(l[t:t + 1].to(DEV), k, balance=False)
            assert torch.equal(i1[0], ids[t]) and torch.equal(w1[0], w[t])
        b = torch.round(4 * torch.randn(G, generator=torch.Generator().manual_seed(G))) / 8
        check_forward(l, k, bias=b, score="sigmoid")


def test_bias_of_any_size():
    """Biases from forbidding to forcing an expert, and large ones that swallow the scores."""
    say("route bias sizes")
    l = logits_of(48, 96, torch.float32, 90)
    b = 0.1 * torch.randn(96, generator=torch.Generator().manual_seed(4))
    for value in (float("-inf"), -1e6, 1e6, 3e38):
        b[7], b[50] = value, value
        ids = check_forward(l, 8, bias=b, score="sigmoid")[0]
        assert ((ids[:, :2] == torch.tensor([7, 50], device=DEV, dtype=torch.int32)).all()
                if value > 0 and value != 1e6 else True)
    b[:] = 1e4 + 0.5 * torch.arange(96) % 3
    check_forward(l, 8, bias=b, score="sigmoid")
    b[7] = float("inf")
    ids, w = mgg.route_topk(l.to(DEV), 8, bias=b.to(DEV), score="sigmoid", balance=False)
    assert (ids[:, 0] == 7).all() and torch.isfinite(w).all()
