"""Pins of the float64 definitions in oracle/layer_ops.py: torch's own float64 operations and
autograd, finite differences, and closed forms (CPU)."""

import numpy as np
import pytest
import torch

from oracle import layer_ops as ref


def rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("ends", [None, [3, 3, 9], [5, 2, 40], [0, 0, 0], [-4, 7, 8]])
def test_route_against_torch(score, renormalize, ends):
    l = rng(1).normal(size=(11, 13))
    r = ref.route(l, 4, score, renormalize, 2.5, seq_ends=ends)
    t = torch.from_numpy(l)
    q = t.softmax(1) if score == "softmax" else t.sigmoid()
    w, ids = q.topk(4, 1)
    w = 2.5 * (w / w.sum(1, keepdim=True) if renormalize else w)
    live = np.zeros(11, bool)
    for a, e in ref.sequence_ranges(11, ends):
        live[a:e] = True
    assert (r["ids"][live] == ids.numpy()[live]).all() and (r["ids"][~live] == -1).all()
    np.testing.assert_allclose(r["weights"][live], w.numpy()[live], rtol=1e-13)
    assert (r["weights"][~live] == 0).all()
    p = q / q.sum(1, keepdim=True)
    for s, (a, e) in enumerate(ref.sequence_ranges(11, ends)):
        assert r["tokens"][s] == e - a
        c = torch.bincount(ids[a:e].reshape(-1), minlength=13).double()
        assert (r["counts"][s] == c.numpy()).all()
        want = 0.0 if e == a else float((c * 13 / (4 * (e - a)) * p[a:e].mean(0)).sum())
        assert r["balance"][s] == pytest.approx(want, rel=1e-13)


def test_route_balance_is_one_when_even():
    l = np.zeros((8, 8)) - 30.0 * (1 - np.eye(8))
    assert ref.route(l, 1)["balance"][0] == pytest.approx(1.0, rel=1e-12)
    # all tokens on one expert: G times as much
    l[:] = l[0]
    assert ref.route(l, 1)["balance"][0] == pytest.approx(8.0, rel=1e-9)


def test_route_special_rows():
    inf = np.inf
    l = np.array([[1.0, 1.0, 1.0, 0.0], [-inf, -inf, 2.0, -inf], [-inf] * 4,
                  [np.nan, 0.0, 3.0, 1.0], [-3e38] * 4, [-2000.0, -2001.0, -5000.0, -2000.0]])
    for score in ("softmax", "sigmoid"):
        r = ref.route(l, 2, score)
        assert r["ids"][:3].tolist() == [[0, 1], [2, -1], [-1, -1]]
        assert r["ids"][3].tolist() == [2, 3] and r["ids"][4].tolist() == [0, 1]
        assert r["ids"][5].tolist() == [0, 3]
        np.testing.assert_allclose(r["weights"][[0, 4, 5]], 0.5)
        assert r["weights"][1].tolist() == [1.0, 0.0] and not r["weights"][2].any()
        assert not r["p"][2].any()
        np.testing.assert_allclose(r["p"][4], 0.25)
        z = np.exp([0.0, -1.0, -3000.0, 0.0])
        np.testing.assert_allclose(r["p"][5], z / z.sum())


def test_route_bias_selects_only():
    l = np.array([[2.0, 0.0, -1.0]])
    r = ref.route(l, 1, "sigmoid", False, bias=np.array([0.0, 0.0, 5.0]))
    assert r["ids"].tolist() == [[2]]
    assert r["weights"][0, 0] == pytest.approx(1 / (1 + np.e))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_grad_against_differences(score, renormalize):
    r = rng(2)
    l, ends = r.normal(size=(7, 6)), [4, 4, 6]
    f = ref.route(l, 3, score, renormalize, 1.7, seq_ends=ends)
    dw, db = r.normal(size=(7, 3)), r.normal(size=3)

    def loss(v):
        o = ref.route(v, 3, score, renormalize, 1.7, seq_ends=ends)
        assert (o["ids"] == f["ids"]).all()
        return (o["weights"] * dw).sum() + (o["balance"] * db).sum()

    d, mag = ref.route_grad(l, f["ids"], f["counts"], f["tokens"], dw, db, score, renormalize,
                            1.7, ends)
    h = 1e-6
    for t in range(7):
        for e in range(6):
            step = np.zeros_like(l)
            step[t, e] = h
            assert d[t, e] == pytest.approx((loss(l + step) - loss(l - step)) / (2 * h), abs=2e-8)
    assert (mag >= np.abs(d) * (1 - 1e-12)).all()


@pytest.mark.parametrize("gate", [None, "token", "element"])
@pytest.mark.parametrize("after", [True, False])
@pytest.mark.parametrize("before", [True, False])
def test_block_grad_against_torch(gate, after, before):
    g = torch.Generator().manual_seed(3)
    T, H = 5, 7

    def leaf(*shape):
        return torch.randn(shape, generator=g, dtype=torch.float64).requires_grad_()

    x, y, scale = leaf(T, H), leaf(T, H), leaf(H)
    wa, wb = leaf(H) if after else None, leaf(H) if before else None
    gt = None if gate is None else leaf(*((T,) if gate == "token" else (T, H)))
    dx, du = leaf(T, H).detach(), leaf(T, H).detach()

    def rms(v, w):
        return torch.nn.functional.rms_norm(v, (H,), w, 1e-3)

    z = rms(y, wa) if after else y
    if gt is not None:
        z = z * torch.sigmoid(gt if gate == "element" else gt[:, None])
    out = 0.7 * x + 1.3 * scale * z
    u = rms(out, wb) if before else None
    out.retain_grad()
    ((out * dx).sum() + ((u * du).sum() if before else 0)).backward()

    def num(t):
        return None if t is None else t.detach().numpy()

    kw = dict(w_after=num(wa), gate=num(gt), scale=num(scale), w_before=num(wb), alpha=0.7,
              beta=1.3, eps=1e-3)
    f = ref.block_residual_norm(num(x), num(y), **kw)
    np.testing.assert_allclose(f["x_out"], num(out), rtol=1e-12)
    if before:
        np.testing.assert_allclose(f["u"], num(u), rtol=1e-11)
    grads = ref.block_residual_norm_grad(num(out), num(y), num(dx), num(du) if before else None,
                                         **kw)
    leaves = dict(x=x, y=y, scale=scale, w_after=wa, w_before=wb, gate=gt)
    assert set(grads) == {n for n, t in leaves.items() if t is not None}
    for n, (d, mag) in grads.items():
        np.testing.assert_allclose(d, leaves[n].grad.numpy(), rtol=1e-9, atol=1e-12, err_msg=n)
        assert (mag >= np.abs(d) * (1 - 1e-12)).all(), n


def test_block_norm_alone():
    x, w = rng(4).normal(size=(3, 9)), rng(5).normal(size=9)
    u = ref.block_residual_norm(x, w_before=w, eps=1e-4)["u"]
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (9,), torch.from_numpy(w), 1e-4)
    np.testing.assert_allclose(u, want.numpy(), rtol=1e-12)


def test_newton_schulz_works_on_singular_values():
    x = rng(6).normal(size=(2, 5, 8))
    co = [(3.4445, -4.775, 2.0315), (2.0, -1.5, 0.5)]
    got = ref.newton_schulz(x, co, eps=1e-9, scale=2.0)
    for m, o in zip(x, got):
        u, s, vt = np.linalg.svd(m, full_matrices=False)
        s = s / (np.linalg.norm(m) + 1e-9)
        for a, b, c in co:
            s = a * s + b * s ** 3 + c * s ** 5
        np.testing.assert_allclose(o, 2.0 * (u * s) @ vt, atol=1e-12)
    np.testing.assert_allclose(ref.newton_schulz(x.transpose(0, 2, 1), co, 1e-9, 2.0),
                               got.transpose(0, 2, 1), atol=1e-12)
    assert not ref.newton_schulz(np.zeros((1, 3, 2)), co).any()
