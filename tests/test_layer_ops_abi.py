"""The entry points of include/mgg/layer_ops.h: exported as declared, and refusing invalid host
arguments with nothing enqueued, in the C ABI and in the binding (CPU: no call here reaches a
GPU)."""

import ctypes
import os
import re

import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg
from moe_grouped_gemm_nt_amd.layer_ops import MggBlock

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EUNSUPPORTED = 1, 2
# never dereferenced: every call below fails host validation
P, MIS, NUL = 1 << 20, (1 << 20) + 1, None
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return mgg.load_library()


def test_header_and_exports(lib):
    text = open(os.path.join(ROOT, "include", "mgg", "layer_ops.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^(?:mgg_status|size_t)\s+([a-z_]+)\(", text, flags=re.M)
    assert sorted(names) == sorted([
        "route_topk", "route_topk_workspace", "route_topk_backward", "block_residual_norm",
        "block_residual_norm_backward", "block_residual_norm_backward_workspace", "block_norm",
        "block_norm_backward", "grouped_newton_schulz", "grouped_newton_schulz_workspace"])
    for n in names:
        assert hasattr(lib, n), n


def refused(lib, status, code, text):
    assert status == code
    assert re.search(text, lib.mgg_last_error().decode()), lib.mgg_last_error()


def route(lib, dt=1, T=8, G=16, k=4, l=P, ld=16, bias=NUL, score=0, renorm=1, scale=1.0, S=1,
          ends=NUL, ids=P, w=P, counts=P, tokens=P, bal=P, ws=P, size=BIG):
    return lib.route_topk(dt, T, G, k, l, ld, bias, score, renorm, scale, S, ends, ids, w, counts,
                          tokens, bal, ws, size, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(dt=2), EINVAL, "element type"), (dict(score=3), EINVAL, "score"),
    (dict(T=-1), EINVAL, "T must"), (dict(G=0), EINVAL, "G must"),
    (dict(G=4097, ld=4097), EINVAL, "G must"), (dict(k=0), EINVAL, "k must"),
    (dict(k=17), EINVAL, "k must"), (dict(G=64, ld=64, k=33), EINVAL, "k must"),
    (dict(l=NUL), EINVAL, "null"), (dict(ld=15), EINVAL, "stride"), (dict(l=MIS), EINVAL, "align"),
    (dict(scale=float("inf")), EINVAL, "scale"), (dict(S=0, ends=P), EINVAL, "S must"),
    (dict(S=65536, ends=P), EINVAL, "S must"), (dict(S=2), EINVAL, "seq_ends"),
    (dict(ends=MIS), EINVAL, "align"), (dict(bias=P), EUNSUPPORTED, "bias"),
    (dict(ids=NUL), EINVAL, "null"), (dict(w=NUL), EINVAL, "null"), (dict(w=MIS), EINVAL, "align"),
    (dict(counts=NUL), EINVAL, "together"), (dict(bal=NUL), EINVAL, "together"),
    (dict(tokens=MIS), EINVAL, "align"), (dict(ws=NUL), EINVAL, "workspace"),
    (dict(size=16), EINVAL, "workspace"), (dict(ws=P + 128), EINVAL, "256"),
])
def test_route_refuses(lib, kw, code, text):
    refused(lib, route(lib, **kw), code, text)


def route_grad(lib, dt=1, T=8, G=16, k=4, l=P, ld=16, score=0, S=1, ends=NUL, ids=P, counts=P,
               tokens=P, dw=P, db=P, out=P):
    return lib.route_topk_backward(dt, T, G, k, l, ld, score, 1, 1.0, S, ends, ids, counts,
                                   tokens, dw, db, out, None)


@pytest.mark.parametrize("kw,text", [
    (dict(dt=-1), "element type"), (dict(k=40), "k must"), (dict(dw=NUL, db=NUL), "one of"),
    (dict(out=NUL), "null"), (dict(ids=NUL), "null"), (dict(counts=NUL), "counts"),
    (dict(tokens=NUL), "counts"), (dict(out=MIS), "align"), (dict(dw=MIS), "align"),
    (dict(S=3), "seq_ends"),
])
def test_route_backward_refuses(lib, kw, text):
    refused(lib, route_grad(lib, **kw), EINVAL, text)


def block(**kw):
    d = dict(dtype=0, param=1, T=4, H=8, x=P, ldx=8, y=P, ldy=8, gate_kind=1, gate=P, ld_gate=1,
             scale=P, w_after=P, w_before=P, alpha=1.0, beta=1.0, eps=1e-6)
    d.update(kw)
    return ctypes.byref(MggBlock(*(d[n] for n, _ in MggBlock._fields_)))


BLOCK_FAULTS = [
    (dict(dtype=5), "element type"), (dict(param=5), "element type"), (dict(T=-1), "T must"),
    (dict(H=0), "H must"), (dict(H=32769, ldx=32769, ldy=32769), "H must"),
    (dict(eps=0.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(alpha=float("inf")), "alpha"),
    (dict(x=NUL), "null"), (dict(y=NUL), "null"), (dict(gate=NUL), "null"),
    (dict(gate_kind=3), "gate kind"), (dict(ldx=7), "stride"), (dict(ldy=7), "stride"),
    (dict(ld_gate=0), "stride"), (dict(gate_kind=2, ld_gate=7), "stride"),
    (dict(x=MIS), "align"), (dict(scale=P + 2), "align"), (dict(w_before=P + 2), "align"),
]


@pytest.mark.parametrize("kw,text", BLOCK_FAULTS)
def test_block_refuses(lib, kw, text):
    refused(lib, lib.block_residual_norm(block(**kw), P, P, None), EINVAL, text)
    refused(lib, lib.block_residual_norm_backward(block(**kw), P, 32769, P, 32769, P, P, P, P, P,
                                                  P, P, BIG, None), EINVAL, text)


def test_block_output_refusals(lib):
    refused(lib, lib.block_residual_norm(None, P, P, None), EINVAL, "null")
    refused(lib, lib.block_residual_norm(block(), NUL, P, None), EINVAL, "null")
    refused(lib, lib.block_residual_norm(block(), P, NUL, None), EINVAL, "go together")
    refused(lib, lib.block_residual_norm(block(w_before=NUL), P, P, None), EINVAL, "go together")

    def grad(b, dx=P, lddx=8, du=P, lddu=8, dxi=P, dy=P, dg=P, ds=P, da=P, db=P, ws=P, size=BIG):
        return lib.block_residual_norm_backward(b, dx, lddx, du, lddu, dxi, dy, dg, ds, da, db,
                                                ws, size, None)

    for kw, text in [(dict(dxi=NUL), "null"), (dict(dy=NUL), "null"), (dict(lddx=7), "stride"),
                     (dict(lddu=7), "stride"), (dict(du=NUL), "go together"),
                     (dict(dg=NUL), "exactly"), (dict(ds=NUL), "exactly"),
                     (dict(da=NUL), "exactly"), (dict(db=NUL), "exactly"), (dict(ds=MIS), "align"),
                     (dict(ws=NUL), "workspace"), (dict(size=8), "workspace"),
                     (dict(ws=P + 4), "256")]:
        refused(lib, grad(block(), **kw), EINVAL, text)
    refused(lib, grad(block(w_before=NUL), dx=NUL, du=NUL, db=NUL), EINVAL, "null")


def test_block_norm_refuses(lib):
    def fwd(dt=0, pd=1, T=4, H=8, x=P, ldx=8, w=P, eps=1e-6, u=P):
        return lib.block_norm(dt, pd, T, H, x, ldx, w, eps, u, None)

    def bwd(x=P, ldx=8, w=P, eps=1e-6, dx=P, lddx=8, du=P, lddu=8, out=P, dw=P, ws=P, size=BIG):
        return lib.block_norm_backward(0, 1, 4, 8, x, ldx, w, eps, dx, lddx, du, lddu, out, dw,
                                       ws, size, None)

    for kw, text in [(dict(dt=3), "element"), (dict(H=0), "H must"), (dict(x=NUL), "null"),
                     (dict(w=NUL), "null"), (dict(u=NUL), "null"), (dict(eps=-1.0), "eps"),
                     (dict(ldx=4), "stride"), (dict(u=MIS), "align")]:
        refused(lib, fwd(**kw), EINVAL, text)
    for kw, text in [(dict(du=NUL), "null"), (dict(out=NUL), "null"), (dict(dw=NUL), "null"),
                     (dict(lddx=1), "stride"), (dict(lddu=1), "stride"), (dict(dw=MIS), "align"),
                     (dict(ws=NUL), "workspace"), (dict(size=0), "workspace")]:
        refused(lib, bwd(**kw), EINVAL, text)


def ns(lib, dt=1, od=1, G=2, M=8, N=8, X=P, out=P, steps=1, co=(1.5, -0.5, 0.0), eps=1e-7,
       scale=1.0, ws=P, size=BIG):
    flat = None if co is None else (ctypes.c_float * len(co))(*co)
    return lib.grouped_newton_schulz(dt, od, G, M, N, X, out, steps, flat, eps, scale, ws, size,
                                     None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(dt=4), EINVAL, "element"), (dict(od=4), EINVAL, "element"), (dict(G=0), EINVAL, "G must"),
    (dict(G=4097), EINVAL, "G must"), (dict(M=0), EINVAL, "M and N"),
    (dict(N=32769), EINVAL, "M and N"), (dict(steps=0), EINVAL, "steps"),
    (dict(steps=33), EINVAL, "steps"), (dict(X=NUL), EINVAL, "null"),
    (dict(out=NUL), EINVAL, "null"), (dict(co=None), EINVAL, "null"), (dict(X=MIS), EINVAL, "align"),
    (dict(eps=0.0), EINVAL, "eps"), (dict(scale=float("nan")), EINVAL, "eps"),
    (dict(co=(5.0, 0.0, 0.0)), EUNSUPPORTED, "range"),
    (dict(co=(float("nan"), 0.0, 0.0)), EUNSUPPORTED, "range"),
    (dict(steps=2, co=(3.0, 0.0, 0.0, 2.0, 0.0, 0.0)), EUNSUPPORTED, "range"),
    (dict(co=(0.0, 100.0, -100.0)), EUNSUPPORTED, "range"),
    (dict(ws=NUL), EINVAL, "workspace"), (dict(size=100), EINVAL, "workspace"),
    (dict(ws=P + 16), EINVAL, "256"),
])
def test_newton_schulz_refuses(lib, kw, code, text):
    refused(lib, ns(lib, **kw), code, text)


def test_usual_coefficients_are_in_range(lib):
    # the checks that follow the coefficients are reached: the refusal is the workspace's
    refused(lib, ns(lib, steps=5, co=(3.4445, -4.775, 2.0315) * 5, size=1), EINVAL, "workspace")
    refused(lib, ns(lib, steps=32, co=(1.5, -0.5, 0.0) * 32, size=1), EINVAL, "workspace")


def test_workspace_sizes(lib):
    assert lib.route_topk_workspace(0, 1, 1) > 0 and lib.route_topk_workspace(8, 0, 1) == 0
    assert lib.route_topk_workspace(8, 4097, 1) == 0 and lib.route_topk_workspace(-1, 4, 1) == 0
    assert lib.block_residual_norm_backward_workspace(0, 8) > 0
    assert lib.block_residual_norm_backward_workspace(4, 0) == 0
    assert lib.grouped_newton_schulz_workspace(1, 1, 1) > 0
    assert lib.grouped_newton_schulz_workspace(1, 0, 1) == 0


# ------------------------------------------------------------------------- the binding

def expect(pattern, fn, *a, exc=ValueError, **kw):
    with pytest.raises(exc) as ei:
        fn(*a, **kw)
    assert re.search(pattern, str(ei.value)), str(ei.value)


def test_binding_route():
    l = torch.zeros(8, 16)
    ids = torch.zeros(8, 4, dtype=torch.int32)
    expect("same GPU", mgg.route_topk, l, 4)  # well formed: stops at the device check
    expect("same GPU", mgg.route_topk, l[:, 1:9], 4)
    expect("T, G", mgg.route_topk, l[0], 4)
    expect("bfloat16 or float32", mgg.route_topk, l.double(), 4, exc=TypeError)
    expect("topk", mgg.route_topk, l, 17)
    expect("topk", mgg.route_topk, l, 0)
    expect("contiguous rows", mgg.route_topk, l.t(), 4)
    expect("overlap", mgg.route_topk, torch.zeros(1, 16).expand(8, 16), 4)
    expect("score", mgg.route_topk, l, 4, score="tanh")
    expect("sigmoid", mgg.route_topk, l, 4, bias=torch.zeros(16))
    expect("bias", mgg.route_topk, l, 4, score="sigmoid", bias=torch.zeros(15))
    expect("int32", mgg.route_topk, l, 4, seq_ends=torch.tensor([8]))
    b = mgg.route_topk_backward
    expect("same GPU", b, l, ids, d_weights=torch.zeros(8, 4))
    expect("one of", b, l, ids)
    expect("ids", b, l, ids.long(), d_weights=torch.zeros(8, 4))
    expect("d_weights", b, l, ids, d_weights=torch.zeros(8, 3))
    expect("counts and tokens", b, l, ids, d_balance=torch.zeros(1))
    expect("counts", b, l, ids, torch.zeros(2, 16, dtype=torch.int32),
           torch.zeros(1, dtype=torch.int32), d_balance=torch.zeros(1))
    expect("d_balance", b, l, ids, d_balance=torch.zeros(2))


def test_binding_block():
    x, w = torch.zeros(4, 8), torch.ones(8)
    f, b = mgg.block_residual_norm, mgg.block_residual_norm_backward
    expect("same GPU", f, x, x, w_before=w)
    expect("y must be", f, x, x[:3])
    expect("y must be", f, x, x.bfloat16())
    expect("gate must be", f, x, x, gate=torch.zeros(5))
    expect("gate must be", f, x, x, gate=torch.zeros(4, 7))
    expect("must be \\[8\\]", f, x, x, scale=torch.ones(7))
    expect("one element type", f, x, x, scale=w, w_after=w.bfloat16())
    expect("go together", f, x.cpu(), x, u=x) if torch.cuda.is_available() else None
    expect("go together", b, x, x, d_x=x, d_u=x)
    expect("one of", b, x, x)
    expect("d_x must be", b, x, x, d_x=x[:2])
    expect("same GPU", b, x, x, d_x=x)
    expect("same GPU", mgg.block_norm, x, w)
    expect("must be \\[8\\]", mgg.block_norm, x, w[:4])
    expect("d_u must be", mgg.block_norm_backward, x, w, x[:1])


def test_binding_newton_schulz():
    X = torch.zeros(2, 4, 6)
    f = mgg.grouped_newton_schulz
    expect("same GPU", f, X)
    expect("G, M, N", f, X[0])
    expect("steps", f, X, steps=0)
    expect("coeffs", f, X, coeffs=[(1.0, 0.0, 0.0)] * 4)
    expect("coeffs", f, X, coeffs=(1.0, 2.0))
    expect("bfloat16 or float32", f, X.half(), exc=TypeError)
