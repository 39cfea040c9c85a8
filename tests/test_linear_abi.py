"""linear_act and linear_act_backward refuse invalid host arguments with nothing enqueued, in the
C ABI and in the binding (CPU: no call here reaches a GPU)."""

import ctypes
import os
import re

import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg
from moe_grouped_gemm_nt_amd.linear import MggLinear

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL = 1
P, MIS, NUL = 1 << 20, (1 << 20) + 1, None  # never dereferenced
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    return mgg.load_library()


def test_header_and_exports(lib):
    text = open(os.path.join(ROOT, "include", "mgg", "linear.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^(?:mgg_status|size_t)\s+([a-z_]+)\(", text, flags=re.M)
    assert sorted(names) == ["linear_act", "linear_act_backward", "linear_act_backward_workspace",
                             "linear_act_workspace"]
    for n in names:
        assert hasattr(lib, n)


def linear(**kw):
    d = dict(dtype=0, out_dt=0, bias_dt=1, M=100, N=48, K=40, func=2, x=P, ldx=40, w=P, ldw=40,
             bias=P, residual=P, ld_res=48)
    d.update(kw)
    return ctypes.byref(MggLinear(*(d[n] for n, _ in MggLinear._fields_)))


def refused(lib, status, text):
    assert status == EINVAL
    assert re.search(text, lib.mgg_last_error().decode()), lib.mgg_last_error()


BOTH = [
    (dict(dtype=2), "element type"), (dict(out_dt=-1), "element type"),
    (dict(bias_dt=7), "element type"), (dict(func=5), "function"), (dict(func=-1), "function"),
    (dict(M=-1), "M must"), (dict(M=(1 << 30) + 1), "M must"), (dict(N=0), "N and K"),
    (dict(N=(1 << 20) + 1), "N and K"), (dict(K=0), "N and K"),
    (dict(K=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21), "N and K"),
    (dict(func=4, N=47), "even"), (dict(ldx=39), "stride"), (dict(ldw=39), "stride"),
    (dict(x=MIS), "align"), (dict(w=MIS), "align"),
]


@pytest.mark.parametrize("kw,text", BOTH)
def test_both_refuse(lib, kw, text):
    refused(lib, lib.linear_act(linear(**kw), P, P, P, BIG, None), text)
    refused(lib, lib.linear_act_backward(linear(**kw), P, 1 << 20, P, 1 << 20, P, P, 0, P, P, BIG,
                                         None), text)
    assert lib.linear_act_workspace(linear(**kw)) == 0
    assert lib.linear_act_backward_workspace(linear(**kw), P, 1 << 20, P, 1 << 20, P, P, P) == 0


def test_forward_refuses(lib):
    f = lib.linear_act
    refused(lib, f(None, P, P, P, BIG, None), "null")
    refused(lib, f(linear(), NUL, P, P, BIG, None), "null")
    refused(lib, f(linear(x=NUL), P, P, P, BIG, None), "null")
    refused(lib, f(linear(w=NUL), P, P, P, BIG, None), "null")
    refused(lib, f(linear(ld_res=47), P, P, P, BIG, None), "stride")
    refused(lib, f(linear(func=4, ld_res=23), P, P, P, BIG, None), "stride")
    for kw, out, z in ((dict(), MIS, P), (dict(), P, MIS), (dict(bias=P + 2), P, P),
                       (dict(residual=MIS), P, P), (dict(out_dt=1), P + 2, P)):
        refused(lib, f(linear(**kw), out, z, P, BIG, None), "align")
    # rows of 41 bf16 are not whole aligned pieces: they are packed, above the few rows
    odd = dict(K=41, ldx=41, ldw=41)
    need = lib.linear_act_workspace(linear(**odd))
    assert need >= (100 + 48) * 48 * 2
    refused(lib, f(linear(**odd), P, P, P, need - 1, None), "workspace")
    refused(lib, f(linear(**odd), P, P, NUL, BIG, None), "workspace")
    refused(lib, f(linear(**odd), P, P, P + 128, BIG, None), "256")
    assert lib.linear_act_workspace(linear(M=3, **odd)) == 0
    assert lib.linear_act(linear(M=0, x=NUL), NUL, NUL, NUL, 0, None) == 0


def test_backward_refuses(lib):
    def f(l, z=P, ldz=48, d=P, ldd=48, dx=P, dw=P, dt=0, db=P, ws=P, size=BIG):
        return lib.linear_act_backward(l, z, ldz, d, ldd, dx, dw, dt, db, ws, size, None)

    refused(lib, f(None), "null")
    refused(lib, f(linear(), d=NUL), "null")
    refused(lib, f(linear(x=NUL)), "null")
    refused(lib, f(linear(w=NUL)), "null")
    refused(lib, f(linear(), dx=NUL, dw=NUL, db=NUL), "one of")
    refused(lib, f(linear(), z=NUL), "z goes")
    refused(lib, f(linear(func=0)), "z goes")
    refused(lib, f(linear(), ldz=47), "stride")
    refused(lib, f(linear(), ldd=47), "stride")
    refused(lib, f(linear(func=4), ldd=23), "stride")
    refused(lib, f(linear(), dt=3), "element type")
    for kw in (dict(z=MIS), dict(d=MIS), dict(dx=MIS), dict(dw=MIS), dict(db=P + 2),
               dict(dw=P + 2, dt=1)):
        refused(lib, f(linear(), **kw), "align")
    need = lib.linear_act_backward_workspace(linear(), P, 48, P, 48, P, P, P)
    assert need >= 100 * 48 * 2
    refused(lib, f(linear(), size=need - 1), "workspace")
    refused(lib, f(linear(), ws=NUL), "workspace")
    refused(lib, f(linear(), ws=P + 64), "256")
    # no function, no bias: the gradients read d_out itself
    assert lib.linear_act_backward_workspace(linear(func=0), NUL, 0, P, 48, P, P, NUL) == 0


def expect(pattern, fn, *a, exc=ValueError, **kw):
    with pytest.raises(exc) as ei:
        fn(*a, **kw)
    assert re.search(pattern, str(ei.value)), str(ei.value)


def test_binding_refuses():
    z, f, b = torch.zeros, mgg.linear_act, mgg.linear_act_backward
    x, w, d = z(4, 8), z(6, 8), z(4, 6)
    expect("same GPU", f, x, w)  # well formed: stops at the device check
    expect("same GPU", f, x, w, z(6).bfloat16(), func="gelu", residual=d, keep_z=True)
    expect("same GPU", f, x, w, func="swiglu", residual=z(4, 3))
    expect("same GPU", f, x, w, out_dtype=torch.bfloat16, residual=d.bfloat16())
    expect("M, K", f, x[0], w)
    expect("bfloat16 or float32", f, x.half(), w.half(), exc=TypeError)
    expect("w must be", f, x, w.bfloat16())
    expect("w must be", f, x, z(6, 7))
    expect("contiguous rows", f, z(8, 4).t(), w)
    expect("overlap", f, z(1, 8).expand(4, 8), w)
    expect("func must", f, x, w, func="tanh")
    expect("up rows", f, x, z(5, 8), func="swiglu")
    expect("bias must", f, x, w, z(5))
    expect("bfloat16 or float32", f, x, w, z(6).double(), exc=TypeError)
    expect("residual must", f, x, w, residual=z(4, 5))
    expect("residual must", f, x, w, residual=d.bfloat16())
    expect("output must be", f, x, w, out_dtype=torch.float16, exc=TypeError)
    expect("same GPU", b, x, w, d)
    expect("same GPU", b, x, w, d.bfloat16(), d, func="relu")
    expect("one gradient", b, x, w, d, need_x=False, need_w=False)
    expect("z goes", b, x, w, d, d)
    expect("z goes", b, x, w, d, func="relu")
    expect("z must be", b, x, w, d, d.bfloat16(), func="relu")
    expect("d_out must be", b, x, w, z(4, 5))
    expect("d_out must be", b, x, w, d, d, func="swiglu")
