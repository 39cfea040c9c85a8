"""moe_few_tokens refuses invalid host arguments with nothing enqueued, in the C ABI and in the
binding (CPU: no call here reaches a GPU)."""

import os
import re

import pytest
import torch

import moe_grouped_gemm_nt_amd as mgg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EUNSUPPORTED = 1, 2
P, MIS, NUL = 1 << 20, (1 << 20) + 1, None  # never dereferenced
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    return mgg.load_library()


def test_header_and_exports(lib):
    text = open(os.path.join(ROOT, "include", "mgg", "few_tokens.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^(?:mgg_status|size_t)\s+([a-z_]+)\(", text, flags=re.M)
    assert sorted(names) == ["moe_few_tokens", "moe_few_tokens_workspace"]
    for n in names:
        assert hasattr(lib, n)


def call(lib, wt=1, T=4, k=2, G=8, H=256, I=128, x=P, ldx=256, ids=P, w=P, w13=P, s13=P, w2=P,
         s2=P, sf=0, gran=0, out_dt=0, res=NUL, ld_res=0, out=P, ws=P, size=BIG):
    return lib.moe_few_tokens(wt, T, k, G, H, I, x, ldx, ids, w, w13, s13, w2, s2, sf, gran,
                              out_dt, res, ld_res, out, ws, size, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(wt=3), EINVAL, "weight type"), (dict(wt=-1), EINVAL, "weight type"),
    (dict(out_dt=2), EINVAL, "element type"), (dict(T=-1), EINVAL, "T must"),
    (dict(T=129), EINVAL, "T must"), (dict(k=0), EINVAL, "k must"), (dict(k=33), EINVAL, "k must"),
    (dict(G=0), EINVAL, "G must"), (dict(G=4097), EINVAL, "G must"),
    (dict(H=0), EINVAL, "H and I"), (dict(H=192), EINVAL, "H and I"),
    (dict(I=64), EINVAL, "H and I"), (dict(I=(1 << 16) + 128), EINVAL, "H and I"),
    (dict(wt=0, s13=NUL, s2=NUL, H=252), EINVAL, "H and I"),
    (dict(sf=2), EINVAL, "scale format"), (dict(gran=2), EUNSUPPORTED, "FP8 weights"),
    (dict(wt=2, gran=2), EUNSUPPORTED, "FP4 weights"),
    (dict(wt=2, sf=1, gran=0), EUNSUPPORTED, "FP4 weights"),
    (dict(s13=NUL), EINVAL, "scales go with"), (dict(s2=NUL), EINVAL, "scales go with"),
    (dict(wt=0), EINVAL, "scales go with"), (dict(w13=NUL), EINVAL, "null"),
    (dict(w2=NUL), EINVAL, "null"), (dict(w13=P + 8), EINVAL, "16-byte"),
    (dict(w2=P + 8), EINVAL, "16-byte"), (dict(s2=P + 2), EINVAL, "4-byte"),
    (dict(x=NUL), EINVAL, "null"), (dict(ids=NUL), EINVAL, "null"), (dict(w=NUL), EINVAL, "null"),
    (dict(out=NUL), EINVAL, "null"), (dict(ldx=255), EINVAL, "stride"),
    (dict(res=P, ld_res=255), EINVAL, "stride"), (dict(x=MIS), EINVAL, "align"),
    (dict(ids=MIS), EINVAL, "align"), (dict(w=P + 2), EINVAL, "align"),
    (dict(out=MIS), EINVAL, "align"), (dict(out_dt=1, out=P + 2), EINVAL, "align"),
    (dict(ws=NUL), EINVAL, "workspace"), (dict(size=100), EINVAL, "workspace"),
    (dict(ws=P + 128), EINVAL, "256"),
])
def test_refuses(lib, kw, code, text):
    assert call(lib, **kw) == code
    assert re.search(text, lib.mgg_last_error().decode()), lib.mgg_last_error()


def test_no_tokens_need_nothing(lib):
    assert call(lib, T=0, x=NUL, ids=NUL, w=NUL, out=NUL, ws=NUL, size=0) == 0


def test_workspace_size(lib):
    size = lib.moe_few_tokens_workspace
    assert size(4, 2, 8, 128) >= 4 * 2 * 128 * 4
    assert size(129, 2, 8, 128) == size(4, 33, 8, 128) == size(4, 2, 0, 128) == size(4, 2, 8, 0) == 0


def expect(pattern, exc=ValueError, **kw):
    a = dict(x=torch.zeros(4, 256, dtype=torch.bfloat16), ids=torch.zeros(4, 2, dtype=torch.int32),
             weights=torch.zeros(4, 2), w13=torch.zeros(8, 256, 256, dtype=torch.uint8),
             w2=torch.zeros(8, 256, 128, dtype=torch.uint8), s13=torch.zeros(8, 2, 2),
             s2=torch.zeros(8, 2, 1))
    a.update(kw)
    with pytest.raises(exc) as ei:
        mgg.moe_few_tokens(**a)
    assert re.search(pattern, str(ei.value)), str(ei.value)


def test_binding_refuses():
    z, u8, bf = torch.zeros, torch.uint8, torch.bfloat16
    expect("same GPU")  # well formed: stops at the device check
    expect("same GPU", s13=z(8, 2, 256), s2=z(8, 1, 256), sfb_gran="channel")
    expect("same GPU", w13=z(8, 256, 128, dtype=u8), w2=z(8, 256, 64, dtype=u8),
           s13=z(8, 2, 256, 4, dtype=u8), s2=z(8, 1, 256, 4, dtype=u8))
    expect("same GPU", w13=z(8, 256, 256, dtype=bf), w2=z(8, 256, 128, dtype=bf), s13=None, s2=None)
    expect("x must be", x=z(256, dtype=bf))
    expect("bfloat16", exc=TypeError, x=z(4, 256))
    expect("contiguous rows", x=z(256, 4, dtype=bf).t())
    expect("ids must be", ids=z(4, 2, dtype=torch.int64))
    expect("ids must be", ids=z(3, 2, dtype=torch.int32))
    expect("weights must be", weights=z(4, 3))
    expect("up rows", w13=z(8, 255, 256, dtype=u8))
    expect("w13 must be", w13=z(8, 256, 256), exc=TypeError)
    expect("one element type", w2=z(8, 256, 128, dtype=bf))
    expect("one element type", w2=z(7, 256, 128, dtype=u8))
    expect("one element type", w2=z(8, 128, 128, dtype=u8))
    expect("need s13", s13=None)
    expect("need s2", s2=None)
    expect("s13 .* must be", s13=z(8, 2, 1))
    expect("s2 .* must be", s2=z(8, 2, 1, dtype=u8))
    expect("s13 .* must be", s13=z(8, 2, 2).double())
    expect("does not fit", sfb_gran="block32")
    expect("no scales", w13=z(8, 256, 256, dtype=bf), w2=z(8, 256, 128, dtype=bf))


@pytest.mark.parametrize("gran", ["block64", "block32"])
def test_bf16_weights_refuse_an_unfit_granularity(gran):
    bf = torch.bfloat16
    expect("does not fit", w13=torch.zeros(8, 256, 256, dtype=bf), s13=None, s2=None,
           w2=torch.zeros(8, 256, 128, dtype=bf), sfb_gran=gran)
