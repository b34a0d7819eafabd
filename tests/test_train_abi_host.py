"""Host-side checks of routing, the 8-bit checkpoints and the weight gradient (no GPU needed): refusals
with the documented status before any device access, and the tensor-level helpers' own.
Fake addresses are only used in calls that must fail validation or are empty."""
import re

import pytest
import torch

import nvfp4_quantized_linear_gb300 as nv
from test_dependent_loads_host import NON_COHERENT, source

OK, INVALID, UNSUPPORTED, ALIGN, ALIAS, CUDA, TIMEOUT, WORKSPACE = range(8)
A, B, C, D, E, F, G, H = (1 << s for s in (20, 30, 34, 36, 38, 39, 40, 41))
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def lib():
    nv.build()
    return nv.load_library()


def call(f, defaults):
    return lambda **kw: f(*{**defaults, **kw}.values())


def test_route_refusals(lib):
    f = call(lib.nvfp4_moe_route, dict(l=A, type=0, ldl=64, bias=B, tokens=16, experts=64, score=0, topk=8, groups=8, group_top=2,
                                       topk_groups=4, renorm=1, scale=1.0, ids=C, w=D, stream=None))
    assert f(tokens=0) == OK
    assert f(type=2) == INVALID and f(score=2) == INVALID and f(score=-1) == INVALID
    assert f(experts=0) == INVALID and f(experts=1025, ldl=2000) == INVALID
    assert f(topk=0) == INVALID and f(topk=65, experts=128, ldl=128) == INVALID
    assert f(topk=9, experts=8, ldl=8, groups=1, topk_groups=1) == INVALID
    assert f(groups=0) == INVALID and f(groups=5) == INVALID and f(groups=64) == INVALID
    assert f(topk_groups=0) == INVALID and f(topk_groups=9) == INVALID
    assert f(group_top=0) == INVALID and f(group_top=3) == INVALID
    assert f(tokens=-1) == INVALID and f(tokens=1 << 40) == INVALID and f(ldl=63) == INVALID
    assert f(scale=float("nan")) == INVALID and f(scale=float("inf")) == INVALID
    for name in ("l", "ids", "w"):
        assert f(**{name: None}) == INVALID, name
    assert f(l=A + 2) == ALIGN and f(l=A + 1, type=1) == ALIGN and f(bias=B + 1) == ALIGN
    assert f(ids=C + 2) == ALIGN and f(w=D + 2) == ALIGN
    assert f(ids=A + 64) == ALIAS and f(w=C) == ALIAS and f(w=B) == ALIAS


def test_route_backward_refusals(lib):
    f = call(lib.nvfp4_moe_route_backward, dict(dw=A, ids=B, l=C, type=0, ldl=64, tokens=16, experts=64, score=0, topk=8,
                                                renorm=1, scale=1.0, dl=D, ldd=64, stream=None))
    assert f(tokens=0) == OK
    assert f(type=-1) == INVALID and f(score=3) == INVALID and f(topk=65) == INVALID and f(experts=2000) == INVALID
    assert f(ldl=10) == INVALID and f(ldd=63) == INVALID and f(tokens=-2) == INVALID
    for name in ("dw", "ids", "l", "dl"):
        assert f(**{name: None}) == INVALID, name
    assert f(dw=A + 2) == ALIGN and f(ids=B + 3) == ALIGN and f(dl=D + 2) == ALIGN and f(l=C + 2) == ALIGN
    assert f(dl=C) == ALIAS and f(dl=A) == ALIAS and f(dl=B) == ALIAS


def test_checkpoint_refusals(lib):
    f = call(lib.nvfp4_act_checkpoint, dict(x=A, ldx=256, m=16, n=128, act=4, off=B, cnt=C, groups=3, out=D, ldo=128, q=E, sf=F,
                                            stream=None))
    assert f(m=0) == OK
    assert f(act=6) == INVALID and f(act=-1) == INVALID and f(n=0) == INVALID and f(m=-1) == INVALID
    assert f(n=1 << 30) == INVALID and f(m=1 << 31) == INVALID
    for name in ("x", "q", "sf", "off", "cnt"):
        assert f(**{name: None}) == INVALID, name
    assert f(groups=0) == INVALID and f(groups=1025) == INVALID and f(groups=-1) == INVALID
    assert f(ldx=248) == INVALID and f(ldo=120) == INVALID
    assert f(x=A + 2) == ALIGN and f(ldx=260) == ALIGN and f(out=D + 8) == ALIGN and f(q=E + 4) == ALIGN and f(sf=F + 8) == ALIGN
    assert f(off=B + 2) == ALIGN and f(cnt=C + 1) == ALIGN
    assert f(out=A) == ALIAS and f(q=A + 4096) == ALIAS and f(sf=E) == ALIAS and f(q=B) == ALIAS and f(out=E) == ALIAS
    g = call(lib.nvfp4_act_checkpoint_backward, dict(d=A, ldd=128, q=B, sf=C, m=16, n=128, act=4, off=None, cnt=None, groups=0,
                                                     dx=D, ldx=256, aq=E, asf=F, stream=None))
    assert g(m=0) == OK
    assert g(act=7) == INVALID and g(n=0) == INVALID and g(off=G) == INVALID and g(groups=2) == INVALID
    assert g(d=None) == INVALID and g(dx=None) == INVALID and g(aq=None) == INVALID and g(asf=None) == INVALID
    assert g(d=None, dx=None, aq=None, asf=None) == INVALID and g(q=None) == INVALID and g(sf=None) == INVALID
    assert g(ldd=120) == INVALID and g(ldx=128) == INVALID
    assert g(d=A + 4) == ALIGN and g(ldx=260) == ALIGN and g(q=B + 8) == ALIGN and g(aq=E + 2) == ALIGN
    assert g(dx=A) == ALIAS and g(dx=B) == ALIAS and g(aq=B) == ALIAS and g(asf=E) == ALIAS and g(aq=D) == ALIAS


def test_wgrad_refusals(lib):
    f = call(lib.nvfp4_checkpoint_wgrad, dict(dy=A, ldd=64, q=B, sf=C, m=16, n=64, k=96, off=None, cnt=None, groups=0, type=0,
                                              acc=0, dw=D, ldw=96, ws=E, ws_bytes=1 << 30, stream=None))
    assert f(type=2) == INVALID and f(acc=1, type=1) == INVALID
    assert f(m=-1) == INVALID and f(n=0) == INVALID and f(k=0) == INVALID and f(n=1 << 31) == INVALID
    assert f(n=(1 << 31) - 2048, k=(1 << 31) - 2048, ldw=1 << 31) == INVALID
    for name in ("dy", "q", "sf", "dw"):
        assert f(**{name: None}) == INVALID, name
    assert f(groups=2) == INVALID and f(off=F, cnt=G) == INVALID and f(off=F, groups=2) == INVALID
    assert f(ldd=56) == INVALID and f(ldw=88) == INVALID
    assert f(dy=A + 8) == ALIGN and f(ldd=68) == ALIGN and f(q=B + 1) == ALIGN and f(dw=D + 4) == ALIGN
    assert f(ldw=98) == ALIGN and f(type=1, ldw=100) == ALIGN and f(ws=E + 8) == ALIGN
    assert f(ws=None) == WORKSPACE and f(ws_bytes=1) == WORKSPACE
    assert f(dw=A) == ALIAS and f(dw=B) == ALIAS and f(dw=E) == ALIAS and f(ws=C) == ALIAS
    assert nv.nvfp4_checkpoint_wgrad_workspace_bytes(0, 5, 5) >= 16


def test_the_kernels_have_no_non_coherent_load():
    """They are launched as programmatic dependents."""
    for name in ("route.cu", "checkpoint.cu", "wgrad.cu"):
        text = source(name)
        assert NON_COHERENT.findall(re.sub("load16_coherent", "", text)) == [], name


def refused(match, f, *args, **kw):
    with pytest.raises(ValueError, match=match):
        f(*args, **kw)


def zeros(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def test_helpers_check_their_tensors():
    """CPU tensors, right in all but the named one; where all are right the refusal is the device's."""
    l = zeros(6, 32, dtype=F32)
    refused("^logits must be a CUDA", nv.moe_route, l, 4)
    refused("^logits must be float32", nv.moe_route, l.double(), 4)
    refused("^logits must be a 2-D", nv.moe_route, l.T, 4)
    refused("^unknown score", nv.moe_route, l, 4, "tanh")
    refused("^bias", nv.moe_route, l, 4, bias=zeros(31, dtype=F32))
    refused("^bias", nv.moe_route, l, 4, bias=zeros(32))
    ids, dw = zeros(6, 4, dtype=I32), zeros(6, 4, dtype=F32)
    refused("^logits must be a CUDA", nv.moe_route_backward, dw, ids, l)
    refused("^expert_ids", nv.moe_route_backward, dw, ids.long(), l)
    refused("^expert_ids", nv.moe_route_backward, dw, ids[:5], l)
    refused("^expert_ids", nv.moe_route_backward, dw, ids[0], l)
    refused("^dweights", nv.moe_route_backward, dw[:, :3].contiguous(), ids, l)
    refused("^dweights", nv.moe_route_backward, dw.double(), ids, l)
    x, off, cnt = zeros(256, 64), zeros(3, dtype=I32), zeros(2, dtype=I32)
    refused("^x must be a CUDA", nv.act_checkpoint, x, "swiglu", off, cnt)
    refused("^x must be bfloat16", nv.act_checkpoint, x.float())
    refused("^unknown activation", nv.act_checkpoint, x, "tanh")
    refused("^swiglu needs", nv.act_checkpoint, zeros(4, 63), "swiglu")
    refused("^group_offsets and", nv.act_checkpoint, x, "relu", off)
    refused("^group_offsets must", nv.act_checkpoint, x, "relu", off[:2], cnt)
    refused("^group_counts", nv.act_checkpoint, x, "relu", off, cnt.long())
    refused("^out", nv.act_checkpoint, x, "swiglu", out=zeros(256, 31))
    q, sf = zeros(256, 64, dtype=U8), zeros(256 * 4, dtype=U8)
    d = zeros(256, 32)
    refused("^dout must be a CUDA", nv.act_checkpoint_backward, d, q, sf, "swiglu")
    refused("^q must", nv.act_checkpoint_backward, d, q[:255], sf, "swiglu")
    refused("^q must", nv.act_checkpoint_backward, d, q.float(), sf, "swiglu")
    refused("^sf must", nv.act_checkpoint_backward, d, q, sf[:-1], "swiglu")
    refused("^dx", nv.act_checkpoint_backward, d, q, sf, "swiglu", dx=zeros(256, 63))
    refused("^dy must be a CUDA", nv.checkpoint_wgrad, d, q, sf, 64)
    refused("^dy must be bfloat16", nv.checkpoint_wgrad, d.float(), q, sf, 64)
    refused("^q must", nv.checkpoint_wgrad, d, q, sf, 65)
    refused("^dw must hold", nv.checkpoint_wgrad, d, q, sf, 64, dw=zeros(31, 64))
    refused("^dw must be float32", nv.checkpoint_wgrad, d, q, sf, 64, dw=zeros(32, 64, dtype=torch.float16))
    refused("^accumulate", nv.checkpoint_wgrad, d, q, sf, 64, accumulate=True)
    refused("^dtype", nv.checkpoint_wgrad, d, q, sf, 64, dtype=torch.float16)
    refused("^workspace", nv.checkpoint_wgrad, d, q, sf, 64, workspace=zeros(16))
