"""Host-side checks of the entry points around the linear layer (no GPU needed):
size queries, and refusals with the documented status before any device access.
Fake addresses are only used in calls that must fail validation or are empty."""
import pytest

import nvfp4_quantized_linear_gb300 as nv

OK, INVALID, UNSUPPORTED, ALIGN, ALIAS, CUDA, TIMEOUT, WORKSPACE = range(8)
A, B, C, D, E, F, G, H = (1 << s for s in (20, 30, 34, 36, 38, 39, 40, 41))


@pytest.fixture(scope="module")
def lib():
    nv.build()
    return nv.load_library()


def call(f, defaults):
    return lambda **kw: f(*{**defaults, **kw}.values())


def test_sizes(lib):
    assert nv.nvfp4_mxfp8_bytes(3, 40) == 3 * 64 and nv.nvfp4_mxfp8_bytes(0, 40) == 0
    assert nv.nvfp4_moe_rows(0, 8, 64) == 0
    assert nv.nvfp4_moe_rows(1, 8, 64) == 8 * 128            # eight groups of one row
    assert nv.nvfp4_moe_rows(1000, 1, 1) == 1024
    assert nv.nvfp4_moe_rows(4096, 2, 8) == (8192 + 8 * 127) // 128 * 128
    assert nv.nvfp4_moe_sort_workspace_bytes(1025, 1, 16) >= 2 * 16 * 4
    assert nv.nvfp4_moe_sort_workspace_bytes(0, 1, 16) >= 16


def test_norm_refusals(lib):
    f = call(lib.nvfp4_add_rmsnorm_quant, dict(x=A, ldx=256, r=B, ldr=256, gamma=C, eps=1e-6, m=16, k=256, fmt=0, gs=D,
                                               h=E, ldh=256, q=F, sf=G, stream=None))
    assert f(m=0) == OK
    assert f(fmt=3) == INVALID and f(fmt=-1) == INVALID
    assert f(m=-1) == INVALID and f(k=0) == INVALID and f(k=65537) == INVALID
    assert f(eps=-1.0) == INVALID and f(eps=float("nan")) == INVALID
    assert f(r=None) == INVALID                              # h without a residual
    for name in ("x", "gamma", "gs", "q", "sf"):
        assert f(**{name: None}) == INVALID, name
    assert f(ldx=100) == INVALID and f(ldr=255) == INVALID and f(ldh=8) == INVALID
    assert f(x=A + 2) == ALIGN and f(r=B + 8) == ALIGN and f(h=E + 4) == ALIGN and f(gamma=C + 2) == ALIGN
    assert f(q=F + 8) == ALIGN and f(sf=G + 8) == ALIGN and f(gs=D + 2) == ALIGN and f(ldx=260) == ALIGN
    assert f(q=A + 512) == ALIAS and f(sf=F) == ALIAS and f(q=C) == ALIAS and f(h=F) == ALIAS
    assert f(h=A + 512) == ALIAS and f(h=B, ldh=512) == ALIAS   # only x or residual as they are
    assert f(h=C) == ALIAS


def test_epilogue_refusals(lib):
    f = call(lib.nvfp4_gemm_act, dict(a=A, a_sf=B, m=16, w=C, w_sf=D, n_w=256, n_out=128, k=256, alpha=B + (1 << 20),
                                      bias=None, act=4, res=F, ldr=128, out=E, ldo=128, stream=None))
    assert f(m=0) == OK
    assert f(act=6) == INVALID and f(act=-1) == INVALID
    assert f(n_out=129, ldo=136, ldr=136) == INVALID         # gated: two weight rows per column
    assert f(ldr=120) == INVALID and f(ldr=132) == ALIGN and f(res=F + 2) == ALIGN
    assert f(res=E) == ALIAS and f(res=E + 64) == ALIAS
    assert f(bias=E - 256) == ALIAS                          # 256 bias entries reach the output
    g = call(lib.nvfp4_linear_act, dict(x=A, m=16, k=256, ldx=256, gs=B, t=None, bs=0, w=C, w_sf=D, n_w=256, n_out=128,
                                        alpha=B + 64, bias=None, act=5, res=F, ldr=128, out=E, ldo=128, ws=G,
                                        ws_bytes=1 << 20, stream=None))
    assert g(m=0) == OK
    assert g(act=9) == INVALID and g(n_out=200) == INVALID and g(res=G + 256) == ALIAS and g(ldr=64) == INVALID
    assert g(ws=None) == WORKSPACE and g(ws_bytes=10) == WORKSPACE
    h = call(lib.nvfp4_mxfp4_gemm_act, dict(a=A, a_sf=B, m=16, w=C, w_sf=D, n_w=256, n_out=128, k=256, bias=None, act=4,
                                            res=F, ldr=128, out=E, ldo=128, stream=None))
    assert h(m=0) == OK and h(act=7) == INVALID and h(n_out=130, ldo=136, ldr=136) == INVALID and h(res=E) == ALIAS
    i = call(lib.nvfp4_mxfp4_linear_act, dict(x=A, m=16, k=256, ldx=256, w=C, w_sf=D, n_w=256, n_out=128, bias=None,
                                              act=5, res=F, ldr=128, out=E, ldo=128, ws=G, ws_bytes=1 << 20, stream=None))
    assert i(m=0) == OK and i(act=7) == INVALID and i(res=E + 16) == ALIAS and i(ws=None) == WORKSPACE
    j = call(lib.nvfp4_grouped_gemm_act, dict(a=A, a_sf=B, rows=256, off=F, groups=2, w=C, w_sf=D, n=64, k=256,
                                              alpha=G, bias=None, act=4, out=E, ldo=64, stream=None))
    assert j(rows=0) == OK
    assert j(n=32) == INVALID                                # 64 weight rows a group
    assert j(act=0) == INVALID                               # not gated: n = 64 itself
    assert j(n=0) == INVALID and j(act=8) == INVALID and j(groups=0) == INVALID


def test_sort_refusals(lib):
    f = call(lib.nvfp4_moe_sort, dict(ids=A, id_bytes=4, tokens=16, topk=2, experts=8, off=B, cnt=C, dest=D, ws=E,
                                      ws_bytes=1 << 20, stream=None))
    assert f(id_bytes=2) == INVALID and f(topk=0) == INVALID and f(topk=65) == INVALID
    assert f(experts=0) == INVALID and f(experts=1025) == INVALID and f(tokens=-1) == INVALID
    assert f(tokens=1 << 40) == INVALID
    for name in ("ids", "off", "cnt", "dest"):
        assert f(**{name: None}) == INVALID, name
    assert f(ids=A + 2) == ALIGN and f(ids=A + 4, id_bytes=8) == ALIGN and f(dest=D + 1) == ALIGN and f(ws=E + 4) == ALIGN
    assert f(ws=None) == WORKSPACE and f(ws_bytes=8) == WORKSPACE
    assert f(dest=A) == ALIAS and f(cnt=B + 4) == ALIAS and f(ws=D) == ALIAS


def test_rows_refusals(lib):
    rows = nv.nvfp4_moe_rows(16, 2, 8)
    f = call(lib.nvfp4_moe_dispatch, dict(x=A, ldx=64, dest=B, tokens=16, topk=2, rows=rows, h=64, off=C, cnt=D,
                                          experts=8, out=E, ldo=64, stream=None))
    assert f(tokens=0) == OK
    assert f(rows=rows - 1) == INVALID and f(h=0) == INVALID and f(ldx=32) == INVALID and f(x=None) == INVALID
    assert f(off=None) == INVALID and f(out=E + 8) == ALIGN and f(ldo=68) == ALIGN and f(out=A) == ALIAS
    g = call(lib.nvfp4_moe_dispatch_quant, dict(x=A, ldx=64, gs=B, dest=C, tokens=16, topk=2, rows=rows, h=64, q=D, sf=E,
                                                stream=None))
    assert g(tokens=0) == OK
    assert g(gs=None) == INVALID and g(rows=0) == INVALID and g(q=D + 4) == ALIGN and g(sf=D) == ALIAS and g(q=A) == ALIAS
    h = call(lib.nvfp4_moe_combine, dict(y=A, ldy=64, w=B, dest=C, tokens=16, topk=2, rows=rows, h=64, res=D, ldr=64,
                                         out=E, ldo=64, stream=None))
    assert h(tokens=0) == OK
    assert h(y=None) == INVALID and h(dest=None) == INVALID and h(ldr=8) == INVALID and h(rows=-1) == INVALID
    assert h(w=B + 2) == ALIGN and h(out=A + 64) == ALIAS and h(out=D) == ALIAS
    i = call(lib.nvfp4_moe_combine_backward, dict(g=A, ldg=64, y=B, ldy=64, w=C, dest=D, tokens=16, topk=2, rows=rows,
                                                  h=64, off=E, cnt=F, experts=8, dy=G, lddy=64, dw=H, stream=None))
    assert i(tokens=0) == OK
    assert i(w=None) == INVALID and i(dw=None) == INVALID and i(rows=rows - 128) == INVALID
    assert i(dw=H + 2) == ALIGN and i(dy=B) == ALIAS and i(dw=G) == ALIAS


def test_helpers_check_their_tensors():
    import torch
    with pytest.raises(ValueError):
        nv.moe_sort(torch.zeros((4, 2), dtype=torch.int16), 4)
    with pytest.raises(ValueError):
        nv.moe_sort(torch.zeros((4, 4), dtype=torch.int32)[:, ::2], 4)
    with pytest.raises(ValueError):
        nv.add_rmsnorm_quant(torch.zeros((4, 8), dtype=torch.bfloat16).T, torch.ones(4, dtype=torch.bfloat16), 1e-6,
                             fmt=nv.NVFP4_FORMAT_MXFP8)
