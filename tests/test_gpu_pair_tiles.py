"""GPU tests of the CTA-pair GEMM on both sides of its tile width: up to one tile
of 128 weight rows per SM pair it takes those, past that tiles of 256.  Odd
sizes, every kind of epilogue, both formats; references and tolerance as for
the other epilogue tests (2^-8 of the value and 1e-3 of the output's rms)."""
import pytest
import torch

from _helpers import nv, require_library
from test_gpu_gemm_epilogue import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


# m, output columns: few and many tiles for any act (a gated one doubles the weight rows)
FEW, MANY = [(129, 130), (300, 1029), (513, 515)], [(1500, 4101), (2600, 2056)]


def pair_tiles(m, nw, width):
    return (m + 255) // 256 * ((nw + width - 1) // width)


@pytest.mark.parametrize("act,bias,res", [("none", False, False), ("none", True, True), ("gelu", True, False),
                                          ("silu", False, True), ("swiglu", True, False), ("geglu", True, True)])
@pytest.mark.parametrize("m,n", FEW + MANY)
def test_tile_widths(m, n, act, bias, res):
    c = Case(m, 264, n, act, bias, res, seed=m + n)
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    assert (pair_tiles(m, c.nw, 128) <= pairs) == ((m, n) in FEW)
    c.gemm()
    c.linear()


@pytest.mark.parametrize("act,res", [("none", False), ("relu", True), ("swiglu", False)])
@pytest.mark.parametrize("m,n", [FEW[1], MANY[0]])
def test_tile_widths_mxfp4(m, n, act, res):
    c = Case(m, 264, n, act, True, res, seed=m + n, mx=True)
    c.gemm()
    c.linear()


def test_widths_agree():
    """Rows of a problem of few tiles have the bits that they have among many."""
    k, n = 1032, 520
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(8192, k, device="cuda", generator=g).bfloat16()
    w = (torch.randn(n, k, device="cuda", generator=g) * 0.05).bfloat16()
    gs, alpha = torch.full((1,), 40.0, device="cuda"), torch.full((1,), 1e-3, device="cuda")
    wq = nv.prepare_weight(w, gs)
    outs = []
    for m in (8192, 300):
        out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        nv.nvfp4_gemm(*nv.quant_act(x[:m], gs), m, *wq, n, n, k, alpha, None, out, n)
        outs.append(out[:300])
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
