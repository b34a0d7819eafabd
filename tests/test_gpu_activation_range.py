"""GPU tests of the epilogue's activations over the whole range of fp32 arguments: SILU
and GELU of a large v are v itself, of a large -v they are 0 (bf16 holds both), also where
v^2 or v^3 overflows fp32, and the gated forms multiply that with their up column.

The operands are exact: one element of 6 per row under a block scale of 448, so that
acc = +-2688^2 or 0 and alpha = V / 2688^2 makes v = +-V or 0 to two roundings of fp32.
Bound: those (2^-23), the factor 1 / (1 + 0) (2^-22) and the rounding to bf16 (2^-8 at most,
2^-9 with the rest to spare): 1.01 * 2^-8 of V."""
import pytest
import torch

from _helpers import dev_scalar, nv, require_library

pytestmark = pytest.mark.gpu
ACC = 2688.0 ** 2
UP = 0.5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def run(path, m, k, act, alpha):
    """Output [m, 128]; column j has v = +, -, 0 times alpha * ACC for j % 3 = 0, 1, 2."""
    n = 128
    gated = act in ("swiglu", "geglu")
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 6.0
    w = torch.zeros((n, k), dtype=torch.bfloat16, device="cuda")
    w[0::3, 0], w[1::3, 0] = 6.0, -6.0
    bias = None
    if gated:                                               # up rows: zero weights, a bias of UP
        w = nv.interleave_gate_up(w, torch.zeros_like(w))
        bias = nv.interleave_gate_up(torch.zeros(n, device="cuda"), torch.full((n,), UP, device="cuda")).bfloat16()
    gs = dev_scalar(448.0)
    wq = nv.prepare_weight(w, gs)
    out = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    al, code = dev_scalar(alpha), nv.ACTIVATIONS[act]
    if path == "linear":
        nv.linear(x, *wq, k, n, gs, al, bias=bias, act=act, out=out)
    else:
        q = nv.quant_act(x, gs)
        if path == "gemm":
            nv.nvfp4_gemm_act(*q, m, *wq, w.shape[0], n, k, al, bias, code, None, 0, out, n)
        else:
            off = torch.tensor([0, m], dtype=torch.int32, device="cuda")
            nv.nvfp4_grouped_gemm_act(*q, m, off, 1, *wq, n, k, al, bias, code, out, n)
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    return out.double()


PATHS = [("linear", 3, 64), ("linear", 3, 2048),            # single launch, whole and with split K
         ("linear", 40, 2048), ("gemm", 40, 64),            # split K behind the quantizer; one CTA
         ("linear", 130, 64), ("grouped", 128, 64)]         # CTA pairs; the wide layout


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu", "geglu"])
@pytest.mark.parametrize("path,m,k", PATHS)
def test_large_finite_arguments(path, m, k, act):
    for v in (1e10, 1.8e19, 1.9e19, 1e20, 1e30, 1e38):
        out = run(path, m, k, act, v / ACC)
        want = v * (UP if act in ("swiglu", "geglu") else 1.0)
        assert ((out[:, 0::3] - want).abs() <= 1.01 * 2.0 ** -8 * want).all(), v
        assert (out[:, 1::3] == 0).all() and (out[:, 2::3] == 0).all(), v


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu", "geglu"])
@pytest.mark.parametrize("path,m,k", PATHS)
def test_positive_infinity(path, m, k, act):
    out = run(path, m, k, act, 3e38)                        # acc * alpha overflows
    assert (out[:, 0::3] == float("inf")).all() and (out[:, 2::3] == 0).all()
