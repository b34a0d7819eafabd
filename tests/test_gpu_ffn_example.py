"""examples/ffn_block.py: the operators together, as a model uses them.

Each layer is compared with the same chain built from the oracle's formats in 64
bits: every operand the layer quantizes is quantized here too, from the values
of the step before rounded to bf16 as the layer rounds them.  The chain's only
freedom is then a value near a rounding threshold, which moves one FP4 code: a
relative Frobenius error of 5e-3 of the FFN branch (the GEMM tolerance) covers it.
"""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
from _block_ref import activation, e4m3_value, unpack_fp4
from _helpers import FROB_REL, nv, require_library, syn

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import ffn_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def _q(v, gs):
    """Values of the NVFP4 quantization of a bf16 tensor, global scale divided out."""
    p, s = oracle.quantize(syn.bf16_bits(v), float(gs))
    return torch.from_numpy(unpack_fp4(p) * np.repeat(e4m3_value(s), 16, 1) / float(gs)).cuda()[:, :v.shape[1]]


def _bf16(v):
    return v.to(torch.float32).to(torch.bfloat16)


def _swiglu(v):
    return torch.from_numpy(activation(v.cpu().numpy(), "swiglu")).cuda()


def _rnd(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)


def _close(got, ref):
    err = float((got - ref).norm() / ref.norm())
    assert err <= FROB_REL, err


@pytest.mark.parametrize("m", [1, 70, 300])
def test_dense_ffn(m):
    rnd, k, f = _rnd(m), 512, 768
    x, r, gamma = rnd(m, k), rnd(m, k), 1 + rnd(k, std=0.1)
    wg, wu, wd = rnd(f, k, std=0.05), rnd(f, k, std=0.05), rnd(k, f, std=0.05)
    ffn = ffn_block.DenseFFN(gamma, wg, wu, wd)
    ffn.calibrate(x, r)
    out = ffn(x, r)
    nv.nvfp4_device_error()
    # the norm's codes (tested by themselves) stand for its output
    x_q, x_sf, h = nv.add_rmsnorm_quant(x, gamma, ffn_block.EPS, residual=r, gs=ffn.gs1)
    sf = oracle.unswizzle(x_sf.cpu().numpy(), m, k // 16)
    n = torch.from_numpy(unpack_fp4(x_q.cpu().numpy()) * np.repeat(e4m3_value(sf), 16, 1)).cuda() / float(ffn.gs1)
    w1 = _q(nv.interleave_gate_up(wg, wu), ffn.gw1)
    hidden = _bf16(_swiglu(n @ w1.T))
    branch = _q(hidden, ffn.gs2) @ _q(wd, ffn.gw2).T
    ref = branch + h.double()
    _close(out.double(), ref)
    assert torch.equal(h, (x.float() + r.float()).to(torch.bfloat16))


@pytest.mark.parametrize("m,topk", [(1, 2), (9, 4), (500, 3)])
def test_moe_ffn_and_its_buffers_do_not_go_stale(m, topk):
    """Two batches through the same layer back to back, without a wait between the calls:
    the kernels overlap (programmatic dependent launches) and each must see its own batch."""
    rnd, k, f, e = _rnd(m), 256, 192, 8
    moe = ffn_block.MoEFFN(rnd(e, k, std=0.1), rnd(e, f, k, std=0.06), rnd(e, f, k, std=0.06), rnd(e, k, f, std=0.06), topk)
    xs = [rnd(m, k) for _ in range(2)]
    moe.calibrate(torch.cat(xs))
    torch.cuda.synchronize()
    outs = [moe(xs[0]), moe(xs[1]), moe(xs[0])]
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    assert torch.equal(outs[0], outs[2])
    deq = lambda w, sf, rows, cols: torch.from_numpy(  # noqa: E731
        unpack_fp4(w.cpu().numpy()) * np.repeat(e4m3_value(oracle.unswizzle(sf.cpu().numpy(), rows, cols // 16)), 16, 1)).cuda()
    w1 = deq(moe.w1, moe.w1_sf, e * 2 * f, k).view(e, 2 * f, k) / float(moe.gw1)
    w2 = deq(moe.w2, moe.w2_sf, e * k, f).view(e, k, f) / float(moe.gw2)
    for x, out in zip(xs, outs):
        ids, weights = moe.route(x)
        n = _q(x, moe.gs1)
        branch = torch.zeros(m, k, dtype=torch.float64, device="cuda")
        for t in range(m):
            for j in range(topk):
                i = int(ids[t, j])
                hid = _bf16(_swiglu((n[t] @ w1[i].T)[None]))
                y = _bf16((_q(hid, moe.gs2) @ w2[i].T)[0]).double()
                branch[t] += y * float(weights[t, j])
        _close(out.double(), branch + x.double())


def test_example_runs(capsys):
    ffn_block.main()
    out = capsys.readouterr().out
    assert "finite True" in out and float(out.split("rel ")[1].split()[0]) < 0.25
