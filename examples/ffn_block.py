"""A transformer block's FFN on the FP4 linear, dense and mixture-of-experts.

    python examples/ffn_block.py

Each class holds weights prepared once and runs its forward pass without an
elementwise pass over memory between the GEMMs:

    DenseFFN    add_rmsnorm_quant -> GEMM + SwiGLU -> linear + residual
    MoEFFN      router -> moe_sort -> moe_dispatch_quant -> grouped GEMM + SwiGLU
                -> quantizer -> grouped GEMM -> moe_combine (+ residual)

The activation scales are calibrated on the first batch (``calibrate``); the
expert layer shares one scale among its experts.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_quantized_linear_gb300 as nv  # noqa: E402

EPS = 1e-6


def global_scale(t: torch.Tensor) -> torch.Tensor:
    """gs = 448 * 6 / amax, a 1-element fp32 tensor."""
    return (2688.0 / t.float().abs().amax().clamp_min(1e-12)).reshape(1)


def rms_norm(x: torch.Tensor, gamma: torch.Tensor) -> torch.Tensor:
    v = x.float()
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * gamma.float()


class DenseFFN:
    """h = x + residual;  out = h + W_down swiglu(W_gate n, W_up n),  n = rms_norm(h) * gamma."""

    def __init__(self, gamma, w_gate, w_up, w_down):
        self.f, self.k = w_gate.shape
        self.gamma, self.n = gamma, w_down.shape[0]
        w1 = nv.interleave_gate_up(w_gate, w_up)
        self.gw1, self.gw2 = global_scale(w1), global_scale(w_down)
        self.w1, self.w1_sf = nv.prepare_weight(w1, self.gw1)
        self.w2, self.w2_sf = nv.prepare_weight(w_down, self.gw2)

    def calibrate(self, x, residual, hidden_amax=8.0):
        self.gs1 = global_scale(rms_norm(x.float() + residual.float(), self.gamma))
        self.gs2 = torch.full_like(self.gs1, 2688.0 / hidden_amax)
        self.alpha1, self.alpha2 = 1.0 / (self.gs1 * self.gw1), 1.0 / (self.gs2 * self.gw2)

    def __call__(self, x, residual):
        m = x.shape[0]
        x_q, x_sf, h = nv.add_rmsnorm_quant(x, self.gamma, EPS, residual=residual, gs=self.gs1)
        hidden = torch.empty((m, self.f), dtype=torch.bfloat16, device=x.device)
        nv.nvfp4_gemm_act(x_q, x_sf, m, self.w1, self.w1_sf, 2 * self.f, self.f, self.k, self.alpha1, None,
                          nv.ACTIVATIONS["swiglu"], None, 0, hidden, self.f)
        return nv.linear(hidden, self.w2, self.w2_sf, self.f, self.n, self.gs2, self.alpha2, residual=h)


class MoEFFN:
    """out = x + sum over a token's topk experts of weight * W_down[e] swiglu(W_gate[e] x, W_up[e] x)."""

    def __init__(self, router, w_gate, w_up, w_down, topk):
        self.e, self.f, self.k = w_gate.shape
        self.router, self.topk = router, topk
        w1 = torch.stack((w_gate, w_up), dim=2).reshape(self.e * 2 * self.f, self.k)    # interleaved per expert
        w2 = w_down.reshape(self.e * self.k, self.f)
        self.gw1, self.gw2 = global_scale(w1), global_scale(w2)
        self.w1, self.w1_sf = nv.prepare_weight(w1, self.gw1)
        self.w2, self.w2_sf = nv.prepare_weight(w2, self.gw2)

    def calibrate(self, x, hidden_amax=8.0):
        self.gs1 = global_scale(x)
        self.gs2 = torch.full_like(self.gs1, 2688.0 / hidden_amax)
        self.alpha1 = (1.0 / (self.gs1 * self.gw1)).expand(self.e).contiguous()
        self.alpha2 = (1.0 / (self.gs2 * self.gw2)).expand(self.e).contiguous()

    def route(self, x):
        top, ids = (x.float() @ self.router.float().T).topk(self.topk, dim=1)
        return ids, torch.softmax(top, dim=1)

    def __call__(self, x):
        ids, weights = self.route(x)
        offsets, _, dest = nv.moe_sort(ids, self.e)
        x_q, x_sf = nv.moe_dispatch_quant(x, self.gs1, dest, self.e)
        rows = x_q.shape[0]
        hidden = torch.empty((rows, self.f), dtype=torch.bfloat16, device=x.device)
        nv.nvfp4_grouped_gemm_act(x_q, x_sf, rows, offsets, self.e, self.w1, self.w1_sf, self.f, self.k, self.alpha1,
                                  None, nv.ACTIVATIONS["swiglu"], hidden, self.f)
        h_q, h_sf = nv.quant_act(hidden, self.gs2)
        y = torch.empty((rows, self.k), dtype=torch.bfloat16, device=x.device)
        nv.nvfp4_grouped_gemm(h_q, h_sf, rows, offsets, self.e, self.w2, self.w2_sf, self.k, self.f, self.alpha2, None,
                              y, self.k)
        return nv.moe_combine(y, dest, weights, residual=x)


def _rel(got, ref):
    return float((got.double() - ref.double()).norm() / ref.double().norm())


def main():
    if not torch.cuda.is_available():
        sys.exit("needs a GB300")
    nv.build()
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    k, f, m = 1024, 2048, 300
    x, r, gamma = rnd(m, k), rnd(m, k), (1 + rnd(k, std=0.1))
    wg, wu, wd = rnd(f, k, std=0.03), rnd(f, k, std=0.03), rnd(k, f, std=0.03)
    ffn = DenseFFN(gamma, wg, wu, wd)
    ffn.calibrate(x, r)
    h = x.float() + r.float()
    n = rms_norm(h, gamma)
    branch = (torch.nn.functional.silu(n @ wg.float().T) * (n @ wu.float().T)) @ wd.float().T
    print(f"dense: {m} x {k} -> {f} -> {k}, FFN branch against fp32 weights: rel {_rel(ffn(x, r).float() - h, branch):.3f}")

    e, topk, f = 16, 4, 512
    moe = MoEFFN(rnd(e, k, std=0.03), rnd(e, f, k, std=0.03), rnd(e, f, k, std=0.03), rnd(e, k, f, std=0.03), topk)
    moe.calibrate(x)
    out = moe(x)
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    print(f"moe:   {m} tokens, {e} experts, top {topk}: out {tuple(out.shape)}, finite {bool(out.isfinite().all())}")


if __name__ == "__main__":
    main()
