"""A training step of the expert layer: FP4 products forward, 8-bit checkpoints kept, gradients of every parameter.

    python examples/moe_training.py

What the forward pass keeps for the backward pass, per routed row: its input and its gate/up product in
MXFP8 (8.25 bits an element), and the second product in bf16.  The hidden activation is not kept; the
activation's gradient writes it again, in MXFP8, for the second weight's gradient.

    forward    moe_route -> moe_sort -> dispatch (bf16 rows) -> act_checkpoint of the rows
               -> FP4 grouped GEMM -> act_checkpoint (SwiGLU) -> FP4 grouped GEMM -> moe_combine
    backward   moe_combine_backward -> rows' gradients times W2 -> act_checkpoint_backward (and the hidden
               activation) -> checkpoint_wgrad of W2 -> times W1, checkpoint_wgrad of W1 -> moe_combine
               (the dispatch's gradient), moe_route_backward

The products with the transposed weights run in bf16 on the master weights, by torch.matmul in a loop over the experts on the
host, which reads the groups' offsets and counts back: the other operators can be captured into a graph, this step as a whole not.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import ffn_block  # noqa: E402
from ffn_block import nv  # noqa: E402


class TrainableMoE(ffn_block.MoEFFN):
    """MoEFFN with its gradients.  The weights are those of MoEFFN, W1 interleaved [e, 2f, k], W2 [e, k, f]."""

    def __init__(self, router, w_gate, w_up, w_down, topk):
        super().__init__(router, w_gate, w_up, w_down, topk)
        self.w1_master = torch.stack((w_gate, w_up), dim=2).reshape(self.e, 2 * self.f, self.k)
        self.w2_master = w_down

    def forward(self, x):
        """(out, what the backward pass needs)."""
        s = {"x": x, "logits": x.float() @ self.router.float().T}
        s["ids"], s["weights"] = nv.moe_route(s["logits"], self.topk)
        s["offsets"], s["counts"], s["dest"] = nv.moe_sort(s["ids"], self.e)
        groups = s["offsets"], s["counts"]
        rows = nv.moe_dispatch(x, s["dest"], *groups)
        _, s["x_q"], s["x_sf"] = nv.act_checkpoint(rows, "none", *groups)
        a_q, a_sf = nv.quant_act(rows, self.gs1)
        m = rows.shape[0]
        pre = torch.empty((m, 2 * self.f), dtype=torch.bfloat16, device=x.device)
        nv.nvfp4_grouped_gemm(a_q, a_sf, m, s["offsets"], self.e, self.w1, self.w1_sf, 2 * self.f, self.k, self.alpha1,
                              None, pre, 2 * self.f)
        hidden, s["pre_q"], s["pre_sf"] = nv.act_checkpoint(pre, "swiglu", *groups)
        h_q, h_sf = nv.quant_act(hidden, self.gs2)
        s["y"] = torch.empty((m, self.k), dtype=torch.bfloat16, device=x.device)
        nv.nvfp4_grouped_gemm(h_q, h_sf, m, s["offsets"], self.e, self.w2, self.w2_sf, self.k, self.f, self.alpha2, None,
                              s["y"], self.k)
        return nv.moe_combine(s["y"], s["dest"], s["weights"], residual=x), s

    def _times(self, rows, weight, s):
        """rows @ weight[expert] for the rows of every expert; rows of nobody stay zero."""
        out = torch.zeros((rows.shape[0], weight.shape[2]), dtype=torch.bfloat16, device=rows.device)
        for e, (o, c) in enumerate(zip(s["offsets"].tolist(), s["counts"].tolist())):
            if c:
                torch.matmul(rows[o:o + c], weight[e], out=out[o:o + c])
        return out

    def backward(self, dout, s, grads=None):
        """(dx, {"router", "w1", "w2"}): fp32 gradients, added to `grads` if given."""
        g = (s["offsets"], s["counts"])
        dy, dweights = nv.moe_combine_backward(dout, s["y"], s["weights"], s["dest"], *g)
        dhidden = self._times(dy, self.w2_master, s)
        dpre, h_q, h_sf = nv.act_checkpoint_backward(dhidden, s["pre_q"], s["pre_sf"], "swiglu", *g, recompute=True)
        add = grads is not None
        old = grads or {"w1": None, "w2": None}
        new = {"w2": nv.checkpoint_wgrad(dy, h_q, h_sf, self.f, *g, dw=old["w2"], accumulate=add),
               "w1": nv.checkpoint_wgrad(dpre, s["x_q"], s["x_sf"], self.k, *g, dw=old["w1"], accumulate=add)}
        dx = nv.moe_combine(self._times(dpre, self.w1_master, s), s["dest"], residual=dout)
        dlogits = nv.moe_route_backward(dweights, s["ids"], s["logits"])
        router = dlogits.T @ s["x"].float()
        new["router"] = router + old["router"] if add else router
        return (dx.float() + dlogits @ self.router.float()).to(torch.bfloat16), new


def main():
    if not torch.cuda.is_available():
        sys.exit("needs a GB300")
    nv.build()
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    t, k, f, e, topk = 300, 512, 256, 8, 2
    layer = TrainableMoE(rnd(e, k, std=0.05), rnd(e, f, k, std=0.04), rnd(e, f, k, std=0.04), rnd(e, k, f, std=0.06), topk)
    x, target = rnd(t, k), rnd(t, k)
    layer.calibrate(x)
    grads = None
    for part in (slice(0, 150), slice(150, t)):              # two micro-batches
        out, saved = layer.forward(x[part].contiguous())
        dout = ((out.float() - target[part].float()) / t).to(torch.bfloat16)
        _, grads = layer.backward(dout, saved, grads)
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    for name, grad in grads.items():
        print(f"{name}: gradient {tuple(grad.shape)}, finite {bool(grad.isfinite().all())}, norm {float(grad.norm()):.4f}")


if __name__ == "__main__":
    main()
