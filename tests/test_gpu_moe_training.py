"""examples/moe_training.py: routing, checkpoints and their gradients together, as a training step runs them.

Every gradient is compared with its formula in 64 bits over what the step itself kept (routing,
checkpoints, the rows' gradients); each operator's own rounding is its test's matter, so the bounds here
are those of the bf16 tensors between them: a product of bf16 operands summed in fp32 and rounded to bf16, 2^-8
of itself, and for sums of such values 2^-8 of the sum of their magnitudes."""
import os
import sys

import numpy as np
import pytest
import torch

import _train_ref as ref
from _helpers import nv, require_library

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_training  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def layer_of(seed, t, k, f, e, topk):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    layer = moe_training.TrainableMoE(rnd(e, k, std=0.1), rnd(e, f, k, std=0.06), rnd(e, f, k, std=0.06),
                                      rnd(e, k, f, std=0.06), topk)
    x, dout = rnd(t, k), rnd(t, k, std=0.1)
    layer.calibrate(x)
    return layer, x, dout


def near(got, want, mag):
    tol = 2.0 ** -8 * (np.abs(want) + mag) + 1e-30
    err = np.abs(ref.f64(got) - want)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("t,k,f,e,topk", [(1, 256, 128, 4, 2), (70, 256, 128, 5, 3), (500, 512, 192, 8, 2), (40, 256, 128, 64, 4)])
def test_step(t, k, f, e, topk):
    layer, x, dout = layer_of(t, t, k, f, e, topk)
    out, s = layer.forward(x)
    dx, grads = layer.backward(dout, s)
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    # the forward pass is the inference layer's (its SwiGLU from the bf16 product instead of the accumulator)
    infer = layer(x).double()
    assert float((out.double() - infer).norm() / infer.norm()) <= 0.02

    ids, w = s["ids"].cpu().numpy(), ref.f64(s["weights"])
    dest, rows = s["dest"].cpu().numpy(), s["y"].shape[0]
    d, y = ref.f64(dout), ref.f64(s["y"])
    xv = ref.decode(s["x_q"], s["x_sf"], rows, k)
    pre = ref.decode(s["pre_q"], s["pre_sf"], rows, 2 * f)
    w1, w2 = ref.f64(layer.w1_master), ref.f64(layer.w2_master)
    bf = lambda v: torch.from_numpy(v).to(torch.float32).to(torch.bfloat16).double().numpy()   # noqa: E731
    dw1, dw2 = np.zeros((e, 2 * f, k)), np.zeros((e, k, f))
    m1, m2 = np.zeros_like(dw1), np.zeros_like(dw2)
    dxr, dxm, dweights = d.copy(), np.abs(d), np.zeros((t, topk))
    for i in range(t):
        for j in range(topk):
            r, ex = dest[i, j], ids[i, j]
            dweights[i, j] = d[i] @ y[r]
            dy = bf(np.float32(w[i, j]) * np.float32(1) * d[i])
            dh = bf(dy @ w2[ex])
            dp = ref.backward(pre[r:r + 1], dh[None], "swiglu")[0][0]
            h = ref.forward(pre[r:r + 1], "swiglu")[0]
            dw2[ex] += np.outer(dy, h)
            m2[ex] += np.outer(np.abs(dy), np.abs(h)) * 2 ** 5      # (h in MXFP8: 2^-4 of itself, an eighth where it saturates)
            dw1[ex] += np.outer(dp, xv[r])
            m1[ex] += np.outer(np.abs(dp) + 2 * np.abs(dp).max(), np.abs(xv[r]))
            dxr[i] += dp @ w1[ex]
            dxm[i] += 4 * (np.abs(dp) + np.abs(dp).max()) @ np.abs(w1[ex])
    near(grads["w2"].view(e, k, f), dw2, m2)
    near(grads["w1"].view(e, 2 * f, k), dw1, m1)
    dl, dlm = ref.route_gradient(dweights, ids.astype(np.int64), ref.f64(s["logits"]), "softmax", True, 1.0)
    router = ref.f64(layer.router)
    near(grads["router"], dl.T @ ref.f64(x), dlm.T @ np.abs(ref.f64(x)))
    near(dx, dxr + dl @ router, dxm + dlm @ np.abs(router))


def test_gradients_accumulate_over_micro_batches():
    """Two halves with accumulation against one after the other: fp32 sums of two."""
    layer, x, dout = layer_of(3, 200, 256, 128, 4, 2)
    parts = []
    for h in (slice(0, 90), slice(90, 200)):
        _, s = layer.forward(x[h].contiguous())
        parts.append((s, dout[h].contiguous()))
    one = [layer.backward(d, s)[1] for s, d in parts]
    total = None
    for s, d in parts:
        _, total = layer.backward(d, s, total)
    torch.cuda.synchronize()
    for name in ("w1", "w2", "router"):
        assert torch.equal(total[name], one[0][name] + one[1][name]), name


def test_back_to_back_steps_see_their_own_batch():
    """Steps without a synchronisation between them (programmatic dependents) give what they give alone."""
    layer, x, dout = layer_of(4, 300, 256, 128, 8, 2)
    xs = [x, (x.float() * 0.5).to(torch.bfloat16), -x]
    alone = []
    for v in xs:
        out, s = layer.forward(v)
        torch.cuda.synchronize()
        dx, g = layer.backward(dout, s)
        torch.cuda.synchronize()
        alone.append((out, dx, g["w1"], g["w2"], g["router"]))
    quick = []
    for v in xs:
        out, s = layer.forward(v)
        dx, g = layer.backward(dout, s)
        quick.append((out, dx, g["w1"], g["w2"], g["router"]))
    torch.cuda.synchronize()
    for a, b in zip(alone, quick):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_routing_to_the_checkpoint_captured_in_one_graph():
    """Routing, sorting, dispatch, checkpoints and gradients of a fixed batch size, replayed on new data."""
    t, h, e, topk, f = 64, 128, 8, 2, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dout = (torch.randn(t, h, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    logits = torch.randn(t, e, device="cuda", generator=g)
    rows = nv.nvfp4_moe_rows(t, topk, e)
    pre = torch.zeros(rows, 2 * f, dtype=torch.bfloat16, device="cuda")
    dhid = torch.randn(rows, f, device="cuda", generator=g).to(torch.bfloat16)

    def step():
        ids, w = nv.moe_route(logits, topk, "sigmoid", scale=2.0)
        offsets, counts, dest = nv.moe_sort(ids, e)
        xr = nv.moe_dispatch(x, dest, offsets, counts)
        _, xq, xsf = nv.act_checkpoint(xr, "none", offsets, counts)
        pre.copy_(xr)                                        # (stands for the product)
        hidden, pq, psf = nv.act_checkpoint(pre, "swiglu", offsets, counts)
        dpre, hq, hsf = nv.act_checkpoint_backward(dhid, pq, psf, "swiglu", offsets, counts, recompute=True)
        dw = nv.checkpoint_wgrad(dpre, xq, xsf, h, offsets, counts)
        dl = nv.moe_route_backward(w, ids, logits, "sigmoid", scale=2.0)
        return ids, w, dw, dl

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (6, 7):
        g.manual_seed(seed)
        x.copy_(torch.randn(t, h, device="cuda", generator=g)), logits.copy_(torch.randn(t, e, device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in captured]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_example_runs(capsys):
    moe_training.main()
    out = capsys.readouterr().out
    assert out.count("finite True") == 3
