"""GPU tests of the training operators past 2^31 elements: rows at the end of tensors whose offsets
do not fit in 32 bits, against the same rows alone."""
import pytest
import torch

from _helpers import nv, require_library

pytestmark = [pytest.mark.gpu, pytest.mark.slow]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def filled(rows, cols, seed):
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    for at in range(0, rows, 8192):
        part = x[at:at + 8192]
        part.copy_(torch.randn(part.shape, device="cuda", generator=g))
    return x


def test_checkpoint_and_its_gradient():
    m, n = 70016, 16384                                      # 2.3e9 columns of x, 1.15e9 of the activation
    x = filled(m, 2 * n, 1)
    out, q, sf = nv.act_checkpoint(x, "swiglu")
    tail = slice(m - 128, m)                                 # a whole band, so that its scales stand alone too
    o2, q2, sf2 = nv.act_checkpoint(x[tail].contiguous(), "swiglu")
    torch.cuda.synchronize()
    assert torch.equal(out[tail], o2) and torch.equal(q[tail], q2) and torch.equal(sf[-sf2.numel():], sf2)
    del x
    dx, aq, asf = nv.act_checkpoint_backward(out, q, sf, "swiglu", recompute=True)
    d2, a2, s2 = nv.act_checkpoint_backward(out[tail].contiguous(), q2, sf2, "swiglu", recompute=True)
    torch.cuda.synchronize()
    assert torch.equal(dx[tail], d2) and torch.equal(aq[tail], a2) and torch.equal(asf[-s2.numel():], s2)


def test_weight_gradient():
    """dy past 2^31 elements and codes past 2^31 bytes: only the last rows are not zero."""
    m, n, k = 140032, 16384, 16384
    dy = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    dy[-100:], x[-100:] = filled(100, n, 2), filled(100, k, 3)
    _, q, sf = nv.act_checkpoint(x)
    tail = x[-100:].contiguous()
    del x
    dw = nv.checkpoint_wgrad(dy, q, sf, k, dtype=torch.bfloat16)
    _, q2, sf2 = nv.act_checkpoint(tail)
    d2 = nv.checkpoint_wgrad(dy[-100:].contiguous(), q2, sf2, k, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    # (the same products, 64 rows a step cut at other places: sums of 100 in another order)
    assert float((dw.float() - d2.float()).norm() / d2.float().norm()) <= 2.0 ** -8


def test_weight_gradient_of_more_than_2_31_elements():
    n, k = 90112, 24832                                      # 2.24e9 elements of dw
    dy, x = filled(64, n, 4), filled(64, k, 5)
    _, q, sf = nv.act_checkpoint(x)
    dw = nv.checkpoint_wgrad(dy, q, sf, k)
    last = nv.checkpoint_wgrad(dy[:, -256:].contiguous(), q, sf, k)
    torch.cuda.synchronize()
    assert torch.equal(dw[-256:], last)


def test_routing():
    t, e = 2_200_000, 1000                                   # 2.2e9 logits
    logits = torch.empty(t, e, dtype=torch.bfloat16, device="cuda")
    logits.normal_()
    ids, w = nv.moe_route(logits, 2)
    i2, w2 = nv.moe_route(logits[-50:].contiguous(), 2)
    torch.cuda.synchronize()
    assert torch.equal(ids[-50:], i2) and torch.equal(w[-50:], w2)
    dl = nv.moe_route_backward(w, ids, logits, renormalize=False)
    d2 = nv.moe_route_backward(w2, i2, logits[-50:].contiguous(), renormalize=False)
    torch.cuda.synchronize()
    assert torch.equal(dl[-50:], d2)
