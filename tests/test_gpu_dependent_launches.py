"""GPU tests of kernels that follow each other without a synchronisation, each reading
what the one before has written while it may still have been running: the same calls
with a synchronisation after each give the same bits.  The buffers are used again with
other data every time, so a stale value shows."""
import pytest
import torch

from _helpers import dev_scalar, nv, require_library
from test_gpu_grouped_pair import on_pairs

pytestmark = pytest.mark.gpu
ROUNDS = 12


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def quick_and_slow(chain):
    """chain(i, wait) -> tensors of round i; `wait` is called after every step."""
    quick = [chain(i, lambda: None) for i in range(ROUNDS)]
    torch.cuda.synchronize()
    slow = [chain(i, torch.cuda.synchronize) for i in range(ROUNDS)]
    torch.cuda.synchronize()
    nv.nvfp4_device_error()
    for i in range(ROUNDS):
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(quick[i], slow[i])), i


def _inputs(m, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(m, k, device="cuda", generator=g) * (1 + i)).bfloat16() for i in range(ROUNDS)]


def _weight(n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return nv.prepare_weight((torch.randn(n, k, device="cuda", generator=g) * 0.05).bfloat16(), dev_scalar(40.0))


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("m,k", [(1, 2048), (64, 2048), (128, 4096), (200, 2048), (700, 1024)])
def test_the_norms_h_as_the_gemms_residual(m, k, act):
    """One-CTA kernel (m <= 128) and CTA pairs."""
    x, r = _inputs(m, k, 1), _inputs(m, k, 2)
    gamma = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    gs, alpha = dev_scalar(60.0), dev_scalar(1e-3)
    w = _weight(k, k, 3)
    h = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(m, k // 2, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(nv.nvfp4_scale_bytes(m, k), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def chain(i, wait):
        out = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
        wait()
        nv.nvfp4_add_rmsnorm_quant(x[i], k, r[i], k, gamma, 1e-6, m, k, nv.NVFP4_FORMAT_NVFP4, gs, h, k, q, sf)
        wait()
        nv.nvfp4_gemm_act(q, sf, m, *w, k, k, k, alpha, None, nv.ACTIVATIONS[act], h, k, out, k)
        wait()
        return [out]

    quick_and_slow(chain)


@pytest.mark.parametrize("m", [8, 60, 300])
def test_a_gemms_output_and_its_dynamic_scale_into_a_linear(m):
    """x, the global scale and alpha of a linear from the kernels before it: the
    single-launch linear (m = 8) and the quantizer in front of both GEMM kernels."""
    k = 1024
    x = _inputs(m, k, 4)
    w1, w2 = _weight(k, k, 5), _weight(k, k, 6)
    gw = dev_scalar(40.0)
    mid = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    gs, alpha = dev_scalar(0.0), dev_scalar(0.0)
    gs1, alpha1 = dev_scalar(50.0), dev_scalar(5e-4)
    ws = torch.zeros(nv.nvfp4_linear_workspace_bytes(m, k, k), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def chain(i, wait):
        out = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
        wait()
        nv.nvfp4_linear_act(x[i], m, k, k, gs1, None, 0, *w1, k, k, alpha1, None, nv.ACTIVATIONS["none"], x[i], k,
                            mid, k, ws, ws.numel())
        wait()
        nv.nvfp4_act_global_scale(mid, m, k, k, None, 0, gw, gs, alpha)
        wait()
        nv.nvfp4_linear(mid, m, k, k, gs, None, 0, *w2, k, k, alpha, None, out, k, ws, ws.numel())
        wait()
        first = out.clone()
        wait()
        # without the scale's pass between them: the quantizer right behind the GEMM that writes x
        nv.nvfp4_linear_act(x[i], m, k, k, gs1, None, 0, *w1, k, k, alpha1, None, nv.ACTIVATIONS["silu"], None, 0,
                            mid, k, ws, ws.numel())
        wait()
        nv.nvfp4_linear(mid, m, k, k, gs, None, 0, *w2, k, k, alpha, None, out, k, ws, ws.numel())
        wait()
        return [first, out]

    quick_and_slow(chain)


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_routing_into_the_one_cta_grouped_gemm(act):
    """Sort, dispatch and grouped GEMM in turn on the same buffers, another routing each
    time, where the groups are small enough for the one-CTA kernel."""
    tokens, topk, experts, h, nw = 600, 2, 16, 512, 1280
    n = nw // 2 if act == "swiglu" else nw
    g = torch.Generator(device="cuda").manual_seed(10)
    x = torch.randn(tokens, h, device="cuda", generator=g).bfloat16()
    wq = _weight(experts * nw, h, 11)
    al = torch.full((experts,), 1e-4, device="cuda")
    bias = torch.randn(experts * nw, device="cuda", generator=g).bfloat16()
    rows = nv.nvfp4_moe_rows(tokens, topk, experts)
    assert not on_pairs(rows, experts, nw)
    q = torch.zeros(rows, h // 2, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(nv.nvfp4_scale_bytes(rows, h), dtype=torch.uint8, device="cuda")
    ws = torch.empty(nv.nvfp4_moe_sort_workspace_bytes(tokens, topk, experts), dtype=torch.uint8, device="cuda")
    off = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(experts, dtype=torch.int32, device="cuda")
    dest = torch.zeros(tokens, topk, dtype=torch.int32, device="cuda")
    gs = dev_scalar(40.0)
    y = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    ids = [torch.randint(0, 1 + (5 * i) % experts, (tokens, topk), device="cuda", generator=g, dtype=torch.int32)
           for i in range(ROUNDS)]
    torch.cuda.synchronize()

    def chain(i, wait):
        out = torch.empty(tokens, n, dtype=torch.bfloat16, device="cuda")
        wait()
        nv.nvfp4_moe_sort(ids[i], 4, tokens, topk, experts, off, cnt, dest, ws, ws.numel())
        wait()
        nv.nvfp4_moe_dispatch_quant(x, h, gs, dest, tokens, topk, rows, h, q, sf)
        wait()
        nv.nvfp4_grouped_gemm_act(q, sf, rows, off, experts, *wq, n, h, al, bias, nv.ACTIVATIONS[act], y, n)
        wait()
        nv.nvfp4_moe_combine(y, n, None, dest, tokens, topk, rows, n, None, 0, out, n)
        wait()
        return [out]

    quick_and_slow(chain)
