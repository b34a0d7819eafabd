"""Host-side refusals of the tensor-level helpers (no GPU needed): types, shapes, strides
and devices that the library, which sees addresses only, would read past the end or
misread.  The CPU tensors here are right in all but the named one; where all are right the
refusal is the device's."""
import pytest
import torch

import nvfp4_quantized_linear_gb300 as nv

M, K, N, T, TOPK, E = 4, 64, 128, 6, 2, 3
BF = torch.bfloat16


def zeros(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def refused(f, name, **kw):
    with pytest.raises(ValueError, match=rf"^{name}\b"):
        f(**kw)


def cases(f, good, bad):
    refused(f, next(iter(good)), **good)                     # the first one's device
    for name, tensors in bad.items():
        for t in tensors:
            refused(f, name, **{**good, name: t})


def linear_args():
    return dict(x=zeros(M, K), w_fp4=zeros(N, K // 2, dtype=torch.uint8), w_sf=zeros(512, dtype=torch.uint8), k=K, n_out=N,
                bias=zeros(N), residual=zeros(M, N), out=zeros(M, N))


ROWS_BAD = [zeros(M, N, dtype=torch.float32), zeros(M, N, dtype=torch.float16), zeros(M - 1, N), zeros(1, N), zeros(M, N - 8),
            zeros(N, M).T, zeros(N)]


@pytest.mark.parametrize("f,more", [(nv.linear, dict(gs=zeros(1, dtype=torch.float32), alpha=zeros(1, dtype=torch.float32))),
                                    (nv.mxfp4_linear, {})])
def test_linear(f, more):
    good = {**linear_args(), **more}
    cases(f, good, {"residual": ROWS_BAD, "out": ROWS_BAD, "x": [zeros(M, K, dtype=torch.float32), zeros(M, K - 8)],
                    "bias": [zeros(N - 1), zeros(N, dtype=torch.float32), zeros(2 * N)[::2]],
                    **{name: [zeros(1, dtype=torch.float64), zeros(0, dtype=torch.float32)] for name in more}})
    refused(f, "bias", **{**good, "act": "swiglu"})          # one entry per gate and up row
    refused(f, "unknown activation", **{**good, "act": "tanh"})


def test_raw_16_bit_storage_and_wider_rows_pass():
    """They reach the last check, the device's."""
    good = dict(linear_args(), gs=None, alpha=None)
    refused(nv.linear, "x must be a CUDA", **{**good, "residual": zeros(M, N, dtype=torch.int16)})
    refused(nv.linear, "x must be a CUDA", **{**good, "residual": zeros(M + 2, N + 8), "x": zeros(M, K + 64)[:, :K]})


def test_norm():
    good = dict(x=zeros(M, K), gamma=zeros(K), eps=1e-6, residual=zeros(M, K), gs=zeros(1, dtype=torch.float32), h=zeros(M, K))
    rows = [zeros(M, K, dtype=torch.float32), zeros(M - 1, K), zeros(1, K), zeros(M, K - 8), zeros(K, M).T]
    cases(nv.add_rmsnorm_quant, good, {
        "residual": rows, "h": rows, "x": [zeros(M, K, dtype=torch.float32)],
        "gamma": [zeros(K, dtype=torch.float32), zeros(K - 1), zeros(2 * K)[::2]], "gs": [zeros(1, dtype=torch.float64)]})


def routing():
    i32 = torch.int32
    return dict(dest=zeros(T, TOPK, dtype=i32), group_offsets=zeros(E + 1, dtype=i32), group_counts=zeros(E, dtype=i32))


ROUTING_BAD = {"dest": [zeros(T, TOPK, dtype=torch.int64), zeros(T, 2 * TOPK, dtype=torch.int32)[:, ::2],
                        zeros(T, dtype=torch.int32)],
               "group_offsets": [zeros(E, dtype=torch.int32), zeros(E + 1, dtype=torch.int64)],
               "group_counts": [zeros(E, dtype=torch.int64), zeros(2 * E, dtype=torch.int32)[::2]]}
WEIGHTS_BAD = [zeros(T, TOPK), zeros(T, TOPK, dtype=torch.float16), zeros(T, TOPK, dtype=torch.float64),
               zeros(T, 4, dtype=torch.float32)[:, :TOPK], zeros(T, TOPK + 1, dtype=torch.float32),
               zeros(T - 1, TOPK, dtype=torch.float32), zeros(TOPK, T, dtype=torch.float32)]


def test_dispatch():
    cases(nv.moe_dispatch, dict(x=zeros(T, K), **routing(), out=zeros(512, K)), {
        "x": [zeros(T - 1, K), zeros(T, K, dtype=torch.float32)], "out": [zeros(512, K - 8), zeros(512, K, dtype=torch.float32)],
        **ROUTING_BAD})
    cases(nv.moe_dispatch_quant, dict(x=zeros(T, K), gs=zeros(1, dtype=torch.float32), dest=routing()["dest"], experts=E), {
        "x": [zeros(T - 1, K), zeros(T, K, dtype=torch.float32)], "gs": [zeros(1, dtype=torch.float64)],
        "dest": ROUTING_BAD["dest"]})


def test_combine():
    rows = [zeros(T - 1, K), zeros(T, K - 8), zeros(T, K, dtype=torch.float32)]
    good = dict(y=zeros(512, K), dest=routing()["dest"], weights=zeros(T, TOPK, dtype=torch.float32), residual=zeros(T, K),
                out=zeros(T, K))
    cases(nv.moe_combine, good, {"weights": WEIGHTS_BAD, "dest": ROUTING_BAD["dest"], "residual": rows, "out": rows,
                                 "y": [zeros(512, K, dtype=torch.float32)]})


def test_combine_backward():
    good = dict(dout=zeros(T, K), y=zeros(512, K), weights=zeros(T, TOPK, dtype=torch.float32), **routing(), dy=zeros(512, K))
    cases(nv.moe_combine_backward, good, {
        "weights": WEIGHTS_BAD, **ROUTING_BAD, "dout": [zeros(T - 1, K), zeros(T, K, dtype=torch.float32)],
        "dy": [zeros(511, K), zeros(512, K - 8), zeros(512, K, dtype=torch.float32)], "y": [zeros(512, K, dtype=torch.float32)]})


def test_sort():
    refused(nv.moe_sort, "expert_ids must be a CUDA", expert_ids=zeros(T, TOPK, dtype=torch.int32), experts=E)


def test_combine_refuses_more_columns_than_its_grid_takes():
    """On the host, with the reason, instead of a failed launch."""
    nv.build()
    f = nv.load_library().nvfp4_moe_combine
    h, (y, dest, out) = 65535 * 1024 + 8, (1 << 40, 1 << 20, 1 << 42)
    assert f(y, h, None, dest, 1, 1, 1, h, None, 0, out, h, None) == 1
    assert str(65535 * 1024) in nv.nvfp4_last_error_string()
