"""Plain 64-bit references of the operators around the linear layer (numpy)."""
from __future__ import annotations

import numpy as np
import torch

FMT_NVFP4, FMT_MXFP4, FMT_MXFP8 = 0, 1, 2


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def bf16_round(v: np.ndarray) -> np.ndarray:
    """fp32 values rounded to bf16 (nearest even), as float64."""
    return f64(torch.from_numpy(np.asarray(v, np.float32)).to(torch.bfloat16))


def _on_steps(a, step):
    """|a| rounded to multiples of `step`, ties to even (np.rint)."""
    return np.rint(a / step) * step


def e4m3(v):
    """Nearest-even saturating E4M3 of v >= 0."""
    v = np.minimum(v, 1e30)
    e = np.floor(np.log2(np.maximum(v, 2.0 ** -6)))
    return np.minimum(_on_steps(v, 2.0 ** (e - 3)), 448.0)


def e2m1(v):
    """Nearest-even saturating E2M1 of v >= 0."""
    step = np.where(v < 2, 0.5, np.where(v < 4, 1.0, 2.0))
    return np.minimum(_on_steps(v, step), 6.0)


E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_value(codes):
    """Values of E4M3 bytes (finite codes)."""
    c = np.asarray(codes).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(c & 128, -v, v)


def unpack_fp4(packed):
    b = np.asarray(packed)
    return E2M1[np.stack((b & 15, b >> 4), -1).reshape(b.shape[0], -1)]


def untile(flat, rows, cols):
    """Linear [rows, cols] of a tiled scale buffer, and the full padded array."""
    rp, cp = (rows + 127) // 128 * 128, (cols + 3) // 4 * 4
    full = np.asarray(flat)[:rp * cp].reshape(rp // 128, cp // 4, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(rp, cp)
    return full[:rows, :cols], full


def floor_log2(v):
    m, e = np.frexp(v)
    return e - 1.0


def activation(v, act):
    if act in ("swiglu", "geglu"):
        return activation(v[:, 0::2], "silu" if act == "swiglu" else "gelu") * v[:, 1::2]
    if act == "relu":
        return np.maximum(v, 0.0)
    if act == "silu":
        return v / (1.0 + np.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (v + 0.044715 * v ** 3)))
    return v


def sort(ids, experts):
    """(offsets, counts, dest) of the stable sort into 128-aligned groups."""
    flat = np.asarray(ids).reshape(-1)
    counts = np.array([(flat == e).sum() for e in range(experts)], np.int64)
    offsets = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    dest = np.full(flat.shape, -1, np.int64)
    nxt = offsets[:-1].copy()
    for i, e in enumerate(flat):
        if 0 <= e < experts:
            dest[i] = nxt[e]
            nxt[e] += 1
    return offsets, counts, dest.reshape(np.asarray(ids).shape)
