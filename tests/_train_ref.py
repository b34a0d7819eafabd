"""Plain 64-bit references of expert routing, the 8-bit activation checkpoints and their gradients."""
from __future__ import annotations

import numpy as np
import torch

from _block_ref import e4m3, e4m3_value, f64, floor_log2, untile

FLT_MAX = float(np.finfo(np.float32).max)


# ------------------------------------------------------------------ routing ----

def clean(logits):
    l = np.asarray(logits, np.float64)
    return np.where(np.isnan(l), -np.inf, np.minimum(l, FLT_MAX))


def scores(l, score):
    """Softmax over the last axis or sigmoid, 0 for -inf."""
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return np.where(l > -np.inf, 1.0 / (1.0 + np.exp(-l)), 0.0)
        m = l.max(1, keepdims=True)
        z = np.exp(l - np.where(m > -np.inf, m, 0.0))
        return z / np.maximum(z.sum(1, keepdims=True), 1e-300)


def best(key, count):
    """Indices of the `count` highest in descending order, ties to the lower index; -1 where the key is -inf."""
    order = np.argsort(-key, axis=1, kind="stable")[:, :count]
    return np.where(np.take_along_axis(key, order, 1) > -np.inf, order, -1)


def choose(logits, topk, score, bias=None, groups=1, group_top=1, topk_groups=1):
    l = clean(logits)
    s = scores(l, score)
    if bias is None:
        key = l
    else:
        b = np.asarray(bias, np.float64)[None]
        key = np.where((l > -np.inf) & (b > -np.inf), s + b, -np.inf)
    if groups > 1:
        by = np.where(key > -np.inf, s, -np.inf) if bias is None and group_top == 2 else key
        by = np.sort(by.reshape(l.shape[0], groups, -1), 2)[..., ::-1][..., :group_top]
        value = np.where(by[..., 0] > -np.inf, np.where(by > -np.inf, by, 0.0).sum(2), -np.inf)
        kept = np.zeros((l.shape[0], groups), bool)
        for t, row in enumerate(best(value, topk_groups)):
            kept[t, row[row >= 0]] = True
        key = np.where(np.repeat(kept, l.shape[1] // groups, 1), key, -np.inf)
    return best(key, topk)


def weights(logits, ids, score, renorm, scale):
    """Weights of given ids (-1: 0).  Shares from exponentials relative to the largest, so that nothing underflows."""
    l = clean(logits)
    have = ids >= 0
    at = np.where(have, np.take_along_axis(l, np.maximum(ids, 0), 1), -np.inf)
    if not renorm:
        s = scores(l, score)
        return scale * np.where(have, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    top = at.max(1, keepdims=True)
    if score == "softmax":
        w = np.exp(at - np.where(top > -np.inf, top, 0.0))
    else:
        shift = np.where(top > -np.inf, np.minimum(top, 0.0), 0.0)
        with np.errstate(over="ignore"):
            w = np.where(at > 0, 1.0 / (1.0 + np.exp(-np.abs(at))), np.exp(np.minimum(at, 0.0) - shift) / (1.0 + np.exp(np.minimum(at, 0.0))))
    w = np.where(have, w, 0.0)
    return scale * w / np.maximum(w.sum(1, keepdims=True), 1e-300)


def route_gradient(dw, ids, logits, score, renorm, scale):
    """(dlogits, a bound of the terms' magnitudes) by the formulas, slot by slot."""
    l = clean(logits)
    have = (ids >= 0) & (np.take_along_axis(l, np.maximum(ids, 0), 1) > -np.inf)
    i = np.maximum(ids, 0)
    out, mag = np.zeros_like(l), np.zeros_like(l)
    g = np.where(have, dw * scale, 0.0)
    w = weights(l, np.where(have, ids, -1), score, renorm, 1.0)
    for t in range(l.shape[0]):
        dot, adot = (w[t] * g[t]).sum(), (w[t] * abs(g[t])).sum()
        for j in range(ids.shape[1]):
            if not have[t, j]:
                continue
            x, a = l[t, i[t, j]], abs(g[t, j])
            if renorm:
                f = w[t, j] * (1.0 if score == "softmax" else 1.0 / (1.0 + np.exp(min(x, 700.0))))
                out[t, i[t, j]] += f * (g[t, j] - dot)
                mag[t, i[t, j]] += f * (a + adot)
            elif score == "sigmoid":
                f = w[t, j] / (1.0 + np.exp(min(x, 700.0)))
                out[t, i[t, j]] += g[t, j] * f
                mag[t, i[t, j]] += a * f
            else:
                out[t, i[t, j]] += g[t, j] * w[t, j]
                mag[t, i[t, j]] += a * w[t, j]
        if not renorm and score == "softmax":
            s = scores(l[t:t + 1], score)[0]
            out[t] -= s * dot
            mag[t] += s * adot
    return out, mag


# -------------------------------------------------------------- checkpoints ----

def mxfp8(v):
    """(values of the codes, scale codes) of [rows, cols], padded to 32 columns; code 255 for blocks with a non-finite."""
    kp = (v.shape[1] + 31) // 32 * 32
    b = np.pad(v, ((0, 0), (0, kp - v.shape[1]))).reshape(v.shape[0], -1, 32)
    amax = np.abs(b).max(2)
    bad = ~np.isfinite(amax)
    s = np.where(amax > 0, np.clip(floor_log2(np.where(bad | (amax == 0), 1.0, amax)) - 8, -127, 127), -127)
    with np.errstate(invalid="ignore"):
        a = np.abs(b) * 2.0 ** -s[..., None]
        q = np.where(np.signbit(b), -1.0, 1.0) * e4m3(np.where(np.isfinite(a), a, 0.0))
    return q.reshape(v.shape[0], kp), np.where(bad, 255, s + 127).astype(np.int64)


def decode(q, sf, rows, cols):
    """[rows, cols] values of an MXFP8 operand (tiled scales), NaN for scale code 255."""
    kp = (cols + 31) // 32 * 32
    codes = untile(sf.cpu().numpy().reshape(-1), rows, kp // 32)[0].astype(np.int64)
    scale = np.where(codes == 255, np.nan, 2.0 ** (codes - 127.0))
    v = e4m3_value(q.cpu().numpy().reshape(rows, kp)).reshape(rows, -1, 32) * scale[..., None]
    return v.reshape(rows, kp)[:, :cols]


def make_mxfp8(v):
    """Device operands (q, sf) of float64 values [rows, cols], written by the definition."""
    rows = v.shape[0]
    q, s = mxfp8(v)
    a = torch.from_numpy(np.abs(q)).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    codes = np.where(np.signbit(q), a + 128, a).astype(np.uint8)
    rp, cp = (rows + 127) // 128 * 128, (s.shape[1] + 3) // 4 * 4
    full = np.zeros((rp, cp), np.uint8)
    full[:rows, :s.shape[1]] = s
    flat = full.reshape(rp // 128, 4, 32, cp // 4, 4).transpose(0, 3, 2, 1, 4).reshape(-1)
    return torch.from_numpy(codes).cuda(), torch.from_numpy(np.ascontiguousarray(flat)).cuda()


def act_and_slope(v, act):
    """(act(v), act'(v), magnitude of the slope's terms)."""
    if act == "none":
        return v, np.ones_like(v), np.ones_like(v)
    if act == "relu":
        return np.maximum(v, 0.0), (v > 0) * 1.0, (v > 0) * 1.0
    b, c = (1.0, 0.0) if act == "silu" else (2.0 * np.sqrt(2.0 / np.pi), 0.044715)
    u, du = b * (v + c * v ** 3), b * (1.0 + 3.0 * c * v * v)
    with np.errstate(over="ignore"):
        s, t = 1.0 / (1.0 + np.exp(-u)), 1.0 / (1.0 + np.exp(u))
    return v * s, s + v * s * t * du, s + np.abs(v * du) * s * t


def forward(v, act):
    if act in ("swiglu", "geglu"):
        return act_and_slope(v[:, 0::2], "silu" if act == "swiglu" else "gelu")[0] * v[:, 1::2]
    return act_and_slope(v, act)[0]


def backward(v, d, act):
    """(dx, magnitude of its terms)."""
    if act not in ("swiglu", "geglu"):
        _, slope, mag = act_and_slope(v, act)
        return d * slope, np.abs(d) * mag
    f, slope, mag = act_and_slope(v[:, 0::2], "silu" if act == "swiglu" else "gelu")
    out, m = np.empty_like(v), np.empty_like(v)
    out[:, 0::2], out[:, 1::2] = d * slope * v[:, 1::2], d * f
    m[:, 0::2], m[:, 1::2] = np.abs(d * v[:, 1::2]) * mag, np.abs(d * f)
    return out, m


# ------------------------------------------------------------------- groups ----

def groups_of(counts):
    """(offsets, counts, rows, bool [rows] of the real ones) of group sizes, rows with a band behind the last group."""
    counts = np.asarray(counts)
    offsets = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    rows = int(offsets[-1]) + 128
    real = np.zeros(rows, bool)
    for o, c in zip(offsets, counts):
        real[o:o + c] = True
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()   # noqa: E731
    return dev(offsets), dev(counts), rows, real


__all__ = [n for n in dir() if not n.startswith("_")] + ["f64"]
