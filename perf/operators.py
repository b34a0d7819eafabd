"""The operators around the FP4 linear of a transformer block, as cases to measure.

Six kinds of case (``op``):

  norm         residual addition + RMS norm + MXFP8 output (E4M3 codes, one E8M0 scale per 32 elements)
  norm_linear  the same norm with NVFP4 output, straight into the FP4 GEMM with its activation epilogue
  linear       FP4 linear (quantizer + GEMM) with bias, activation (gated or not) and residual in the epilogue
  dispatch     tokens sorted by expert into 128-row aligned groups, their rows copied there
  combine      expert rows gathered back per token with weights and residual; ``grad`` runs the gradient
  moe          a whole FP4 mixture-of-experts layer: sort, quantizing dispatch, two grouped GEMMs, combine

``run`` has two forms over the same state: ``own`` False is elementary torch in fp32, ``own`` True the calls of
``nvfp4_quantized_linear_gb300``.  Weights are interleaved (gate row 2j, up row 2j + 1), quantized and laid out
once in ``prepare``, as a user does at load time; every output buffer is the caller's.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
GATED = ("swiglu", "geglu")


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one decoded token through a norm whose layer is kept in 8 bits: pure latency
        dict(name="norm_token", op="norm", m=1, k=4096, pad=0, res=True),
        # a small batch, K not a multiple of 512, rows of a wider buffer, the first layer's norm (no residual)
        dict(name="norm_ragged", op="norm", m=333, k=5128, pad=56, res=False),
        # a long prompt's norm
        dict(name="norm_prompt", op="norm", m=16384, k=5120, pad=0, res=True),
        # a decode batch: norm into NVFP4, then the gate/up projection with SwiGLU in its epilogue
        dict(name="norm_linear_batch", op="norm_linear", m=64, k=4096, n=14336, act="swiglu", res=True),
        # one decoded token's down projection with the residual added in the epilogue
        dict(name="linear_token", op="linear", m=1, k=14336, n=4096, act="none", bias=False, res=True),
        # odd rows, padded K, columns that end inside a tile; bias + GELU (the MLP of an encoder-style block)
        dict(name="linear_ragged", op="linear", m=333, k=4104, n=2072, act="gelu", bias=True, res=True),
        # a prompt's gate/up projection with SwiGLU
        dict(name="linear_prompt", op="linear", m=8192, k=4096, n=14336, act="swiglu", bias=False, res=False),
        # a few decoded tokens routed to many experts: latency
        dict(name="dispatch_decode", op="dispatch", t=8, h=2048, e=64, topk=4),
        # a training batch's dispatch
        dict(name="dispatch_train", op="dispatch", t=16384, h=2048, e=128, topk=8),
        # a ragged prompt's combine with the residual
        dict(name="combine_ragged", op="combine", t=1003, h=5120, e=40, topk=6, weights=True, res=True, grad=False),
        # the combine's gradient in training: rows and routing weights
        dict(name="combine_grad", op="combine", t=8192, h=2048, e=64, topk=8, weights=True, res=False, grad=True),
        # a whole FP4 MoE layer on a prompt
        dict(name="moe_prompt", op="moe", t=2048, h=2048, f=768, e=32, topk=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges (sizes of 1536 and 3072 are moved on by one step of 8, but for the
    layer whose sizes are multiples of 128)."""
    c = _draw(rng)
    return c if c["op"] == "moe" else {k: v + 8 if type(v) is int and v in (1536, 3072) else v for k, v in c.items()}


def _draw(rng):
    op = rng.choice(["norm", "norm_linear", "linear", "dispatch", "combine", "moe"])
    if op == "norm":
        return dict(op=op, m=_log(rng, 1, 16384), k=8 * _log(rng, 32, 640), pad=8 * rng.randint(0, 9),
                    res=rng.random() < 0.7)
    if op in ("norm_linear", "linear"):
        act = rng.choice(["none", "relu", "gelu", "silu", "swiglu", "geglu"])
        m, k, n = _log(rng, 1, 8192), 8 * _log(rng, 32, 1792), 8 * _log(rng, 16, 1792)
        while m * k * n > 8192 * 4096 * 14336 // 2:
            m = max(1, m // 2)
        c = dict(op=op, m=m, k=k, n=n, act=act)
        if op == "norm_linear":
            return dict(c, res=rng.random() < 0.7)
        return dict(c, bias=rng.random() < 0.5, res=rng.random() < 0.5)
    topk = rng.randint(1, 8)
    e = max(topk, _log(rng, 4, 128))
    if op == "moe":
        return dict(op=op, t=_log(rng, 1, 2048), h=128 * rng.randint(2, 16), f=64 * rng.randint(2, 12),
                    e=min(e, 32), topk=min(topk, 4, e))
    c = dict(op=op, t=_log(rng, 1, 16384), h=8 * _log(rng, 32, 640), e=e, topk=topk)
    while c["t"] * c["topk"] * c["h"] > 8192 * 8 * 2048:
        c["t"] = max(1, c["t"] // 2)
    if op == "dispatch":
        return c
    grad = rng.random() < 0.5
    weights = grad or rng.random() < 0.7
    return dict(c, weights=weights, res=not grad and rng.random() < 0.5, grad=grad)


# -------------------------------------------------- formats (plain torch) ----

def _pad32(k):
    return (k + 31) // 32 * 32


def _rows(t, topk, e):
    """Rows of a dispatched operand: every group padded to 128 rows, whatever the routing."""
    n = t * topk
    return (n + 127 * min(e, n)) // 128 * 128


def _tile(codes):
    """[rows, cols] scale bytes -> the GEMM's 512-byte tiles of 128 rows x 4 columns (zero padding), flat."""
    r, c = codes.shape
    rp, cp = (r + 127) // 128 * 128, (c + 3) // 4 * 4
    full = torch.zeros(rp, cp, dtype=codes.dtype, device=codes.device)
    full[:r, :c] = codes
    return full.view(rp // 128, 4, 32, cp // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile(flat, r, c):
    rp, cp = (r + 127) // 128 * 128, (c + 3) // 4 * 4
    return flat.view(rp // 128, cp // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rp, cp)[:r, :c]


def _e4m3(v):
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _fp4(v, gs):
    """NVFP4 of [rows, kp] fp32: E2M1 values (fp32) and E4M3 block scales (fp32), every step one fp32 rounding."""
    r, kp = v.shape
    b = v.view(r, kp // 16, 16)
    six = torch.full_like(gs, 6.0)
    sf = _e4m3(b.abs().amax(-1) * gs / six).float()
    inv = torch.where(sf > 0, gs / sf, torch.zeros_like(sf))
    a = (b * inv[..., None]).abs()
    q = (0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75) + 1.0 * (a > 2.5)
         + 1.0 * (a >= 3.5) + 2.0 * (a > 5.0))
    return torch.copysign(q, b).view(r, kp), sf


def _widen(x, k):
    """fp32 copy of [m, k], zero-padded to a multiple of 32 columns."""
    v = torch.zeros(x.shape[0], _pad32(k), dtype=torch.float32, device=x.device)
    v[:, :k] = x
    return v


def _pack(q):
    """E2M1 values -> two 4-bit codes per byte (even element in the low nibble)."""
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + 8 * torch.signbit(q).to(torch.uint8)
    return (code[:, 0::2] + 16 * code[:, 1::2]).contiguous()


def _dequant(packed, sf_flat, rows, k):
    """The fp32 values (without global scale) of a packed NVFP4 operand with tiled scales: [rows, kp]."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=packed.device)
    v = torch.stack((grid[(packed & 15).int()], grid[(packed >> 4).int()]), -1).view(rows, -1, 16)
    sf = _untile(sf_flat, rows, _pad32(k) // 16).view(torch.float8_e4m3fn).float()
    return (v * sf[..., None]).view(rows, -1)


# ---------------------------------------------------------------- prepare ----

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _act(g, m, k, std=1.0):
    """Activations with a few large channels, as hidden states have."""
    x = torch.randn(m, k, generator=g, device=DEV) * std
    x[:, torch.randint(0, k, (max(1, k // 1000),), generator=g, device=DEV)] *= 20.0
    return x.to(torch.bfloat16)


def _scalar(v):
    return v.float().reshape(1).contiguous()


def _gs(x):
    return _scalar(2688.0 / x.float().abs().amax().clamp_min(1e-20))


def _weight(g, n, k):
    """A quantized [n, k] weight: packed codes, tiled scale bytes, global scale."""
    w = (torch.randn(n, k, generator=g, device=DEV) * 0.02).to(torch.bfloat16)
    gs = _gs(w)
    q, sf = _fp4(_widen(w, k), gs)
    return _pack(q), _tile(sf.to(torch.float8_e4m3fn).view(torch.uint8)), gs


def _routing(g, t, e, topk):
    """Expert ids of a skewed router (some experts busy, some empty), each token's distinct; a few assignments
    masked with -1 (padding tokens, experts of another device).  Softmax weights."""
    logits = torch.randn(t, e, generator=g, device=DEV) + 1.5 * torch.randn(1, e, generator=g, device=DEV)
    top, ids = logits.topk(topk, dim=1)
    drop = torch.rand(t, topk, generator=g, device=DEV) < 0.02
    return torch.where(drop, -1, ids).to(torch.int32), torch.softmax(top, 1)


def prepare(case, seed):
    g = _gen(seed)
    c, op = case, case["op"]
    s = {"case": dict(case)}
    if op in ("norm", "norm_linear"):
        m, k = c["m"], c["k"]
        s["x"] = _act(g, m, k + c.get("pad", 0))[:, :k]
        s["r"] = _act(g, m, k) if c["res"] else None
        s["gamma"] = (1.0 + 0.1 * torch.randn(k, generator=g, device=DEV)).to(torch.bfloat16)
        s["h"] = torch.empty(m, k, dtype=torch.bfloat16, device=DEV) if c["res"] else None
        kp, mp = _pad32(k), (m + 127) // 128 * 128
        if op == "norm":
            s["q"] = torch.empty(m, kp, dtype=torch.uint8, device=DEV)
            s["sf"] = torch.empty(mp * ((kp // 32 + 3) // 4 * 4), dtype=torch.uint8, device=DEV)
        else:
            s["q"] = torch.empty(m, kp // 2, dtype=torch.uint8, device=DEV)
            s["sf"] = torch.empty(mp * ((kp // 16 + 3) // 4 * 4), dtype=torch.uint8, device=DEV)
            s["gs"] = torch.full((1,), 2688.0 / 64.0, device=DEV)      # calibrated on earlier data
    if op in ("norm_linear", "linear"):
        m, k, n = c["m"], c["k"], c["n"]
        nw = 2 * n if c["act"] in GATED else n
        if op == "linear":
            s["x"] = _act(g, m, k)
            s["gs"] = _gs(s["x"])
            s["r"] = _act(g, m, n, 0.5) if c["res"] else None
            need = [m * _pad32(k) // 2, (m + 127) // 128 * 128 * ((_pad32(k) // 16 + 3) // 4 * 4)]
            s["ws"] = torch.empty(sum((b + 255) // 256 * 256 for b in need), dtype=torch.uint8, device=DEV)
        s["w"], s["wsf"], gw = _weight(g, nw, k)
        s["alpha"] = _scalar(1.0 / (s["gs"] * gw))
        s["bias"] = (0.1 * torch.randn(nw, generator=g, device=DEV)).to(torch.bfloat16) if c.get("bias") else None
        s["out"] = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    if op in ("dispatch", "combine", "moe"):
        t, h, e, topk = c["t"], c["h"], c["e"], c["topk"]
        rows = _rows(t, topk, e)
        s["ids"], s["wt"] = _routing(g, t, e, topk)
        s["offsets"] = torch.zeros(e + 1, dtype=torch.int32, device=DEV)
        s["counts"] = torch.zeros(e, dtype=torch.int32, device=DEV)
        s["dest"] = torch.zeros(t, topk, dtype=torch.int32, device=DEV)
        # as many bytes as the library's size query answers: one 32-bit count per expert and 1024 assignments
        s["sort_ws"] = torch.empty(max(16, 4 * e * ((t * topk + 1023) // 1024)), dtype=torch.uint8, device=DEV)
        if op != "combine":
            s["x"] = _act(g, t, h)
        if op == "dispatch":
            s["rows"] = torch.zeros(rows, h, dtype=torch.bfloat16, device=DEV)
        if op == "combine":
            s["offsets"], s["counts"], s["dest"] = _sorted(s["ids"], e)
            s["y"] = torch.randn(rows, h, generator=g, device=DEV).to(torch.bfloat16)
            if c["grad"]:
                s["dout"] = torch.randn(t, h, generator=g, device=DEV).to(torch.bfloat16)
                s["dy"] = torch.zeros(rows, h, dtype=torch.bfloat16, device=DEV)
                s["dw"] = torch.empty(t, topk, device=DEV)
            s["r"] = _act(g, t, h) if c["res"] else None
            s["out"] = torch.empty(t, h, dtype=torch.bfloat16, device=DEV)
        if op == "moe":
            f = c["f"]
            s["gs"] = _gs(s["x"])
            s["gs2"] = torch.full((1,), 2688.0 / 16.0, device=DEV)     # calibrated on earlier data
            s["w1"], s["w1sf"], g1 = _weight(g, e * 2 * f, h)
            s["w2"], s["w2sf"], g2 = _weight(g, e * h, f)
            s["alpha1"] = (1.0 / (s["gs"] * g1)).expand(e).contiguous()
            s["alpha2"] = (1.0 / (s["gs2"] * g2)).expand(e).contiguous()
            byte = lambda n: torch.zeros(n, dtype=torch.uint8, device=DEV)   # noqa: E731
            s["a1"], s["a1sf"] = byte(rows * _pad32(h) // 2), byte(rows * ((_pad32(h) // 16 + 3) // 4 * 4))
            s["a2"], s["a2sf"] = byte(rows * _pad32(f) // 2), byte(rows * ((_pad32(f) // 16 + 3) // 4 * 4))
            s["hid"] = torch.zeros(rows, f, dtype=torch.bfloat16, device=DEV)
            s["y"] = torch.zeros(rows, h, dtype=torch.bfloat16, device=DEV)
            s["out"] = torch.empty(t, h, dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------- plain form ----

def _sorted(ids, e):
    """(offsets [e + 1], counts [e], dest [t, topk]) of the stable sort by expert into 128-aligned groups."""
    flat = ids.reshape(-1)
    hit = (flat[None] == torch.arange(e, dtype=flat.dtype, device=flat.device)[:, None]).int()
    counts = hit.sum(1, dtype=torch.int32)
    padded = (counts + 127) // 128 * 128
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = padded.cumsum(0)
    place = (hit.cumsum(1, dtype=torch.int32) - 1 + offsets[:e, None]) * hit
    valid = (flat >= 0) & (flat < e)
    dest = torch.where(valid, place.sum(0, dtype=torch.int32), -1)
    return offsets, counts, dest.view_as(ids)


def _scatter(src, dest, rows):
    """rows[dest[t, k]] = src[t, k]; rows without a source are zero (dropped assignments go to a spare row)."""
    out = torch.zeros(rows + 1, src.shape[-1], dtype=src.dtype, device=src.device)
    out[torch.where(dest < 0, rows, dest).long()] = src
    return out[:rows]


def _activate(v, act):
    if act == "none":
        return v
    if act == "relu":
        return v.clamp_min(0.0)
    if act in GATED:
        gate, up = v[:, 0::2], v[:, 1::2]
        return _activate(gate, "silu" if act == "swiglu" else "gelu") * up
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    z = 0.7978845608028654 * (v + 0.044715 * v * v * v)
    return 0.5 * v * (1.0 + torch.tanh(z))


def _norm(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    y = h * (1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)) * s["gamma"].float()
    return (None if s["r"] is None else h.to(torch.bfloat16)), y


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        h, y = _norm(s)
        b = _widen(y, c["k"]).view(c["m"], -1, 32)
        amax = b.abs().amax(-1)
        e = torch.where(amax > 0, (torch.frexp(amax)[1] - 9).clamp(-127, 127), -127)
        q = _e4m3(torch.ldexp(b, -e[..., None])).view(c["m"], -1)
        sf = _tile((e + 127).to(torch.uint8)).view(torch.float8_e8m0fnu)
        return {"q": q, "sf": sf} if h is None else {"h": h, "q": q, "sf": sf}
    if op in ("norm_linear", "linear"):
        h, y = _norm(s) if op == "norm_linear" else (None, s["x"].float())
        q, sf = _fp4(_widen(y, c["k"]), s["gs"])
        a = (q.view(c["m"], -1, 16) * sf[..., None]).view(c["m"], -1)
        w = _dequant(s["w"], s["wsf"], s["w"].shape[0], c["k"])
        v = (a @ w.T) * s["alpha"]
        if s["bias"] is not None:
            v = v + s["bias"].float()
        v = _activate(v, c["act"])
        if op == "linear" and s["r"] is not None:
            v = v + s["r"].float()
        out = {"out": v.to(torch.bfloat16)}
        return out if h is None else dict(out, h=h)
    if op == "dispatch":
        offsets, counts, dest = _sorted(s["ids"], c["e"])
        rows = _scatter(s["x"][:, None].expand(-1, c["topk"], -1), dest, s["rows"].shape[0])
        return {"offsets": offsets, "counts": counts, "dest": dest, "rows": rows}
    if op == "combine":
        return _plain_combine(s, s["dest"], s["y"], s["r"])
    # moe
    e, f, h, topk = c["e"], c["f"], c["h"], c["topk"]
    offsets, counts, dest = _sorted(s["ids"], e)
    rows = s["y"].shape[0]
    q, sf = _fp4(_widen(s["x"], h), s["gs"])
    a = _scatter((q.view(c["t"], -1, 16) * sf[..., None]).view(c["t"], 1, -1).expand(-1, topk, -1), dest, rows)
    # the expert of each 128-row band (bands past the last group compute with the last expert: never gathered)
    band = torch.arange(0, rows, 128, device=DEV)
    expert = ((band[:, None] >= offsets[None, 1:]).sum(1)).clamp_max(e - 1)
    w1 = _dequant(s["w1"], s["w1sf"], e * 2 * f, h).view(e, 2 * f, -1)
    v = torch.bmm(a.view(rows // 128, 128, -1), w1[expert].transpose(1, 2)).view(rows, -1)
    hid = _activate(v * s["alpha1"].view(-1)[expert].repeat_interleave(128)[:, None], "swiglu").to(torch.bfloat16)
    q, sf = _fp4(_widen(hid, f), s["gs2"])
    a = (q.view(rows, -1, 16) * sf[..., None]).view(rows // 128, 128, -1)
    w2 = _dequant(s["w2"], s["w2sf"], e * h, f).view(e, h, -1)
    v = torch.bmm(a, w2[expert].transpose(1, 2)).view(rows, h)
    y = (v * s["alpha2"].view(-1)[expert].repeat_interleave(128)[:, None]).to(torch.bfloat16)
    s = dict(s, case=dict(c, weights=True, grad=False))
    return _plain_combine(s, dest, y, s["x"])


def _plain_combine(s, dest, y, res):
    c = s["case"]
    valid = (dest >= 0)[..., None]
    rows = torch.where(valid, y[dest.clamp_min(0).long()].float(), 0.0)
    if not c["grad"]:
        out = (rows * s["wt"][..., None]).sum(1) if c["weights"] else rows.sum(1)
        return {"out": (out if res is None else out + res.float()).to(torch.bfloat16)}
    d = s["dout"].float()[:, None]
    dy = _scatter((d * s["wt"][..., None]).to(torch.bfloat16), dest, y.shape[0])
    return {"dy": dy, "dw": (d * rows).sum(-1)}


# ------------------------------------------------------- framework's form ----

def _ours(s):
    import nvfp4_quantized_linear_gb300 as nv
    c, op = s["case"], s["case"]["op"]
    if op in ("norm", "norm_linear"):
        m, k = c["m"], c["k"]
        fmt = nv.NVFP4_FORMAT_MXFP8 if op == "norm" else nv.NVFP4_FORMAT_NVFP4
        nv.nvfp4_add_rmsnorm_quant(s["x"], s["x"].stride(0), s["r"], k, s["gamma"], EPS, m, k, fmt, s.get("gs"),
                                   s["h"], k, s["q"], s["sf"])
        if op == "norm":
            out = {"q": s["q"].view(torch.float8_e4m3fn), "sf": s["sf"].view(torch.float8_e8m0fnu)}
            return out if s["h"] is None else dict(out, h=s["h"])
        nv.nvfp4_gemm_act(s["q"], s["sf"], m, s["w"], s["wsf"], s["w"].shape[0], c["n"], k, s["alpha"], s["bias"],
                          nv.ACTIVATIONS[c["act"]], None, 0, s["out"], c["n"])
        return {"out": s["out"]} if s["h"] is None else {"out": s["out"], "h": s["h"]}
    if op == "linear":
        nv.nvfp4_linear_act(s["x"], c["m"], c["k"], c["k"], s["gs"], None, 0, s["w"], s["wsf"], s["w"].shape[0], c["n"],
                            s["alpha"], s["bias"], nv.ACTIVATIONS[c["act"]], s["r"], c["n"], s["out"], c["n"], s["ws"],
                            s["ws"].numel())
        return {"out": s["out"]}
    t, h, e, topk = c["t"], c["h"], c["e"], c["topk"]
    if op == "combine":
        rows = s["y"].shape[0]
        if c["grad"]:
            nv.nvfp4_moe_combine_backward(s["dout"], h, s["y"], h, s["wt"], s["dest"], t, topk, rows, h, s["offsets"],
                                          s["counts"], e, s["dy"], h, s["dw"])
            return {"dy": s["dy"], "dw": s["dw"]}
        nv.nvfp4_moe_combine(s["y"], h, s["wt"] if c["weights"] else None, s["dest"], t, topk, rows, h, s["r"], h,
                             s["out"], h)
        return {"out": s["out"]}
    nv.nvfp4_moe_sort(s["ids"], 4, t, topk, e, s["offsets"], s["counts"], s["dest"], s["sort_ws"],
                      s["sort_ws"].numel())
    if op == "dispatch":
        nv.nvfp4_moe_dispatch(s["x"], h, s["dest"], t, topk, s["rows"].shape[0], h, s["offsets"], s["counts"], e,
                              s["rows"], h)
        return {"offsets": s["offsets"], "counts": s["counts"], "dest": s["dest"], "rows": s["rows"]}
    f, rows = c["f"], s["y"].shape[0]
    nv.nvfp4_moe_dispatch_quant(s["x"], h, s["gs"], s["dest"], t, topk, rows, h, s["a1"], s["a1sf"])
    nv.nvfp4_grouped_gemm_act(s["a1"], s["a1sf"], rows, s["offsets"], e, s["w1"], s["w1sf"], f, h, s["alpha1"], None,
                              nv.ACTIVATIONS["swiglu"], s["hid"], f)
    nv.nvfp4_quant_act(s["hid"], rows, f, f, s["gs2"], None, 0, s["a2"], s["a2sf"])
    nv.nvfp4_grouped_gemm(s["a2"], s["a2sf"], rows, s["offsets"], e, s["w2"], s["w2sf"], h, f, s["alpha2"], None,
                          s["y"], h)
    nv.nvfp4_moe_combine(s["y"], h, s["wt"], s["dest"], t, topk, rows, h, s["x"], h, s["out"], h)
    return {"out": s["out"]}


def run(state):
    return _ours(state) if own else _plain(state)


# ------------------------------------------------------------------- work ----

def work(case):
    c, op = case, case["op"]
    if op in ("norm", "norm_linear"):
        m, k = c["m"], c["k"]
        b = m * k * (2 + (4 if c["res"] else 0)) + 2 * k
        if op == "norm":
            return {"bytes": b + m * k + m * k // 32, "flops": 8 * m * k}
        nw = 2 * c["n"] if c["act"] in GATED else c["n"]
        return {"bytes": b + nw * k * 9 // 16 + 2 * m * c["n"], "flops": 2 * m * nw * k}
    if op == "linear":
        m, k, n = c["m"], c["k"], c["n"]
        nw = 2 * n if c["act"] in GATED else n
        b = 2 * m * k + nw * k * 9 // 16 + m * n * (4 if c["res"] else 2) + (2 * nw if c["bias"] else 0)
        return {"bytes": b, "flops": 2 * m * nw * k}
    t, h, e, topk = c["t"], c["h"], c["e"], c["topk"]
    n = t * topk
    if op == "dispatch":
        return {"bytes": 2 * t * h + 2 * n * h + 8 * n, "flops": 0}
    if op == "combine":
        if c["grad"]:
            return {"bytes": 2 * t * h + 4 * n * h + 12 * n, "flops": 3 * n * h}
        return {"bytes": 2 * n * h + t * h * (4 if c["res"] else 2) + (8 if c["weights"] else 4) * n, "flops": 2 * n * h}
    w = min(e, n) * (2 * c["f"] * h + h * c["f"]) * 9 // 16
    return {"bytes": w + 6 * t * h, "flops": 2 * n * 3 * c["f"] * h}


# ------------------------------------------------------------------ exact ----
# From the definitions in 64 bits, on other routes than above: rounding by exponent arithmetic, sorting by a
# stable argsort, codes unpacked through shifts.

def _x_round(v, step):
    return torch.round(v / step) * step


def _x_e4m3(v):
    a = v.abs().clamp_max(1e30)
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -6)))
    return torch.sign(v) * _x_round(a, torch.exp2(e - 3)).clamp_max(448.0)


def _x_e2m1(v):
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    return torch.sign(v) * _x_round(a, step).clamp_max(6.0)


def _x_nvfp4(v, gs):
    """Values on the NVFP4 grid of [rows, k], still times the global scale."""
    k = v.shape[1]
    b = torch.nn.functional.pad(v, (0, _pad32(k) - k)).reshape(v.shape[0], -1, 16)
    f32 = lambda t: t.float().double()   # noqa: E731  (the format defines these steps in fp32)
    sf = _x_e4m3(f32(f32(b.abs().amax(2) * gs) / 6.0))[..., None]
    q = _x_e2m1(f32(b * torch.where(sf > 0, f32(gs / sf.clamp_min(1e-30)), 0.0)))
    return (q * sf).reshape(v.shape[0], -1)


def _x_weight(packed, sf, n, k):
    """[n, kp] doubles of a packed weight, scales read through the tiled offset formula."""
    kp = _pad32(k)
    cols = (kp // 16 + 3) // 4 * 4
    r = torch.arange(n, device=DEV)[:, None]
    j = torch.arange(kp // 16, device=DEV)[None]
    off = ((r // 128) * (cols // 4) + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
    raw = sf[off].int()
    scale = torch.where(raw >= 8, (8.0 + raw % 8).double() * torch.exp2((raw // 8 - 10).double()), raw * 2.0 ** -9)
    nib = torch.stack((packed % 16, packed // 16), 2).reshape(n, kp).int()
    mag = nib % 8
    val = torch.where(mag < 2, mag * 0.5, (2.0 + mag % 2).double() * torch.exp2((mag // 2 - 2).double()))
    val = torch.where(nib >= 8, -val, val.double())
    return (val.reshape(n, -1, 16) * scale[..., None]).reshape(n, kp)


def _x_activate(v, act):
    if act in GATED:
        return _x_activate(v[:, ::2], "silu" if act == "swiglu" else "gelu") * v[:, 1::2]
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    return torch.relu(v) if act == "relu" else v


def _x_norm(s):
    h = s["x"].double() + (s["r"].double() if s["r"] is not None else 0.0)
    y = h * torch.rsqrt(h.square().mean(1) + EPS)[:, None] * s["gamma"].double()
    return (None if s["r"] is None else h), y


def _x_dest(ids, e):
    """Rows of the assignments by a stable argsort; None where one is dropped is -1."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= e), e, flat)
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=e + 1)[:e]
    start = torch.cumsum((counts + 127) // 128 * 128, 0) - (counts + 127) // 128 * 128
    first = torch.cumsum(counts, 0) - counts
    k = key[order]
    kk = k.clamp_max(e - 1)
    row = torch.where(k < e, torch.arange(k.numel(), device=DEV) - first[kk] + start[kk], -1)
    dest = torch.empty_like(row)
    dest[order] = row
    return dest.view_as(ids), start, counts


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "norm":
        h, y = _x_norm(s)
        kp = _pad32(c["k"])
        b = torch.nn.functional.pad(y, (0, kp - c["k"])).reshape(c["m"], -1, 32)
        amax = b.abs().amax(2)
        e = torch.where(amax > 0, torch.floor(torch.log2(amax.clamp_min(1e-300))) - 8.0, -127.0).clamp(-127, 127)
        q = _x_e4m3(b * torch.exp2(-e)[..., None]).reshape(c["m"], kp)
        scale = torch.full(((c["m"] + 127) // 128 * 128, (kp // 32 + 3) // 4 * 4), 2.0 ** -127, dtype=torch.float64,
                           device=DEV)
        scale[:c["m"], :kp // 32] = torch.exp2(e)
        sf = scale.reshape(scale.shape[0] // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).reshape(-1)
        return {"q": q, "sf": sf} if h is None else {"h": h, "q": q, "sf": sf}
    if op in ("norm_linear", "linear"):
        nw = s["w"].shape[0]
        if 2 * c["m"] * nw * c["k"] > 4e12:
            return None
        h, y = _x_norm(s) if op == "norm_linear" else (None, s["x"].double())
        v = _x_nvfp4(y, s["gs"].double()) @ _x_weight(s["w"], s["wsf"], nw, c["k"]).T * s["alpha"].double()
        if s["bias"] is not None:
            v = v + s["bias"].double()
        v = _x_activate(v, c["act"])
        if op == "linear" and s["r"] is not None:
            v = v + s["r"].double()
        return {"out": v} if h is None else {"out": v, "h": h}
    if op == "dispatch":
        dest, _, _ = _x_dest(s["ids"], c["e"])
        rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device=DEV)
        at, src = dest.reshape(-1), torch.arange(c["t"], device=DEV).repeat_interleave(c["topk"])
        rows[at[at >= 0]] = s["x"].double()[src[at >= 0]]
        return {"offsets": None, "counts": None, "dest": None, "rows": rows}
    if op == "combine":
        if c["grad"]:
            dy = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
            dw = torch.zeros(c["t"], c["topk"], dtype=torch.float64, device=DEV)
            for j in range(c["topk"]):
                at = (s["dest"][:, j] >= 0).nonzero()[:, 0]
                row, d = s["dest"][at, j].long(), s["dout"][at].double()
                dy[row] = d * s["wt"][at, j].double()[:, None]
                dw[at, j] = (d * s["y"][row].double()).sum(1)
            return {"dy": dy, "dw": dw}
        return {"out": _x_combine(s, s["dest"], s["y"].double(), s["r"], c["weights"])}
    dest, start, counts = _x_dest(s["ids"], c["e"])
    f, h = c["f"], c["h"]
    q = _x_nvfp4(s["x"].double(), s["gs"].double())
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    w1 = _x_weight(s["w1"], s["w1sf"], c["e"] * 2 * f, h).view(c["e"], 2 * f, -1)
    w2 = _x_weight(s["w2"], s["w2sf"], c["e"] * h, f).view(c["e"], h, -1)
    for i in range(c["e"]):
        tok = (s["ids"] == i).nonzero()[:, 0]
        if tok.numel():
            a = _x_activate(q[tok] @ w1[i].T * s["alpha1"][i].double(), "swiglu")
            a = _x_nvfp4(a.to(torch.bfloat16).double(), s["gs2"].double())
            y[int(start[i]):int(start[i]) + tok.numel()] = a @ w2[i].T * s["alpha2"][i].double()
    return {"out": _x_combine(s, dest, y, s["x"], True)}


def _x_combine(s, dest, y, res, weights):
    out = torch.zeros(dest.shape[0], y.shape[1], dtype=torch.float64, device=DEV)
    tok, j = (dest >= 0).nonzero(as_tuple=True)
    w = s["wt"][tok, j].double()[:, None] if weights else 1.0
    out.index_add_(0, tok, y[dest[tok, j].long()] * w)
    return out if res is None else out + res.double()
