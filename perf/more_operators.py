"""Routing to experts, 8-bit activation checkpoints and the gradients that use them, as cases to measure.

Five kinds of case (``op``):

  route       router logits -> expert ids and weights (softmax or sigmoid, bias, groups, top-k, renormalised)
  route_grad  gradient of the routing weights -> gradient of the logits
  ckpt        a GEMM's output -> its activation in bf16, and the output itself kept in MXFP8
  ckpt_grad   gradient of the activation from the MXFP8 checkpoint, and the activation again in MXFP8
  wgrad       weight gradient dY^T X with X in MXFP8, of one weight or of every expert's

``run`` has two forms over the same state: ``own`` False is elementary torch, ``own`` True the calls of
``nvfp4_quantized_linear_gb300``.  With ``e`` > 0 the rows of ckpt, ckpt_grad and wgrad are the sorted rows of a
mixture-of-experts layer: groups padded to 128 rows, whose padding rows nobody reads.
"""
import math

import torch

own = False

DEV = "cuda"
GATED = ("swiglu", "geglu")
FLT_MAX = 3.4028234663852886e38


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one decoded token: pure latency
        dict(name="route_token", op="route", t=1, e=128, topk=8, score="softmax", bf16=False, bias=False, groups=1,
             group_top=1, topk_groups=1, renorm=True, scale=1.0),
        # a long prompt through a softmax router
        dict(name="route_prompt", op="route", t=16384, e=128, topk=8, score="softmax", bf16=True, bias=False, groups=1,
             group_top=1, topk_groups=1, renorm=True, scale=1.0),
        # sigmoid scores with a balance bias, half of the expert groups, an odd number of tokens
        dict(name="route_groups", op="route", t=4099, e=256, topk=8, score="sigmoid", bf16=False, bias=True, groups=8,
             group_top=2, topk_groups=4, renorm=True, scale=2.5),
        # the same prompt's gradient in training: only chosen experts have one
        dict(name="route_grad_prompt", op="route_grad", t=16384, e=128, topk=8, score="softmax", bf16=True, renorm=True,
             scale=1.0),
        # weights not renormalised: every expert of a row has a gradient; a ragged batch
        dict(name="route_grad_ragged", op="route_grad", t=1003, e=40, topk=6, score="softmax", bf16=False, renorm=False,
             scale=1.0),
        # the MLP of an encoder-style block, columns that end inside a block of 32
        dict(name="ckpt_ragged", op="ckpt", m=333, n=2072, act="gelu", e=0, topk=0),
        # a training batch's gate/up projection
        dict(name="ckpt_prompt", op="ckpt", m=8192, n=14336, act="swiglu", e=0, topk=0),
        # the expert rows of 2048 tokens
        dict(name="ckpt_grad_moe", op="ckpt_grad", m=2048, n=768, act="swiglu", e=32, topk=4),
        # a training batch, with the next weight gradient's operand
        dict(name="ckpt_grad_prompt", op="ckpt_grad", m=8192, n=14336, act="swiglu", e=0, topk=0),
        # a small weight's gradient over a ragged batch
        dict(name="wgrad_ragged", op="wgrad", m=333, n=2072, k=4104, f32=False, e=0, topk=0),
        # the gate/up weight's gradient over a training batch
        dict(name="wgrad_prompt", op="wgrad", m=8192, n=28672, k=4096, f32=False, e=0, topk=0),
        # every expert's gate/up weight in fp32
        dict(name="wgrad_moe", op="wgrad", m=8192, n=1536, k=2048, f32=True, e=32, topk=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges."""
    op = rng.choice(["route", "route_grad", "ckpt", "ckpt_grad", "wgrad"])
    if op in ("route", "route_grad"):
        e = _log(rng, 4, 512)
        t = min(_log(rng, 1, 16384), 16384 * 128 // e)
        c = dict(op=op, t=t, e=e, topk=rng.randint(1, min(8, e)), score=rng.choice(["softmax", "sigmoid"]),
                 bf16=rng.random() < 0.5, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))
        if op == "route_grad":
            return c
        groups = rng.choice([g for g in (1, 2, 4, 8) if e % g == 0 and e >= 4 * g])
        kept = rng.randint(1, groups)
        return dict(c, topk=min(c["topk"], e // groups * kept), bias=rng.random() < 0.5, groups=groups,
                    group_top=rng.randint(1, 2), topk_groups=kept)
    e = _log(rng, 4, 64) if rng.random() < 0.4 else 0
    topk = rng.randint(1, 4) if e else 0
    if op == "wgrad":
        if e:
            return dict(op=op, m=_log(rng, 1, 8192), n=128 * rng.randint(1, 12), k=rng.randint(64, 2048),
                        f32=rng.random() < 0.5, e=min(e, 32), topk=topk)
        c = dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 64, 28672), k=_log(rng, 64, 14336), f32=rng.random() < 0.5,
                 e=0, topk=0)
        while c["n"] * c["k"] > 28672 * 4096:
            c["n"] = c["n"] // 2 + 1
        return c
    c = dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 64, 14336),
             act=rng.choice(["relu", "gelu", "silu", "swiglu", "geglu"]), e=e, topk=topk)
    while e and (c["m"] * topk + 127 * e) * c["n"] > 4096 * 14336:
        c["n"] = c["n"] // 2 + 1
    return c


# -------------------------------------------------- formats (plain torch) ----

def _up(v, to):
    return (v + to - 1) // to * to


def _rows(c):
    """Rows of the operands: m, or those of a dispatched operand whatever the routing."""
    n = c["m"] * c["topk"]
    return (n + 127 * min(c["e"], n)) // 128 * 128 if c["e"] else c["m"]


def _tile(codes):
    """[rows, cols] scale bytes -> 512-byte tiles of 128 rows x 4 columns (zero padding), flat."""
    r, c = codes.shape
    full = torch.zeros(_up(r, 128), _up(c, 4), dtype=codes.dtype, device=codes.device)
    full[:r, :c] = codes
    return full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile(flat, r, c):
    rp, cp = _up(r, 128), _up(c, 4)
    return flat.view(rp // 128, cp // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rp, cp)[:r, :c]


def _mxfp8(v):
    """E4M3 codes [rows, kp] and E8M0 scale bytes [rows, kp / 32] of fp32 values."""
    b = torch.nn.functional.pad(v, (0, -v.shape[1] % 32)).view(v.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 9).clamp(-127, 127), -127)
    # (2^-e in two factors: one of them alone leaves fp32 for the largest and the smallest blocks)
    half = torch.div(-e, 2, rounding_mode="floor")
    q = torch.ldexp(torch.ldexp(b, half[..., None]), (-e - half)[..., None])
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(v.shape[0], -1), (e + 127).to(torch.uint8)


def _values(q, sf, k):
    """fp32 values of an MXFP8 operand with tiled scales."""
    r, kp = q.shape
    e = _untile(sf, r, kp // 32).int() - 127
    return torch.ldexp(q.view(torch.float8_e4m3fn).float().view(r, -1, 32), e[..., None]).view(r, kp)[:, :k]


# ---------------------------------------------------------------- prepare ----

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _act(g, m, k, std=1.0):
    """bf16 values with a few large channels, as hidden states have; rows on 16-byte boundaries."""
    x = torch.randn(m, _up(k, 8), generator=g, device=DEV) * std
    x[:, torch.randint(0, k, (max(1, k // 1000),), generator=g, device=DEV)] *= 20.0
    return x.to(torch.bfloat16)[:, :k]


def _groups(g, c):
    """Offsets and counts of a skewed routing (some experts busy, some empty), and which rows are real."""
    logits = torch.randn(c["m"], c["e"], generator=g, device=DEV) + torch.randn(1, c["e"], generator=g, device=DEV)
    ids = logits.topk(min(c["topk"], c["e"]), dim=1)[1]
    counts = (ids.reshape(-1)[None] == torch.arange(c["e"], device=DEV)[:, None]).sum(1).int()
    offsets = torch.zeros(c["e"] + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = ((counts + 127) // 128 * 128).cumsum(0)
    return offsets, counts


def _columns(c):
    """Columns of the pre-activation."""
    return 2 * c["n"] if c["act"] in GATED else c["n"]


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    s = {"case": dict(case)}
    if op in ("route", "route_grad"):
        t, e, topk = c["t"], c["e"], c["topk"]
        # router logits of a batch with a little padding: a padded token's row is masked whole
        l = 1.5 * torch.randn(t, e, generator=g, device=DEV) + 0.5 * torch.randn(1, e, generator=g, device=DEV)
        if t > 64:
            l[torch.rand(t, generator=g, device=DEV) < 0.01] = -math.inf
        s["logits"] = l.to(torch.bfloat16) if c["bf16"] else l
        if op == "route":
            s["bias"] = 0.1 * torch.randn(e, generator=g, device=DEV) if c["bias"] else None
            s["ids"] = torch.empty(t, topk, dtype=torch.int32, device=DEV)
            s["weights"] = torch.empty(t, topk, device=DEV)
        else:
            top, ids = s["logits"].float().sort(dim=1, descending=True, stable=True)
            s["ids"] = torch.where(top > -math.inf, ids, -1)[:, :topk].to(torch.int32).contiguous()
            s["dw"] = torch.randn(t, topk, generator=g, device=DEV)
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    rows = _rows(c)
    s["offsets"], s["counts"] = _groups(g, c) if c["e"] else (None, None)
    byte = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=DEV)   # noqa: E731
    if op == "wgrad":
        n, k = c["n"], c["k"]
        q, sf = _mxfp8(_act(g, rows, k).float())
        s["q"], s["sf"] = q.view(torch.uint8), _tile(sf)
        # rows of a gradient; padding rows are zero, as the kernels that make them leave them
        s["dy"] = _act(g, rows, n, 0.01)
        if c["e"]:
            s["dy"].mul_(_real(s)[:, None])
        # as the library's size query answers: sums of row ranges where one weight has few tiles
        s["out"] = torch.empty(max(1, c["e"]) * n, _up(k, 8), dtype=torch.float32 if c["f32"] else torch.bfloat16, device=DEV)
        s["ws"] = torch.empty(_workspace(c), dtype=torch.uint8, device=DEV)
        return s
    n, k = c["n"], _columns(c)
    if op == "ckpt":
        s["x"] = _act(g, rows, k)
        s["q"], s["sf"] = byte(rows, _up(k, 32)), byte(_up(rows, 128) * _up(_up(k, 32) // 32, 4))
        s["out"] = torch.zeros(rows, _up(n, 8), dtype=torch.bfloat16, device=DEV)[:, :n]
        return s
    q, sf = _mxfp8(_act(g, rows, k).float())
    s["q"], s["sf"] = q.view(torch.uint8), _tile(sf)
    s["dout"] = _act(g, rows, n, 0.01)
    s["dx"] = torch.zeros(rows, _up(k, 8), dtype=torch.bfloat16, device=DEV)[:, :k]
    s["hq"], s["hsf"] = byte(rows, _up(n, 32)), byte(_up(rows, 128) * _up(_up(n, 32) // 32, 4))
    return s


def _workspace(c):
    """At most eight fp32 copies of a weight of up to 76 tiles of 256 x 256."""
    tiles = ((c["n"] + 255) // 256) * ((c["k"] + 255) // 256)
    return 16 if c["e"] or tiles > 76 else 8 * tiles * 256 * 256 * 4


# ------------------------------------------------------------- plain form ----

def _real(s):
    """Truth value per row of a dispatched operand: whether a token stands there."""
    r = torch.arange(_rows(s["case"]), device=DEV)
    e = (r[:, None] >= s["offsets"][None, 1:]).sum(1)
    return (e < s["case"]["e"]) & (r < (s["offsets"][:-1] + s["counts"])[e.clamp_max(s["case"]["e"] - 1)])


def _softmax_of(l, over):
    """exp(l - m) / sum over the last axis of `over`'s, 0 in rows where nothing is left."""
    m = over.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    z = torch.exp(over - m).sum(-1, keepdim=True)
    return torch.exp(l - m) / torch.where(z > 0, z, 1.0)


def _sigmoid(l):
    return 1.0 / (1.0 + torch.exp(-l))


def _clean(logits, dtype):
    l = logits.to(dtype)
    return torch.where(l > -math.inf, l, -math.inf).clamp_max(FLT_MAX)


def _chosen(s):
    """Expert ids [t, topk] in descending order of their keys, ties to the lowest index, -1 where none is left."""
    c = s["case"]
    l = _clean(s["logits"], torch.float64)
    score = _softmax_of(l, l) if c["score"] == "softmax" else _sigmoid(l)
    key = l if s["bias"] is None else torch.where(l > -math.inf, score + s["bias"].double(), -math.inf)
    if c["groups"] > 1:
        by = key if c["group_top"] == 1 or s["bias"] is not None else torch.where(l > -math.inf, score, -math.inf)
        top = by.view(c["t"], c["groups"], -1).sort(dim=2, descending=True)[0][..., :c["group_top"]]
        value = torch.where(top > -math.inf, top, 0.0).sum(2)
        value = torch.where(top[..., 0] > -math.inf, value, -math.inf)
        order = value.sort(dim=1, descending=True, stable=True)[1]
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order[:, :c["topk_groups"]], True)
        key = torch.where(kept.repeat_interleave(c["e"] // c["groups"], 1), key, -math.inf)
    top, ids = key.sort(dim=1, descending=True, stable=True)
    return torch.where(top > -math.inf, ids, -1)[:, :c["topk"]]


def _activate(v, act):
    """act(v) and act'(v)."""
    if act == "relu":
        return v.clamp_min(0.0), (v > 0).to(v.dtype)
    if act == "silu":
        sg = _sigmoid(v)
        return v * sg, sg * (1.0 + v * (1.0 - sg))
    a = 1.5957691216057308                                   # 2 sqrt(2 / pi): gelu(v) = v sigmoid(u)
    sg = _sigmoid(a * (v + 0.044715 * v * v * v))
    return v * sg, sg + v * sg * (1.0 - sg) * a * (1.0 + 0.134145 * v * v)


def _forward(v, act):
    if act in GATED:
        return _activate(v[:, 0::2], "silu" if act == "swiglu" else "gelu")[0] * v[:, 1::2]
    return _activate(v, act)[0]


def _backward(v, d, act):
    if act in GATED:
        a, da = _activate(v[:, 0::2], "silu" if act == "swiglu" else "gelu")
        return torch.stack((d * v[:, 1::2] * da, d * a), 2).flatten(1)
    return d * _activate(v, act)[1]


def _fp8(q, sf):
    return {"q": q.view(torch.float8_e4m3fn), "sf": sf.view(torch.float8_e8m0fnu)}


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "route":
        ids = _chosen(s)
        l = _clean(s["logits"], torch.float32)
        at = torch.where(ids >= 0, l.gather(1, ids.clamp_min(0)), -math.inf)
        if c["score"] == "softmax":
            w = _softmax_of(at, at if c["renorm"] else l)
        else:
            w = torch.where(ids >= 0, _sigmoid(at), 0.0)
            if c["renorm"]:
                w = w / torch.where(w > 0, w, 0.0).sum(1, keepdim=True).clamp_min(1e-30)
        return {"ids": ids.to(torch.int32), "weights": w * c["scale"]}
    if op == "route_grad":
        l, have = _clean(s["logits"], torch.float32), s["ids"] >= 0
        ids = s["ids"].long().clamp_min(0)
        at = torch.where(have, l.gather(1, ids), -math.inf)
        g = torch.where(have, s["dw"] * c["scale"], 0.0)
        sg = torch.where(have, _sigmoid(at), 0.0)
        if c["renorm"]:
            u = _softmax_of(at, at) if c["score"] == "softmax" else sg / sg.sum(1, keepdim=True).clamp_min(1e-30)
            d = u * (g - (u * g).sum(1, keepdim=True))
            d = d if c["score"] == "softmax" else d * (1.0 - sg)
        elif c["score"] == "sigmoid":
            d = g * sg * (1.0 - sg)
        else:
            p = _softmax_of(l, l)
            dense = torch.zeros_like(p).scatter_add_(1, ids, g)
            return {"dlogits": (p * (dense - (p * dense).sum(1, keepdim=True))).to(s["logits"].dtype)}
        return {"dlogits": torch.zeros_like(l).scatter_add_(1, ids, d).to(s["logits"].dtype)}
    rows = _rows(c)
    real = _real(s)[:, None] if c["e"] else torch.ones(rows, 1, dtype=torch.bool, device=DEV)
    if op == "ckpt":
        v = s["x"].float()
        q, sf = _mxfp8(v)
        out = torch.where(real, _forward(v, c["act"]).to(torch.bfloat16), 0.0)
        return dict(_fp8(q.view(torch.uint8) * real, _tile(sf * real)), out=out)
    if op == "ckpt_grad":
        v = _values(s["q"], s["sf"], _columns(c))
        q, sf = _mxfp8(_forward(v, c["act"]))
        dx = torch.where(real, _backward(v, s["dout"].float(), c["act"]).to(torch.bfloat16), 0.0)
        return dict(_fp8(q.view(torch.uint8) * real, _tile(sf * real)), dx=dx)
    x = torch.where(real, _values(s["q"], s["sf"], c["k"]), 0.0)
    dy = torch.where(real, s["dy"].float(), 0.0)
    if not c["e"]:
        return {"dw": (dy.T @ x).to(s["out"].dtype)}
    # 128-row bands, then the bands of each expert (bands past the last group belong to none)
    bands = rows // 128
    part = torch.bmm(dy.view(bands, 128, -1).transpose(1, 2), x.view(bands, 128, -1))
    first = torch.arange(0, rows, 128, device=DEV)[None]
    mine = (first >= s["offsets"][:-1, None]) & (first < s["offsets"][1:, None])
    return {"dw": (mine.float() @ part.view(bands, -1)).to(s["out"].dtype).view(c["e"] * c["n"], -1)}


# ------------------------------------------------------- framework's form ----

def _ours(s):
    import nvfp4_quantized_linear_gb300 as nv
    c, op = s["case"], s["case"]["op"]
    if op in ("route", "route_grad"):
        kind, score = nv.NVFP4_TYPE_BF16 if c["bf16"] else nv.NVFP4_TYPE_F32, nv.SCORES[c["score"]]
        if op == "route":
            nv.nvfp4_moe_route(s["logits"], kind, c["e"], s["bias"], c["t"], c["e"], score, c["topk"], c["groups"],
                               c["group_top"], c["topk_groups"], c["renorm"], c["scale"], s["ids"], s["weights"])
            return {"ids": s["ids"], "weights": s["weights"]}
        nv.nvfp4_moe_route_backward(s["dw"], s["ids"], s["logits"], kind, c["e"], c["t"], c["e"], score, c["topk"],
                                    c["renorm"], c["scale"], s["dlogits"], c["e"])
        return {"dlogits": s["dlogits"]}
    rows, e = _rows(c), c["e"]
    if op == "ckpt":
        nv.nvfp4_act_checkpoint(s["x"], s["x"].stride(0), rows, c["n"], nv.ACTIVATIONS[c["act"]], s["offsets"], s["counts"],
                                e, s["out"], s["out"].stride(0), s["q"], s["sf"])
        return dict(_fp8(s["q"], s["sf"]), out=s["out"])
    if op == "ckpt_grad":
        nv.nvfp4_act_checkpoint_backward(s["dout"], s["dout"].stride(0), s["q"], s["sf"], rows, c["n"],
                                         nv.ACTIVATIONS[c["act"]], s["offsets"], s["counts"], e, s["dx"],
                                         s["dx"].stride(0), s["hq"], s["hsf"])
        return dict(_fp8(s["hq"], s["hsf"]), dx=s["dx"])
    kind = nv.NVFP4_TYPE_F32 if c["f32"] else nv.NVFP4_TYPE_BF16
    nv.nvfp4_checkpoint_wgrad(s["dy"], s["dy"].stride(0), s["q"], s["sf"], rows, c["n"], c["k"], s["offsets"], s["counts"],
                              e, kind, False, s["out"], s["out"].stride(0), s["ws"], s["ws"].numel())
    return {"dw": s["out"][:, :c["k"]]}


def run(state):
    return _ours(state) if own else _plain(state)


# ------------------------------------------------------------------- work ----

def work(case):
    c, op = case, case["op"]
    if op in ("route", "route_grad"):
        size, n = (2 if c["bf16"] else 4), c["t"] * c["topk"]
        row = c["t"] * c["e"] * size
        if op == "route":
            return {"bytes": row + 8 * n, "flops": 5 * c["t"] * c["e"]}
        dense = not c["renorm"] and c["score"] == "softmax"
        return {"bytes": row + (row if dense else n * size) + 8 * n, "flops": 5 * (c["t"] * c["e"] if dense else n)}
    r = c["m"] * min(c["topk"], c["e"]) if c["e"] else c["m"]
    if op == "wgrad":
        n, k = c["n"], c["k"]
        return {"bytes": 2 * r * n + r * k * 33 // 32 + max(1, c["e"]) * n * k * (4 if c["f32"] else 2), "flops": 2 * r * n * k}
    n, k = c["n"], _columns(c)
    if op == "ckpt":
        return {"bytes": r * (2 * k + 2 * n + k * 33 // 32), "flops": 10 * r * k}
    return {"bytes": r * (2 * n + k * 33 // 32 + 2 * k + n * 33 // 32), "flops": 20 * r * k}


# ------------------------------------------------------------------ exact ----
# From the definitions in 64 bits, on other routes than above: experts picked by rank, formats by exponent
# arithmetic, scales read through the tiled offset formula, weight gradients expert by expert.

def _x_pick(key, count):
    """The `count` best of the last axis, by how many are better: [.., count] indices, -1 where none is left."""
    i = torch.arange(key.shape[-1], device=DEV)
    mine, other = key[..., :, None], key[..., None, :]
    rank = ((other > mine) | ((other == mine) & (i[None, :] < i[:, None]))).sum(-1)
    at = torch.full_like(rank, -1).scatter_(-1, rank, torch.where(key > -math.inf, i, -1))
    return at[..., :count]


def _x_logits(s):
    l = s["logits"].double()
    return torch.where(torch.isnan(l), -math.inf, l).clamp(max=FLT_MAX)


def _x_scores(l, score):
    return torch.nan_to_num(torch.softmax(l, 1)) if score == "softmax" else torch.sigmoid(l)


def _x_weights(l, ids, c):
    """Weights of the chosen, and their probabilities where renormalised (a softmax over the chosen, or shares)."""
    s = _x_scores(l, c["score"])
    w = torch.where(ids >= 0, s.gather(1, ids.clamp_min(0)), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return w


def _x_values(q, sf, k):
    """[rows, k] doubles of an MXFP8 operand."""
    r, kp = q.shape
    cols = _up(kp // 32, 4)
    i, j = torch.arange(r, device=DEV)[:, None], torch.arange(kp // 32, device=DEV)[None]
    off = (i // 128 * (cols // 4) + j // 4) * 512 + i % 32 * 16 + i % 128 // 32 * 4 + j % 4
    scale = torch.exp2(sf[off].double() - 127.0)
    mag = (q % 128).int()
    v = torch.where(mag < 8, mag * 2.0 ** -9, (8.0 + mag % 8).double() * torch.exp2((mag // 8 - 10).double()))
    v = torch.where(q >= 128, -v, v)
    return (v.view(r, -1, 32) * scale[..., None]).view(r, kp)[:, :k]


def _x_exponent(a):
    """floor(log2 a) of positive doubles (a logarithm next to a whole number may fall on its other side)."""
    e = torch.round(torch.log2(a))
    return torch.where(torch.exp2(e) > a, e - 1.0, e)


def _x_mxfp8(v):
    """Values of the codes [rows, kp], and of the scales in their tiled order."""
    r, kp = v.shape[0], _up(v.shape[1], 32)
    b = torch.nn.functional.pad(v, (0, kp - v.shape[1])).view(r, -1, 32)
    amax = b.abs().amax(2)
    e = torch.where(amax > 0, _x_exponent(amax.clamp_min(1e-300)) - 8.0, -127.0).clamp(-127, 127)
    a = (b * torch.exp2(-e)[..., None]).abs()
    step = torch.exp2(_x_exponent(a.clamp_min(2.0 ** -6)) - 3.0)
    q = torch.sign(b) * (torch.round(a / step) * step).clamp_max(448.0)
    return q.view(r, kp), torch.exp2(e)


def _x_spread(sf, real):
    """The tiled order of [rows, cols] scale values; 2^-127 where nothing is written."""
    r, k = sf.shape
    full = torch.full((_up(r, 128), _up(k, 4)), 2.0 ** -127, dtype=torch.float64, device=DEV)
    full[:r, :k] = torch.where(real, sf, 2.0 ** -127)
    return full.reshape(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _x_act(v, act):
    """act(v) and its derivative."""
    if act == "relu":
        return torch.relu(v), (v > 0).double()
    b = 1.0 if act == "silu" else 2.0 * math.sqrt(2.0 / math.pi)
    cube = 0.0 if act == "silu" else 0.044715
    u, du = b * (v + cube * v ** 3), b * (1.0 + 3.0 * cube * v ** 2)
    sg = torch.sigmoid(u)
    return v * sg, sg + v * du * sg * torch.sigmoid(-u)


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "route":
        l = _x_logits(s)
        key = l
        if s["bias"] is not None:
            key = torch.where(l > -math.inf, _x_scores(l, c["score"]) + s["bias"].double(), -math.inf)
        if c["groups"] > 1:
            by = key
            if c["group_top"] == 2 and s["bias"] is None:
                by = torch.where(l > -math.inf, _x_scores(l, c["score"]), -math.inf)
            by = by.reshape(c["t"], c["groups"], -1)
            top = by.topk(min(c["group_top"], by.shape[2]), 2)[0]
            value = torch.where(top[..., 0] > -math.inf, top.clamp_min(-1e300).where(top > -math.inf, 0.0).sum(2), -math.inf)
            kept = _x_pick(value, c["topk_groups"])
            group = torch.arange(c["e"], device=DEV) // (c["e"] // c["groups"])
            key = torch.where((kept[:, :, None] == group[None, None]).any(1), key, -math.inf)
        return {"ids": None, "weights": c["scale"] * _x_weights(l, _x_pick(key, c["topk"]), c)}
    if op == "route_grad":
        l, ids = _x_logits(s), s["ids"].long()
        w, have = _x_weights(l, ids, c), ids >= 0
        g = torch.where(have, c["scale"] * s["dw"].double(), 0.0)
        sg = _x_scores(l, c["score"])
        if c["renorm"]:                                      # the Jacobian of shares, then of the score's logarithm
            d = w * g - w * (w * g).sum(1, keepdim=True)
            if c["score"] == "sigmoid":
                d = d * torch.sigmoid(-l.gather(1, ids.clamp_min(0)))
            d = torch.where(have, d, 0.0)
        elif c["score"] == "sigmoid":
            at = l.gather(1, ids.clamp_min(0))
            d = torch.where(have, g * torch.sigmoid(at) * torch.sigmoid(-at), 0.0)
        else:
            d = torch.where(have, g * w, 0.0)
        out = torch.zeros_like(l)
        for j in range(c["topk"]):
            out.scatter_add_(1, ids[:, j:j + 1].clamp_min(0), d[:, j:j + 1])
        if not c["renorm"] and c["score"] == "softmax":
            out = out - sg * d.sum(1, keepdim=True)
        return {"dlogits": out}
    rows = _rows(c)
    real = torch.ones(rows, dtype=torch.bool, device=DEV)
    if c["e"]:
        real[:] = False
        for o, k in zip(s["offsets"].tolist(), s["counts"].tolist()):
            real[o:o + k] = True
    real = real[:, None]
    if op == "wgrad":
        if 2 * rows * c["n"] * c["k"] > 4e12:
            return None
        x, dy = _x_values(s["q"], s["sf"], c["k"]), s["dy"].double()
        if not c["e"]:
            return {"dw": torch.matmul(x.T, dy).T.contiguous()}
        dw = torch.zeros(c["e"], c["n"], c["k"], dtype=torch.float64, device=DEV)
        for i, (o, k) in enumerate(zip(s["offsets"].tolist(), s["counts"].tolist())):
            if k:
                dw[i] = dy[o:o + k].T @ x[o:o + k]
        return {"dw": dw.view(-1, c["k"])}
    v = s["x"].double() if op == "ckpt" else _x_values(s["q"], s["sf"], _columns(c))
    if c["act"] in GATED:
        a, da = _x_act(v[:, ::2], "silu" if c["act"] == "swiglu" else "gelu")
        act = a * v[:, 1::2]
    else:
        act, da = _x_act(v, c["act"])
    q, sf = _x_mxfp8(v if op == "ckpt" else act)
    out = {"q": torch.where(real, q, 0.0), "sf": _x_spread(sf, real)}
    if op == "ckpt":
        return dict(out, out=torch.where(real, act, 0.0))
    d = s["dout"].double()
    if c["act"] in GATED:
        dx = torch.empty_like(v)
        dx[:, ::2], dx[:, 1::2] = d * da * v[:, 1::2], d * a
    else:
        dx = d * da
    return dict(out, dx=torch.where(real, dx, 0.0))
