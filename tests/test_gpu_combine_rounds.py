"""GPU tests of combine where its persistent blocks take several steps each (six times as
many steps as resident blocks, or more): the next step's rows and weights are requested
ahead, and the last steps cover fewer tokens.  For topk 1 every step has its own block.

Reference in 64 bits on the GPU; bound as in the other tests of combine."""
import pytest
import torch

from _helpers import nv, require_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def tokens_per_round(topk, h):
    """Tokens that the resident blocks take in one step (1024 threads per SM, eight columns each)."""
    threads = 128 if h >= 1024 else ((h + 7) // 8 + 31) // 32 * 32
    parts = -(-h // (threads * 8))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    resident = max(1, sms * (1024 // threads) // parts)
    return resident * (2 if topk == 2 else 1)


@pytest.mark.parametrize("weights,residual", [(True, True), (True, False), (False, False)])
@pytest.mark.parametrize("topk,h", [(2, 264), (2, 4104), (3, 4100), (4, 1024), (5, 2048), (8, 520), (9, 1032), (17, 2052)])
def test_several_steps_per_block(topk, h, weights, residual):
    per = tokens_per_round(topk, h)
    tokens = 7 * per + 1                                     # eight steps in one block, seven in the others
    experts = 24
    g = torch.Generator(device="cuda").manual_seed(topk * h)
    ids = torch.randint(-1, experts + 1, (tokens, topk), generator=g, device="cuda", dtype=torch.int32)
    offsets, _, dest = nv.moe_sort(ids, experts)
    rows, ld = nv.nvfp4_moe_rows(tokens, topk, experts), (h + 7) // 8 * 8 + 8
    y = torch.randn(rows, ld, generator=g, device="cuda").bfloat16()[:, :h]
    y[int(offsets[-1]):] = float("nan")
    w = torch.rand(tokens, topk, generator=g, device="cuda") if weights else None
    if weights:
        w[dest < 0] = float("nan")
    res = torch.randn(tokens, ld, generator=g, device="cuda").bfloat16()[:, :h] if residual else None
    out = torch.full((tokens + 1, ld), -3.0, dtype=torch.bfloat16, device="cuda")
    nv.moe_combine(y, dest, w, res, out=out[:tokens, :h])
    torch.cuda.synchronize()
    assert (out[:, h:] == -3.0).all() and (out[tokens] == -3.0).all()
    ref = torch.zeros(tokens, h, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(ref)
    for j in range(topk):
        here = dest[:, j] >= 0
        term = torch.where(here[:, None], y[dest[:, j].clamp_min(0).long()].double(), 0.0)
        if weights:
            term = torch.where(here[:, None], term * w[:, j, None].double(), 0.0)
        ref += term
        size += term.abs()
    if residual:
        ref += res.double()
        size += res.double().abs()
    err = (out[:tokens, :h].double() - ref).abs()
    assert (err <= 2.0 ** -8 * ref.abs() + 66 * 2.0 ** -23 * size).all()


@pytest.mark.parametrize("topk,h", [(2, 520), (8, 1024)])
def test_both_sides_of_the_rule_agree(topk, h):
    """The same tokens in calls below the rule (a block per step) have the same bits."""
    per = tokens_per_round(topk, h)
    tokens, experts = 6 * per + per // 2, 16
    g = torch.Generator(device="cuda").manual_seed(h)
    ids = torch.randint(0, experts, (tokens, topk), generator=g, device="cuda", dtype=torch.int32)
    _, _, dest = nv.moe_sort(ids, experts)
    y = torch.randn(nv.nvfp4_moe_rows(tokens, topk, experts), h, generator=g, device="cuda").bfloat16()
    w = torch.rand(tokens, topk, generator=g, device="cuda")
    whole = nv.moe_combine(y, dest, w)
    cut = 2 * per + 3
    parts = [nv.moe_combine(y, dest[i:i + cut], w[i:i + cut]) for i in range(0, tokens, cut)]
    torch.cuda.synchronize()
    assert torch.equal(whole.view(torch.int16), torch.cat(parts).view(torch.int16))
