"""GPU tests of the grouped GEMM with bias on the one-CTA kernel where a CTA meets
unused row bands between the tiles it computes.  The tile walk runs row bands
fastest, so the bands before and after the groups recur in every column block, and
buffers sized for any routing always have some.  The kernel's bias buffers are
handed from the loader to the epilogue by barriers: only tiles that are computed may
count.

Tolerance as in the tests of the grouped GEMM on CTA pairs."""
import numpy as np
import pytest
import torch

from _helpers import require_library
from test_gpu_grouped_pair import Groups, on_pairs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return require_library()


def skips_between_tiles(bands, lead, used, col_blocks):
    """CTAs that skip a tile after one they compute and compute another after it
    (up to 64 bands: one group of the walk)."""
    assert bands <= 64
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = np.arange(bands * col_blocks)
    computed = (tiles % bands >= lead) & (tiles % bands < lead + used)
    count = 0
    for cta in range(min(sms, tiles.size)):
        own = computed[cta::sms]
        at = np.flatnonzero(own)
        count += at.size > 1 and not own[at[0]:at[-1]].all()
    return count


@pytest.mark.parametrize("act,k", [("none", 264),      # three operand stages and wide staging, no activation
                                   ("none", 1288),     # four operand stages
                                   ("silu", 264), ("silu", 3592), ("swiglu", 264), ("swiglu", 2056)])
def test_bias_with_unused_bands_between_the_tiles(act, k):
    rng = np.random.default_rng(k)
    lead, trail, nw = 4, 19, 1920
    group_m = [int(v) for v in rng.integers(1, 128, 32)]
    for g in (3, 11, 12, 30):
        group_m[g] += 128
    group_m[7] = 0
    c = Groups(group_m, nw, k, seed=k, lead=lead)
    rows = c.rows + 128 * trail
    assert not on_pairs(rows, c.count, nw)
    assert skips_between_tiles(rows // 128, lead, c.rows // 128 - lead, (nw + 255) // 256) >= 10
    c.check(c.run(act, rows), act, groups=range(c.count) if k < 1000 else (0, 1, 3, 10, 11, 12, 13, 24, 30, 31))


def test_first_tiles_skipped():
    """Most bands are unused, so that CTAs skip one tile or more before their first
    one.  (With an activation and K below 2048 the groups stay on the one-CTA kernel.)"""
    c = Groups([100, 1, 128], 12800, 264, seed=3, lead=7)
    rows = c.rows + 128 * 3
    c.check(c.run("silu", rows), "silu")
