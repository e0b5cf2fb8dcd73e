"""Attention weight of cached keys where units of many rows are cut into pieces, in lists longer than a warp."""
import pytest
import torch

import test_gpu_paged as base
from test_gpu_weigh import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    from long_context_fm_gb300 import fm as mod
    return mod


def test_cut_requests_behind_the_first_32(fm):
    """44 requests of many rows, of which those with more than a piece's row tiles are cut, on both sides of the 32nd; the joining kernel
    walks the list 32 entries at a time and carries the pieces before them on."""
    R, tpt = 44, 16                                 # 16 tokens a row tile
    g = torch.Generator().manual_seed(11)
    ctx, new = torch.randint(0, 900, (R,), generator=g).tolist(), torch.randint(40, 200, (R,), generator=g).tolist()
    new[7], new[30] = 45, 50                        # (whole ones next to them)
    b = base.Batch(fm, ctx, new, 8, 1, 64, 16, seed=9)
    check(fm, b)
    # int32 20 of the plan's header: row tiles of a piece, 0 where nothing was cut.
    length = int(b.att.plan_buffer[:256].view(torch.int32)[20])
    assert length > 0
    cut = [-(-new[r] // tpt) > length for r in sorted(range(R), key=lambda r: -(ctx[r] + new[r]))]       # the longest keys first
    assert any(cut[:32]) and any(cut[32:]) and not all(cut[:32]) and not all(cut[32:])
