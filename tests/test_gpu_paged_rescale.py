"""Running maxima that rise: every tile of 128 keys lifts the scores of some or all rows beyond the band within which
the kernels keep a maximum (2^8; 2^32 in the many-rows kernel over bf16), so that outputs and sums
already there are scaled down, or one key rises far above all others in the middle of a long row."""
import pytest
import torch

import test_gpu_paged as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    from long_context_fm_gb300 import fm as mod
    return mod


def lifted(fm, new, e4m3, d, per_tile, seed, Hq, Hkv, ctx=1500, window=0, sink=0):
    """Keys with a coordinate of their own that grows by the tile; rows of q with the factor that lifts (or sinks) their scores
    by about `per_tile` of base 2 a tile, a different one for every row."""
    b = base.Batch(fm, [ctx, 5], [new, 1], Hq, Hkv, d, 16, window, sink, e4m3, seed=seed)
    for j in range(ctx + new):
        page, at = b.table[0][j // 16], j % 16
        if page < 0:                # behind the window
            continue
        step = float(j // 128 + 1) * (32.0 if e4m3 else 4.0)        # e4m3: as a code's value, 448 at most
        b.k64[page, :, at, 7] = step * (float(b.kd) if e4m3 else 1.0)
        b.k[page, :, at, 7] = torch.tensor(step).to(torch.float8_e4m3fn).view(torch.uint8).item() if e4m3 else step
    unit = (32.0 * float(b.kd) if e4m3 else 4.0) * b.scale * 1.4426950408889634
    lift = torch.tensor([[per_tile / unit * (1 - 0.23 * ((3 * i + h) % 9)) for h in range(Hq)] for i in range(b.q64.shape[0])]).bfloat16()
    q = b.q64.clone()
    q[:, :, 7] = lift.double()
    b.q64, b.q = q, q.bfloat16().cuda()
    return b


TYPES = pytest.mark.parametrize("e4m3,o_dtype", [(x, y) for x in (False, True) for y in (torch.bfloat16, torch.float32)])


# 96 KV heads: eight tiles or so a CTA, most units in one or two of them.
@TYPES
@pytest.mark.parametrize("per_tile", [11.0, 45.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 6, 13])
def test_maxima_that_rise_few_rows(fm, new, d, e4m3, per_tile, o_dtype):
    lifted(fm, new, e4m3, d, per_tile, new, 192, 96).check(o_dtype)


# 2 KV heads: split along the keys; 160: whole units.
@TYPES
@pytest.mark.parametrize("per_tile", [11.0, 45.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,Hq,Hkv,window,sink", [(40, 4, 2, 0, 0), (90, 4, 2, 500, 20), (40, 160, 160, 0, 0)])
def test_maxima_that_rise_many_rows(fm, new, Hq, Hkv, window, sink, d, e4m3, per_tile, o_dtype):
    lifted(fm, new, e4m3, d, per_tile, new, Hq, Hkv, window=window, sink=sink).check(o_dtype, few=False)


@TYPES
@pytest.mark.parametrize("q_scale", [12.0, 60.0])
@pytest.mark.parametrize("new", [2, 12, 100])
def test_scores_spread_widely(fm, new, q_scale, e4m3, o_dtype):
    b = base.Batch(fm, [1800, 300], [new, 1], 96, 48, 128, 32, e4m3=e4m3, seed=4, q_scale=q_scale)
    b.check(o_dtype, few=new * 2 <= 32)
