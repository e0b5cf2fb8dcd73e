"""NaN in every place that no row attends (behind the window, behind the last token, pages that are gone) stays out of every
output: each element is finite and within the bounds."""
import pytest
import torch

import paged_strict
import test_gpu_paged as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    from long_context_fm_gb300 import fm as mod
    return mod


def strict(fm, case, seed, d, e4m3, o_dtype, few):
    ctx, new, Hq, Hkv, page, window, sink = case
    b = base.Batch(fm, ctx, new, Hq, Hkv, d, page, window, sink, e4m3, seed=seed, layout=["heads", "tokens", "pairs"][seed % 3])
    o, lse = b.run(o_dtype)
    paged_strict.check_attention(b.reference(), new, o, lse, d, b.p_err(o_dtype, few), e4m3, e4m3 and not few)


@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", range(len(base.FEW)))
def test_few_rows(fm, case, d, e4m3, o_dtype):
    strict(fm, base.FEW[case], case, d, e4m3, o_dtype, True)


@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", range(len(base.MANY)))
def test_many_rows(fm, case, d, e4m3, o_dtype):
    strict(fm, base.MANY[case], 100 + case, d, e4m3, o_dtype, False)
