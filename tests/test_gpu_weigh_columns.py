"""Attention weight of cached keys where requests of many rows have columns that no token fills (128 is no multiple of the query
heads of a KV head)."""
import pytest
import torch

import long_ref as ref
import test_gpu_paged as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    from long_context_fm_gb300 import fm as mod
    return mod


@pytest.mark.parametrize("Hq", [3, 2])
def test_a_million_rows(fm, Hq):
    """Scores and log-sum-exps of zero: a key gets one from each row and head that attend it, whole numbers below 2^24, which
    fp32 adds up exactly in any order."""
    n, page, d = (1 << 20) + 3000, 64, 64
    pages = -(-n // page)
    att = fm.PagedAttention(1, Hq, 1, d, page, pages, pages, n, n)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    att.plan(base.i32([0]), base.i32([n]), table)
    k = torch.zeros(pages, 1, page, d, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(pages, 1, page, device="cuda")
    att.weigh(torch.zeros(n, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, Hq, device="cuda"), k, table, pool)
    att.check_status()
    assert torch.equal(pool.view(-1)[:n].long(), Hq * torch.arange(n, 0, -1, device="cuda"))
