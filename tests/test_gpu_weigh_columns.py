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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,new", [(3, 1, 150), (5, 1, 90), (14, 2, 130), (20, 1, 33), (28, 1, 40), (8, 2, 150), (6, 2, 2)])
def test_keys_whose_scores_are_minus_infinity(fm, Hq, Hkv, new, d):
    """A row that scores a key at -infinity gives it nothing, and the key keeps what it had; rows of zeros, which the kernel
    puts where no token is, have no score there."""
    b = base.Batch(fm, [300, 40], [new, 1], Hq, Hkv, d, 16, seed=5)
    b.q[:, :, 2] = 0.5
    b.q64[:, :, 2] = 0.5
    below = [5, 130, 299]                           # cached keys of request 0: one that every row attends without a mask among them
    at = [(b.table[0][j // 16], slice(None), j % 16) for j in below]
    for place in at:
        b.k64[place] = 0.0
    lse = attended(b, below)
    for place in at:
        b.k[(*place, 2)] = float("-inf")
    before = torch.rand(b.k.shape[:3], generator=torch.Generator().manual_seed(1))
    pool = before.clone().cuda()
    b.att.weigh(b.q, lse, b.k, b.dev_table, pool, b.scale)
    b.att.check_status()
    got = pool.double().cpu()
    want, tol = ref.weights(b.q64, b.k64, lse.double().cpu(), before.double(), b.table, b.ctx, b.new, b.scale)
    for place in at:
        want[place], tol[place] = before.double()[place], 0.0
    assert ((got - want).abs() <= tol).all()


def attended(b, without):
    """Log-sum-exps (fp32 [T, Hq]) of a batch whose request 0 has no such keys, from 64 bits."""
    out, t0, G = torch.empty(b.q64.shape[:2], dtype=torch.float64), 0, b.Hq // b.Hkv
    for r, (c, n) in enumerate(zip(b.ctx, b.new)):
        j = torch.arange(c + n)
        see = j <= torch.arange(c, c + n)[:, None]
        if r == 0:
            see[:, without] = False
        k = b.k64[[b.table[r][x // b.page] for x in range(c + n)], :, j % b.page]
        for h in range(b.Hq):
            x = b.scale * b.q64[t0:t0 + n, h] @ k[:, h // G].T
            out[t0:t0 + n, h] = x.masked_fill(~see, -torch.inf).logsumexp(1)
        t0 += n
    return out.float().cuda()
