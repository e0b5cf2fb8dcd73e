"""Attention weight of a step some of whose drafted tokens were refused: their rows are left out by an lse of +infinity."""
import math

import pytest
import torch

import long_ref as ref
import test_gpu_paged as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    from long_context_fm_gb300 import fm as mod
    return mod


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sink", [(0, 0), (60, 3)])
@pytest.mark.parametrize("new", [[3, 5, 1], [4, 100, 60]])
def test_refused_drafts_leave_nothing(fm, new, window, sink, d, e4m3):
    """As a program does it: attend, verify, weigh with the refused rows' lse at +infinity, against the sums over the kept rows."""
    b = base.Batch(fm, [300, 40, 17], new, 8, 2, d, 16, window=window, sink=sink, e4m3=e4m3, seed=3, poison=False)
    T, V, g = sum(new), 50, torch.Generator().manual_seed(4)
    _, lse = b.run(torch.float32)
    p = torch.softmax(torch.randn(T, V, generator=g), 1).cuda()
    tokens = torch.randint(V, (T,), generator=g).int().cuda()
    u = torch.full((T,), 0.9)                       # the drafts up to these rows are kept, the next one is not
    for r, keep in enumerate([1, 2, 0]):
        u[sum(new[:r]):sum(new[:r]) + keep] = 0.0
    out, n_out, _ = b.att.verify(p, None, tokens, u.cuda(), torch.rand(3, generator=g).cuda())
    assert n_out.tolist() == [2, 3, 1]
    z = lse.masked_fill((out < 0)[:, None], math.inf)
    assert int(z.isinf().all(1).sum()) == T - 6
    before = torch.rand(b.k.shape[:3], generator=g)
    pool = before.clone().cuda()
    b.att.weigh(b.q, z, b.k, b.dev_table, pool, b.scale, b.kd)
    b.att.check_status()
    terms = [r for r, n in enumerate(new) if n * 4 <= 32] if e4m3 else []
    z = z.double().cpu().masked_fill(z.cpu().isinf(), 1e30)         # (the bound of a weight of zero is zero)
    want, tol = ref.weights(b.q64, b.k64, z, before.double(), b.table, b.ctx, new, b.scale, window, sink, terms)
    assert ((pool.double().cpu() - want).abs() <= tol).all()
