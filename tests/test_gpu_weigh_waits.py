"""The weight kernels' own recovery: a tile's load is one byte short, its wait runs out after 2e6 cycles, the call ends with
FM_ERR_TIMEOUT and, planned again, gives what it gave before."""
import pytest
import torch

import test_gpu_paged as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    from long_context_fm_gb300 import fm as mod
    return mod


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kernel,new", [("few", [1, 2, 0]), ("many", [100, 1, 40]), ("few", [100, 1, 40])])
def test_a_wait_that_runs_out(fm, kernel, new, e4m3):
    """Lengths that give every CTA several key tiles."""
    b = base.Batch(fm, [9000, 5000, 700], new, 32, 8, 128, 16, e4m3=e4m3, seed=1)
    _, lse = b.run(torch.float32)

    def weigh():
        pool = torch.zeros(b.k.shape[:3], device="cuda")
        b.att.weigh(b.q, lse, b.k, b.dev_table, pool, b.scale, b.kd)
        torch.cuda.synchronize()
        return pool

    before = weigh()
    b.att.check_status()
    fm.fm_debug_wait_test(fm.KERNEL_NAMES.index("paged_weigh_" + kernel), 2_000_000)
    try:
        weigh()
    finally:
        fm.fm_debug_wait_test(-1, 0)
    assert int(b.att.status.item()) == fm.FM_ERR_TIMEOUT
    b.att.status.zero_()
    b.att.plan(base.i32(b.ctx), base.i32(new), b.dev_table)
    assert torch.equal(before, weigh())
    b.att.check_status()
