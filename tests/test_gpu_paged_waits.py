"""The paged attention kernels' own recovery: a tile's load is withheld, its wait runs out after 2e6 cycles, the call ends with
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
@pytest.mark.parametrize("kernel,new", [("few", [1, 2, 0]), ("many", [100, 1, 40]), ("many", [400, 1, 0]), ("few", [100, 1, 40])])
def test_a_wait_that_runs_out(fm, kernel, new, e4m3):
    """Few rows alone, whole and split chunks, and few rows behind chunks."""
    b = base.Batch(fm, [3000, 5000, 700], new, 32, 8, 128, 16, e4m3=e4m3, seed=1)
    before = b.run(torch.float32)
    fm.fm_debug_wait_test(fm.KERNEL_NAMES.index("paged_decode" if kernel == "few" else "paged_chunk"), 2_000_000)
    try:
        b.att.attend(b.q, b.k, b.v, b.dev_table, b.scale, torch.float32, b.kd, b.vd)
        torch.cuda.synchronize()
    finally:
        fm.fm_debug_wait_test(-1, 0)
    assert int(b.att.status.item()) == fm.FM_ERR_TIMEOUT
    b.att.status.zero_()
    b.att.plan(base.i32(b.ctx), base.i32(new), b.dev_table)
    for x, y in zip(before, b.run(torch.float32)):      # (bits: an e4m3 cast beyond 464 is NaN, and so is what attends it)
        assert torch.equal(x.view(torch.int32), y.view(torch.int32))
