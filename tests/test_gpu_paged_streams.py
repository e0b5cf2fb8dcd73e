"""Two plans at work at once, on two streams: chunks, split chunks and single tokens, each with the bits it has alone."""
import pytest
import torch

import test_gpu_paged as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e4m3", [False, True])
def test_two_calls_at_once(e4m3):
    from long_context_fm_gb300 import fm
    jobs = [base.Batch(fm, [3000, 40, 700, 9], new, 8, 2, 128, 32, e4m3=e4m3, seed=seed)
            for seed, new in ((1, [30, 1, 100, 2]), (2, [1, 60, 3, 0]))]
    alone = [[x.clone() for x in b.run(torch.float32, rows_behind=0)] for b in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(12):
        for i, b in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                b.att.plan(base.i32(b.ctx), base.i32(b.new), b.dev_table)
                got[i] += [b.att.attend(b.q, b.k, b.v, b.dev_table, b.scale, torch.float32, b.kd, b.vd) for _ in range(4)]
    torch.cuda.synchronize()
    for b, want, outs in zip(jobs, alone, got):
        b.att.check_status()
        for out in outs:
            for x, y in zip(out, want):
                assert torch.equal(x.view(torch.int32), y.view(torch.int32))
