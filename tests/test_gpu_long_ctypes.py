"""The calls around the attention of long conversations without the CPython extension: the same bits and the same refusals through ctypes."""
import pytest
import torch

import test_gpu_long_run as base

pytestmark = pytest.mark.gpu


@pytest.fixture
def fm(monkeypatch):
    from long_context_fm_gb300 import fm as mod
    assert mod._call is not mod._NoCall, "the extension is built with the library"
    return mod


def conversation(fm, e4m3):
    s = base.Server(fm, e4m3)
    s.step([60, 0, 5], False)
    s.step([1, 90, 40], False)
    s.step([3, 2, 1], True)
    x = torch.randn(2, 3, 7, 64, generator=torch.Generator().manual_seed(1)).cuda()
    pos = torch.arange(7, dtype=torch.int32, device="cuda")
    out = [fm.fm_rope(x, pos, s.rot), fm.fm_rope(x, pos.repeat(2, 1), s.rot, out_dtype=torch.bfloat16, inverse=True), fm.fm_rope(x[0].transpose(0, 1), pos, s.rot)]
    return [y.contiguous().view(torch.uint8) for y in (s.lens, s.table, s.free, s.head, *s.weights, *(c for pair in s.caches for c in pair), *out)]


@pytest.mark.parametrize("e4m3", [False, True])
def test_the_same_bits(fm, monkeypatch, e4m3):
    with_it = conversation(fm, e4m3)
    monkeypatch.setattr(fm, "_call", fm._NoCall)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        without = conversation(fm, e4m3)
    for x, y in zip(with_it, without):
        assert torch.equal(x, y)


@pytest.mark.parametrize("extension", [True, False])
def test_refusals(fm, monkeypatch, extension):
    if not extension:
        monkeypatch.setattr(fm, "_call", fm._NoCall)
    rot, cpu = fm.Rotary(64), fm.Rotary(64, device="cpu")
    x = torch.zeros(5, 4, 64, dtype=torch.bfloat16, device="cuda")
    pos, slots, word = base.i32(range(5)), torch.arange(5, device="cuda"), base.i32([0])
    cache, pool = torch.zeros(6, 4, 16, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(6, 4, 16, device="cuda")
    p, u = torch.full((5, 9), 1 / 9, device="cuda"), torch.zeros(5, device="cuda")
    step = fm.PagedStep(1, 5, 5, 6, 6, 16, 4, 4, 64, 0, 0)
    plan = torch.zeros(fm.fm_paged_plan_bytes(step), dtype=torch.uint8, device="cuda")
    lse, table, lens, cu = torch.zeros(5, 4, device="cuda"), base.i32([range(6)]), base.i32([40]), base.i32([0, 5])
    calls = [
        (TypeError, lambda: fm.fm_rope(x.half(), pos, rot)), (TypeError, lambda: fm.fm_rope(x, pos, cpu)), (TypeError, lambda: fm.fm_rope(x, pos.long(), rot)),
        (ValueError, lambda: fm.fm_rope(x, pos[:4], rot)), (ValueError, lambda: fm.fm_rope(x[0], pos, rot)), (ValueError, lambda: fm.fm_rope(x, pos, rot, out=x[:4])),
        (TypeError, lambda: fm.fm_rope(x, pos, rot, out=x, out_dtype=torch.float32)), (ValueError, lambda: fm.fm_rope(x.transpose(1, 2), pos, rot)),
        (fm.FmError, lambda: fm.fm_rope(x, pos, rot, out=x[:1].expand(5, 4, 64))), (fm.FmError, lambda: fm.fm_rope(x[..., :32].contiguous(), pos, rot)),
        (ValueError, lambda: fm.fm_paged_append_rope(x, x[:4], x, slots, pos, rot, cache, cache, word)),
        (ValueError, lambda: fm.fm_paged_append_rope(x, x, x, slots[:4], pos, rot, cache, cache, word)),
        (TypeError, lambda: fm.fm_paged_append_rope(x, x, x, slots, pos.long(), rot, cache, cache, word)),
        (TypeError, lambda: fm.fm_paged_append_rope(x, x, x, slots, pos, None, cache, cache, word)),
        (ValueError, lambda: fm.fm_paged_weights(step, x, lse[:4], cache, table, plan, 0.1, pool, word)),
        (ValueError, lambda: fm.fm_paged_weights(step, x, lse, cache, table, plan, 0.1, pool[:5], word)),
        (fm.FmError, lambda: fm.fm_paged_weights(step, x, lse, cache, table, plan, 0.0, pool, word)),
        (TypeError, lambda: fm.fm_paged_weights(step, x, lse.bfloat16(), cache, table, plan, 0.1, pool, word)),
        (fm.FmError, lambda: fm.fm_paged_evict(lens, table, cache, cache, pool, 0, word)),
        (fm.FmError, lambda: fm.fm_paged_evict(lens, table, cache, cache, pool, 10, word, recent=11)),
        (fm.FmError, lambda: fm.fm_paged_evict(lens, table, cache, cache, pool, 10, word, new_lens=lens)),
        (ValueError, lambda: fm.fm_paged_evict(lens, table, cache, cache, pool, 1 << 32, word)),
        (ValueError, lambda: fm.fm_paged_evict(lens, table, cache, cache, pool[:, :3].contiguous(), 10, word)),
        (ValueError, lambda: fm.fm_paged_evict(lens, base.i32([[1], [2]]), cache, cache, pool, 10, word)),
        (ValueError, lambda: fm.fm_paged_release(lens, lens, table, 16, 6, pos, None, word)),
        (fm.FmError, lambda: fm.fm_paged_release(lens, lens, table, 15, 6, pos, word, word)),
        (ValueError, lambda: fm.fm_paged_release(lens, base.i32([1, 2]), table, 16, 6, pos, word, word)),
        (ValueError, lambda: fm.fm_verify_drafts(p, p[:4], pos, u, u[:1], cu, lens, word)),
        (ValueError, lambda: fm.fm_verify_drafts(p, p.bfloat16(), pos, u, u[:1], cu, lens, word)),
        (TypeError, lambda: fm.fm_verify_drafts(p, None, pos.long(), u, u[:1], cu, lens, word)),
        (ValueError, lambda: fm.fm_verify_drafts(p, None, pos, u, u, cu, lens, word)),
        (TypeError, lambda: fm.fm_verify_drafts(p.half(), None, pos, u, u[:1], cu, lens, word))]
    for error, call in calls:
        with pytest.raises(error):
            call()
    assert int(word.item()) == 0
