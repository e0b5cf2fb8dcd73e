"""The paged calls without the CPython extension: the same bits and the same refusals through ctypes."""
import pytest
import torch

import test_gpu_paged_run as base

pytestmark = pytest.mark.gpu


@pytest.fixture
def fm(monkeypatch):
    from long_context_fm_gb300 import fm as mod
    assert mod._call is not mod._NoCall, "the extension is built with the library"
    return mod


def step(fm, e4m3):
    g = torch.Generator(device="cuda").manual_seed(7)
    att = fm.PagedAttention(3, 8, 2, 64, 16, 40, 12, 60, 40)
    lens, new = base.i32([70, 3, 100]), base.i32([1, 40, 5])
    table = torch.randperm(40, generator=g, device="cuda")[:36].to(torch.int32).view(3, 12)
    kc, vc = (torch.randn(40, 2, 16, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    ds = torch.tensor([0.02], device="cuda") if e4m3 else None
    if e4m3:
        kc, vc = ((x.float() / ds).clamp(-448, 448).to(torch.float8_e4m3fn) for x in (kc, vc))
    q, k, v = (torch.randn(46, h, 64, generator=g, device="cuda").bfloat16() for h in (8, 2, 2))
    att.plan(lens, new, table, free_pages=torch.arange(36, 40, dtype=torch.int32, device="cuda"), free_head=base.i32([0]))
    att.append(k, v, kc, vc, ds, ds)
    o, lse = att.attend(q, kc, vc, table, k_descale=ds, v_descale=ds)
    att.check_status()
    return [x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in (table, att.cu_q, att.slots, att.positions, att.seq_lens, kc, vc, o, lse)]


@pytest.mark.parametrize("e4m3", [False, True])
def test_the_same_bits(fm, monkeypatch, e4m3):
    with_it = step(fm, e4m3)
    monkeypatch.setattr(fm, "_call", fm._NoCall)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        without = step(fm, e4m3)
    for x, y in zip(with_it, without):
        assert torch.equal(x, y)


@pytest.mark.filterwarnings("ignore:the paged calls")
def test_the_same_refusals(fm, monkeypatch):
    monkeypatch.setattr(fm, "_call", fm._NoCall)
    base.test_python_refusals(fm)
