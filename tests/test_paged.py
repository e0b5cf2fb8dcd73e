"""Paged-cache operators: what the host refuses, before anything is launched (no GPU is used)."""
import ctypes

import pytest
import torch

from long_context_fm_gb300 import build as fmbuild


@pytest.fixture(scope="module")
def fm():
    fmbuild.build()
    from long_context_fm_gb300 import fm as mod
    return mod


STEP = dict(requests=4, max_tokens=64, max_q=8, max_pages=10, num_pages=40, page_size=32, Hq=8, Hkv=4, d=128, window=0,
            sink=0)


def step_of(fm, **kw):
    return fm.PagedStep(*[{**STEP, **kw}[n] for n, _ in fm.PagedStep._fields_])


BAD_STEPS = [
    (dict(requests=0), 1), (dict(max_tokens=0), 1), (dict(max_q=0), 1), (dict(max_q=65), 1), (dict(max_pages=0), 1),
    (dict(num_pages=0), 1), (dict(page_size=0), 1), (dict(Hq=6), 1), (dict(Hkv=0), 1), (dict(window=-1), 1), (dict(sink=-3), 1),
    (dict(d=96), 2), (dict(page_size=24), 2), (dict(Hq=132, Hkv=4), 2), (dict(requests=8193), 2),
    (dict(max_pages=1 << 26), 2), (dict(max_tokens=(1 << 24) + 1), 2), (dict(page_size=65552), 2), (dict(Hq=8192, Hkv=8192), 2),
]


@pytest.mark.parametrize("change,code", BAD_STEPS)
def test_sizes_of_a_step_that_are_refused(fm, change, code):
    s = step_of(fm, **change)
    assert fm.fm_paged_plan_bytes(s) == 0
    got = fm._lib.fm_paged_plan(ctypes.byref(s), *[None] * 4, 0, *[None] * 7, 0, None, None)
    assert got == code


def test_a_sink_without_a_window_is_a_step(fm):
    assert fm.fm_paged_plan_bytes(step_of(fm, sink=3)) == fm.fm_paged_plan_bytes(step_of(fm)) > 0


def test_plan_bytes(fm):
    small, more = step_of(fm), step_of(fm, requests=4096)
    assert fm.fm_paged_plan_bytes(more) >= fm.fm_paged_plan_bytes(small) + 4092 * 24 - 512   # sections begin on 256 bytes
    assert fm._lib.fm_paged_plan_bytes(None) == 0


A = 0x10000     # an aligned address that no refused call reads


def plan_args(fm, **kw):
    s = kw.pop("step", None) or step_of(fm)
    d = dict(ctx=A, new=A, table=A, free=A, n_free=5, head=A, next=A, seq=A, cu=A, slots=A, pos=A, plan=A, bytes=1 << 40, status=A)
    d.update(kw)
    return [ctypes.byref(s), d["ctx"], d["new"], d["table"], d["free"], d["n_free"], d["head"], d["next"], d["seq"], d["cu"],
            d["slots"], d["pos"], d["plan"], d["bytes"], d["status"], None]


@pytest.mark.parametrize("change,code", [
    (dict(ctx=None), 1), (dict(new=A + 2), 1), (dict(table=None), 1), (dict(head=None), 1), (dict(next=None), 1), (dict(n_free=-1), 1),
    (dict(seq=None), 1), (dict(cu=A + 1), 1), (dict(slots=None), 1), (dict(slots=A + 4), 1), (dict(pos=A + 2), 1),
    (dict(status=None), 1), (dict(plan=None), 6), (dict(plan=A + 16), 6), (dict(bytes=255), 6)])
def test_plan_arguments_that_are_refused(fm, change, code):
    assert fm._lib.fm_paged_plan(*plan_args(fm, **change)) == code


def cache_of(fm, **kw):
    d = dict(k=A, v=A, k_page=4 * 32 * 128, k_head=32 * 128, k_tok=128, v_page=4 * 32 * 128, v_head=32 * 128, v_tok=128,
             k_descale=A, v_descale=A, num_pages=40, page_size=32, Hkv=4, d=128, dtype=0)
    d.update(kw)
    return fm.PagedCache(*[d[n] for n, _ in fm.PagedCache._fields_])


BAD_CACHES = [(dict(k=None), 1), (dict(v=A + 8), 1), (dict(k_tok=127), 1), (dict(k_tok=64), 1), (dict(v_head=-128), 1), (dict(v_page=0), 1),
              (dict(k_page=4), 1), (dict(dtype=1), 1), (dict(dtype=3), 1), (dict(dtype=2, k_descale=None), 1), (dict(dtype=2, v_tok=136), 1),
              (dict(num_pages=0), 1), (dict(d=256), 2), (dict(page_size=40), 2), (dict(page_size=65552), 2), (dict(Hkv=4097), 2)]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_caches_that_are_refused(fm, change, code):
    c = cache_of(fm, **change)
    got = fm._lib.fm_paged_append(A, 1024, 128, A, 1024, 128, A, 5, ctypes.byref(c), A, None)
    assert got == code
    s = step_of(fm)
    got = fm._lib.fm_attn_paged(ctypes.byref(s), A, 1024, 128, 8, ctypes.byref(c), A, A, 1 << 40, 0.1, A, 0, A, A, None)
    assert got == code


@pytest.mark.parametrize("at,value", [(0, None), (0, A + 2), (1, 1025), (2, -8), (3, None), (4, 4), (6, None), (6, A + 4), (7, -1), (8, None),
                                      (9, None)])
def test_append_arguments_that_are_refused(fm, at, value):
    c = cache_of(fm)
    args = [A, 1024, 128, A, 1024, 128, A, 5, ctypes.byref(c), A, None]
    args[at] = value
    assert fm._lib.fm_paged_append(*args) == 1


@pytest.mark.parametrize("at,value,code", [
    (0, None, 1), (1, None, 1), (1, A + 8, 1), (2, 1020, 1), (3, -8, 1), (4, -1, 1), (5, None, 1), (6, None, 1), (7, None, 6), (7, A + 128, 6), (8, 100, 6),
    (9, 0.0, 1), (9, float("nan"), 1), (9, float("inf"), 1), (10, None, 1), (11, 2, 1), (12, None, 1), (13, A + 1, 1)])
def test_attention_arguments_that_are_refused(fm, at, value, code):
    s, c = step_of(fm), cache_of(fm)
    args = [ctypes.byref(s), A, 1024, 128, 8, ctypes.byref(c), A, A, 1 << 40, 0.1, A, 0, A, A, None]
    args[at] = value
    assert fm._lib.fm_attn_paged(*args) == code


@pytest.mark.parametrize("change", [dict(num_pages=39), dict(page_size=16), dict(Hkv=8), dict(d=64)])
def test_a_cache_of_other_sizes_than_the_step(fm, change):
    s, c = step_of(fm), cache_of(fm, **change)
    assert fm._lib.fm_attn_paged(ctypes.byref(s), A, 1024, 128, 8, ctypes.byref(c), A, A, 1 << 40, 0.1, A, 0, A, A, None) == 1


def test_python_refuses_what_is_not_on_the_gpu(fm):
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cache = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fm.fm_paged_append(x, x, torch.zeros(4, dtype=torch.int64), cache, cache, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        fm.PagedAttention(4, 6, 4, 128, 32, 40, 10, 64, 8, device="cpu")


FAKE = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from long_context_fm_gb300 import fm
with FakeTensorMode():
    k = torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache = torch.empty(8, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(4, dtype=torch.int64, device="cuda")
    word = torch.empty(1, dtype=torch.int32, device="cuda")
    table = torch.empty(1, 8, dtype=torch.int32, device="cuda")
    two = torch.empty(2, dtype=torch.int32, device="cuda")
    plan = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    o = torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(4, 2, device="cuda")
step = fm.PagedStep(1, 4, 4, 8, 8, 16, 2, 2, 64, 0, 0)
raised = 0
for call in (lambda: fm.fm_paged_append(k, k, slots, cache, cache, word),
             lambda: fm.fm_paged_plan(step, word, word, table, word, two, slots, word, plan, word),
             lambda: fm._call.attend(__import__("ctypes").addressof(step), k, cache, cache, table, plan, 0.1, False, word, None, None) or 1 / 0):
    try:
        call()
    except Exception:
        raised += 1
print("raised", raised)
"""


def test_a_tensor_without_memory_raises(fm):
    """torch's exceptions (here: no device, or a tensor without storage) end as Python's."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FAKE], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and "raised 3" in r.stdout, r.stderr


@pytest.mark.parametrize("name", ["max_tokens", "window", "num_pages"])
@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 64, -(1 << 31) - 1])
def test_sizes_past_32_bits_are_refused(fm, name, value):
    with pytest.raises(ValueError):
        step_of(fm, **{name: value})
