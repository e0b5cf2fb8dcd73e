"""Operators around the attention of long conversations: the frequency table, and what the host refuses before anything is
launched (no GPU is used)."""
import ctypes
import math

import pytest
import torch

import long_ref as ref
from long_context_fm_gb300 import build as fmbuild
from test_paged import A, BAD_CACHES, BAD_STEPS, cache_of, step_of


@pytest.fixture(scope="module")
def fm():
    fmbuild.build()
    from long_context_fm_gb300 import fm as mod
    return mod


SPEC = dict(rot=64, scaling=0, base=10000.0, factor=1.0, original=4096.0, slow=1.0, fast=32.0)


def spec_of(fm, **kw):
    return fm.RotarySpec(*[{**SPEC, **kw}[n] for n, _ in fm.RotarySpec._fields_])


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot,base,factor", [(2, 10000.0, 1.0), (8, 1.5, 3.0), (64, 10000.0, 4.0), (128, 1e6, 32.0)])
def test_frequencies(fm, rot, base, factor, scaling):
    """Each within a few roundings of a double of theta / 2 pi turns."""
    if scaling == "ntk" and rot == 2:
        return
    turns, m = fm.fm_rotary_table(spec_of(fm, rot=rot, base=base, factor=factor, scaling=fm.ROPE_SCALINGS[scaling], original=8192.0, slow=2.0, fast=20.0))
    theta, want = ref.frequencies(rot, base, scaling, factor, 8192.0, 2.0, 20.0)
    assert abs(m - want) <= 2.0 ** -24 * want
    assert len(turns) == rot // 2
    for t, f in zip(turns.tolist(), theta.tolist()):
        f = f / (2 * math.pi)
        assert abs(t * 2.0 ** -64 - f) <= f * 2.0 ** -49 + 2.0 ** -64


@pytest.mark.parametrize("change", [dict(rot=0), dict(rot=-2), dict(rot=3), dict(rot=130), dict(base=1.0), dict(base=math.nan), dict(base=math.inf), dict(scaling=4),
                                    dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=2, factor=math.nan), dict(scaling=2, rot=2), dict(scaling=3, factor=math.inf),
                                    dict(scaling=3, original=0.0), dict(scaling=3, slow=-1.0), dict(scaling=3, slow=32.0), dict(scaling=3, fast=math.inf)])
def test_tables_that_are_refused(fm, change):
    with pytest.raises(fm.FmError) as e:
        fm.fm_rotary_table(spec_of(fm, **change))
    assert e.value.code == 1


def test_rotaries_that_are_refused(fm):
    for bad in (dict(rot=12), dict(rot=0), dict(rot=136), dict(rot=64, scaling="longer")):
        with pytest.raises(ValueError):
            fm.Rotary(**bad, device="cpu")
    with pytest.raises(fm.FmError):
        fm.Rotary(64, scaling="linear", factor=0.1, device="cpu")


def rotary_of(fm, **kw):
    return fm.RotaryTable(*[{**dict(turns=A, rot=64, interleaved=0, magnitude=1.0), **kw}[n] for n, _ in fm.RotaryTable._fields_])


ROPE = dict(x=A, xt=0, xb=8 * 64 * 128, xh=64 * 128, xn=128, pos=A, pb=64, B=2, H=8, N=64, d=128, y=2 * A, yt=0, yb=8 * 64 * 128, yh=64 * 128, yn=128)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), 1), (dict(x=A + 8), 1), (dict(y=None), 1), (dict(pos=None), 1), (dict(pos=A + 2), 1), (dict(pb=-1), 1), (dict(xt=2), 1), (dict(yt=3), 1),
    (dict(B=0), 1), (dict(N=0), 1), (dict(H=-1), 1), (dict(d=96), 2), (dict(xn=129), 1), (dict(xt=1, xn=130), 1), (dict(yh=4), 1), (dict(xh=-128), 1),
    (dict(yn=64), 1), (dict(yh=0), 1), (dict(yb=0), 1), (dict(yh=128, yn=128), 1), (dict(yh=63 * 128), 1), (dict(y=A, yt=1), 1), (dict(y=A, yn=8 * 128, yh=128), 1),
    (dict(xb=1 << 41), 1)])
def test_rope_arguments_that_are_refused(fm, change, code):
    a = {**ROPE, **change}
    r = rotary_of(fm)
    got = fm._lib.fm_rope(a["x"], a["xt"], fm.Strides(a["xb"], a["xh"], a["xn"]), a["pos"], a["pb"], a["B"], a["H"], a["N"], a["d"], ctypes.byref(r), 0,
                          a["y"], a["yt"], fm.Strides(a["yb"], a["yh"], a["yn"]), None)
    assert got == code


BAD_ROTARIES = [(dict(turns=None), 1), (dict(turns=A + 8), 1), (dict(rot=0), 1), (dict(magnitude=math.nan), 1), (dict(rot=136), 2), (dict(rot=60), 2)]


@pytest.mark.parametrize("change,code", BAD_ROTARIES)
def test_rotary_tables_that_are_refused(fm, change, code):
    r, c, s = rotary_of(fm, **change), cache_of(fm), fm.Strides(8 * 64 * 128, 64 * 128, 128)
    assert fm._lib.fm_rope(A, 0, s, A, 64, 2, 8, 64, 128, ctypes.byref(r), 0, 2 * A, 0, s, None) == code
    assert fm._lib.fm_paged_append_rope(*append_args(fm, rotary=ctypes.byref(r), cache=ctypes.byref(c))) == code
    assert fm._lib.fm_rope(A, 0, s, A, 64, 2, 8, 64, 128, None, 0, 2 * A, 0, s, None) == 1


def append_args(fm, **kw):
    d = dict(q=A, qt=1024, qh=128, Hq=8, k=A, kt=1024, kh=128, v=A, vt=1024, vh=128, slots=A, pos=A, T=5, rotary=ctypes.byref(rotary_of(fm)),
             cache=ctypes.byref(cache_of(fm)), out=2 * A, ot=1024, oh=128, status=A)
    d.update(kw)
    return [*d.values(), None]


@pytest.mark.parametrize("change,code", [
    (dict(q=None), 1), (dict(qt=1025), 1), (dict(qh=-8), 1), (dict(Hq=0), 1), (dict(Hq=4097), 2), (dict(k=A + 8), 1), (dict(kt=4), 1), (dict(v=None), 1), (dict(vh=0), 1),
    (dict(slots=None), 1), (dict(slots=A + 4), 1), (dict(pos=None), 1), (dict(pos=A + 2), 1), (dict(T=-1), 1), (dict(T=(1 << 24) + 1), 1), (dict(out=None), 1),
    (dict(ot=512), 1), (dict(oh=64), 1), (dict(out=A, oh=128, ot=2048), 1), (dict(status=None), 1), (dict(rotary=None), 1)])
def test_append_rope_arguments_that_are_refused(fm, change, code):
    assert fm._lib.fm_paged_append_rope(*append_args(fm, **change)) == code


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_caches_that_are_refused(fm, change, code):
    c = ctypes.byref(cache_of(fm, **change))
    assert fm._lib.fm_paged_append_rope(*append_args(fm, cache=c)) == code
    assert fm._lib.fm_paged_weights(*weigh_args(fm, cache=c)) == code
    assert fm._lib.fm_paged_evict(*evict_args(fm, cache=c)) == code


def weigh_args(fm, **kw):
    d = dict(step=ctypes.byref(step_of(fm)), q=A, qt=1024, qh=128, rows=8, cache=ctypes.byref(cache_of(fm)), table=A, plan=A, bytes=1 << 40, scale=0.1, lse=A,
             weights=A, status=A)
    d.update(kw)
    return [*d.values(), None]


@pytest.mark.parametrize("change,code", [
    (dict(step=None), 1), (dict(q=None), 1), (dict(qt=1020), 1), (dict(qh=-8), 1), (dict(rows=-1), 1), (dict(cache=None), 1), (dict(table=None), 1), (dict(plan=None), 6),
    (dict(plan=A + 128), 6), (dict(bytes=100), 6), (dict(scale=0.0), 1), (dict(scale=math.inf), 1), (dict(lse=None), 1), (dict(lse=A + 2), 1), (dict(weights=None), 1),
    (dict(status=A + 1), 1)])
def test_weights_arguments_that_are_refused(fm, change, code):
    assert fm._lib.fm_paged_weights(*weigh_args(fm, **change)) == code


@pytest.mark.parametrize("change,code", BAD_STEPS)
def test_steps_that_are_refused(fm, change, code):
    assert fm._lib.fm_paged_weights(*weigh_args(fm, step=ctypes.byref(step_of(fm, **change)))) == code


@pytest.mark.parametrize("change", [dict(num_pages=39), dict(page_size=16), dict(Hkv=8), dict(d=64)])
def test_a_cache_of_other_sizes_than_the_step(fm, change):
    assert fm._lib.fm_paged_weights(*weigh_args(fm, cache=ctypes.byref(cache_of(fm, **change)))) == 1


def evict_args(fm, **kw):
    d = dict(cache=ctypes.byref(cache_of(fm)), R=4, width=10, lens=A, table=A, weights=A, budget=100, recent=10, sink=4, kept=A, new=2 * A, status=A)
    d.update(kw)
    return [*d.values(), None]


@pytest.mark.parametrize("change,code", [
    (dict(cache=None), 1), (dict(R=0), 1), (dict(R=8193), 2), (dict(width=0), 1), (dict(width=1 << 26), 2), (dict(lens=None), 1), (dict(table=A + 2), 1), (dict(weights=None), 1),
    (dict(budget=0), 1), (dict(recent=-1), 1), (dict(sink=-1), 1), (dict(recent=97), 1), (dict(recent=2 ** 31 - 1, sink=2 ** 31 - 1), 1), (dict(kept=None), 1), (dict(new=None), 1),
    (dict(new=A), 1), (dict(status=None), 1)])
def test_evict_arguments_that_are_refused(fm, change, code):
    assert fm._lib.fm_paged_evict(*evict_args(fm, **change)) == code


@pytest.mark.parametrize("change,code", [
    (dict(R=0), 1), (dict(R=8193), 2), (dict(width=0), 1), (dict(P=0), 1), (dict(page=0), 1), (dict(page=24), 2), (dict(page=65552), 2), (dict(width=1 << 26), 2),
    (dict(held=None), 1), (dict(lens=A + 2), 1), (dict(table=None), 1), (dict(n=-1), 1), (dict(free=A + 1), 1), (dict(head=None), 1), (dict(next=None), 1), (dict(seq=None), 1),
    (dict(status=None), 1)])
def test_release_arguments_that_are_refused(fm, change, code):
    d = dict(R=4, width=10, P=40, page=32, held=A, lens=A, table=A, free=A, n=40, head=A, next=A, seq=A, status=A)
    assert fm._lib.fm_paged_release(*{**d, **change}.values(), None) == code


@pytest.mark.parametrize("change,code", [
    (dict(target=None), 1), (dict(target=A + 2), 1), (dict(tr=99), 1), (dict(draft=A + 3), 1), (dict(dr=99), 1), (dict(dtype=2), 1), (dict(V=0), 1), (dict(rows=-1), 1),
    (dict(V=(1 << 24) + 1, tr=1 << 25, dr=1 << 25), 2), (dict(rows=(1 << 24) + 1), 2), (dict(tr=1 << 39), 1), (dict(tokens=None), 1), (dict(ua=A + 2), 1), (dict(us=None), 1),
    (dict(cu=None), 1), (dict(seq=None), 1), (dict(R=0), 1), (dict(R=8193), 2), (dict(out=None), 1), (dict(n_out=None), 1), (dict(new=A + 1), 1), (dict(status=None), 1)])
def test_verify_arguments_that_are_refused(fm, change, code):
    d = dict(target=A, tr=100, draft=A, dr=100, dtype=1, V=100, rows=8, tokens=A, ua=A, us=A, cu=A, seq=A, R=4, out=A, n_out=A, new=A, status=A)
    assert fm._lib.fm_verify_drafts(*{**d, **change}.values(), None) == code


def test_python_refuses_what_is_not_on_the_gpu(fm):
    rot = fm.Rotary(64, device="cpu")
    x, cache = torch.zeros(4, 2, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    i, l, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    step = step_of(fm)
    for call in (lambda: fm.fm_rope(x, i, rot), lambda: fm.fm_paged_append_rope(x, x, x, l, i, rot, cache, cache, i[:1]),
                 lambda: fm.fm_paged_weights(step, x, f, cache, i, l, 0.1, f, i[:1]), lambda: fm.fm_paged_evict(i, i.view(4, 1), cache, cache, f, 3, i[:1]),
                 lambda: fm.fm_paged_release(i, i, i.view(4, 1), 16, 4, None, None, i[:1]),
                 lambda: fm.fm_verify_drafts(f.view(4, 1), None, i, f, f, i, i[:3], i[:1])):
        with pytest.raises(TypeError):
            call()


def test_the_status_has_a_name(fm):
    assert "unknown" not in fm.fm_status_string(fm.FM_ERR_PROBS)
