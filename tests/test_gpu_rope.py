"""Rotary positions on the GPU against 64-bit references (long_ref states the bounds)."""
import pytest
import torch

import long_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    from long_context_fm_gb300 import fm as mod
    return mod


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(got, want, tol, skip=None):
    half = ref.HALF[got.dtype]
    err, tol = (got.double().cpu() - want).abs(), tol * (1 + half) + half * want.abs() + 1e-37
    if skip is not None:
        err, tol = err[skip], tol[skip]
    assert (err <= tol).all(), f"worst error / bound {float((err / tol).max()):.3f}"


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("x_type,y_type", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16), (torch.float32, torch.float32),
                                           (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("B,H,N,d,rot", [(1, 1, 1, 64, 64), (2, 5, 37, 128, 128), (1, 9, 33, 64, 24), (3, 2, 16, 128, 8), (1, 3, 300, 128, 120)])
def test_rope(fm, B, H, N, d, rot, x_type, y_type, interleaved, inverse):
    g = torch.Generator().manual_seed(N)
    x = torch.randn(B, H, N, d, generator=g).to(x_type)
    pos = torch.randint(0, 200000, (B, N), generator=g, dtype=torch.int32)
    rot_ = fm.Rotary(rot, interleaved=interleaved)
    y = fm.fm_rope(x.cuda(), pos.cuda(), rot_, out_dtype=y_type, inverse=inverse)
    theta, m = ref.frequencies(rot)
    want, tol = ref.rope(x.double(), pos[:, None], theta, m, interleaved, inverse)
    assert y.dtype == y_type
    check(y, want, tol)
    if x_type == y_type:
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:])        # copied, not computed


@pytest.mark.parametrize("scaling,factor", [("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0), ("yarn", 1.0)])
def test_long_contexts(fm, scaling, factor):
    """Far positions, to the last int32."""
    g = torch.Generator().manual_seed(1)
    pos = torch.tensor([0, 1, 127, 4095, 131071, 2 ** 20, 2 ** 24 + 1, 10 ** 8 + 7, 2 ** 31 - 1], dtype=torch.int32)
    x = torch.randn(1, 2, len(pos), 128, generator=g)
    rot = fm.Rotary(128, scaling=scaling, factor=factor, original=8192, fast=16.0, slow=2.0)
    theta, m = ref.frequencies(128, scaling=scaling, factor=factor, original=8192, fast=16.0, slow=2.0)
    assert abs(rot.magnitude - m) <= 2.0 ** -24 * m
    want, tol = ref.rope(x.double(), pos[None, None], theta, m, False)
    check(fm.fm_rope(x.cuda(), pos.cuda(), rot), want, tol)


def test_a_magnitude_and_a_base_of_the_callers(fm):
    x = torch.randn(5, 3, 64)
    pos = torch.arange(5, dtype=torch.int32)
    rot = fm.Rotary(64, base=500000.0, magnitude=0.75)
    theta, _ = ref.frequencies(64, base=500000.0)
    want, tol = ref.rope(x.double(), pos[:, None], theta, 0.75, False)
    check(fm.fm_rope(x.cuda(), pos.cuda(), rot), want, tol)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_views_and_places(fm, interleaved):
    """Rows of a step inside a projection's output, in place and not, positions of a batch's own, and what is not written."""
    g = torch.Generator().manual_seed(2)
    wide = torch.randn(50, 7, 136, generator=g).bfloat16()
    pos = torch.randint(0, 9999, (50,), generator=g, dtype=torch.int32)
    pos[[3, 49]] = -1
    on = pos >= 0
    theta, m = ref.frequencies(96)
    rot = fm.Rotary(96, interleaved=interleaved)
    want, tol = ref.rope(wide[:, 2:6, :128].double(), pos.clamp_min(0)[:, None], theta, m, interleaved)
    a = wide.cuda()
    out = torch.full((50, 4, 128), 3.0, dtype=torch.float32, device="cuda")
    fm.fm_rope(a[:, 2:6, :128], pos.cuda(), rot, out=out)
    check(out, want, tol, on)
    assert (out[~on.cuda()] == 3).all() and torch.equal(a.cpu(), wide)
    fm.fm_rope(a[:, 2:6, :128], pos.cuda(), rot, out=a[:, 2:6, :128])
    check(a[:, 2:6, :128], want, tol, on)
    keep = a.cpu()
    keep[:, 2:6, :96][on] = wide[:, 2:6, :96][on]
    assert torch.equal(keep, wide)                                   # nothing beside the turned elements
    t = torch.randn(2, 30, 3, 64, generator=g).cuda().transpose(1, 2)  # tokens before heads
    rot = fm.Rotary(64, interleaved=interleaved)
    y = torch.empty(2, 3, 30, 64, device="cuda")
    fm.fm_rope(t, pos[:30].cuda(), rot, out=y)
    theta, m = ref.frequencies(64)
    want, tol = ref.rope(t.double().cpu(), pos[:30].clamp_min(0)[None, None], theta, m, interleaved)
    check(y, want, tol, (pos[:30] >= 0)[None, None].expand(2, 3, 30))


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_inverse_is_the_gradient(fm, interleaved):
    """Against differences: <fm_rope(x + e) - fm_rope(x - e), dy> / 2 = <e, fm_rope(dy, inverse)>, the map being linear; the bound is that of
    the values."""
    g = torch.Generator().manual_seed(3)
    x, e, dy = (torch.randn(2, 3, 20, 128, generator=g) for _ in range(3))
    pos = torch.randint(0, 5000, (20,), generator=g, dtype=torch.int32).cuda()
    rot = fm.Rotary(112, interleaved=interleaved, scaling="yarn", factor=4.0)
    run = lambda t, inverse=False: fm.fm_rope(t.cuda(), pos, rot, inverse=inverse).double().cpu()  # noqa: E731
    dx = run(dy, True)
    left = ((run(x + e) - run(x - e)) / 2 * dy.double()).sum((0, 1, 3))
    right = (e.double() * dx).sum((0, 1, 3))
    size = ((x.abs() + e.abs()).amax() * dy.abs().sum((0, 1, 3)) + e.abs().amax() * dy.abs().sum((0, 1, 3))).double()
    assert ((left - right).abs() <= 4 * rot.magnitude * (2.0 ** -21 + 2.0 ** -21) * size).all()


def test_positions_leave_products_to_distance(fm):
    """q at p + s times k at p depends on s alone."""
    g = torch.Generator().manual_seed(4)
    q, k = torch.randn(1, 1, 1, 128, generator=g), torch.randn(1, 1, 1, 128, generator=g)
    rot = fm.Rotary(128)
    at = lambda t, p: fm.fm_rope(t.cuda(), i32([p]), rot).double()  # noqa: E731
    want = float((at(q, 77) * at(k, 0)).sum())
    for p in (1, 1000, 10 ** 6, 10 ** 9):
        # Each turned element is within (|a| + |b|) (2^-21 + 2^-22 + 2^-50 p) of its own.
        tol = 4 * 4.0 * (2.0 ** -20 + 2.0 ** -49 * p) * float((q.abs().amax() * k.abs().sum() + k.abs().amax() * q.abs().sum()))
        assert abs(float((at(q, p + 77) * at(k, p)).sum()) - want) <= tol


# ---- into the cache ---------------------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,page", [(1, 1, 1, 64, 64, 16), (33, 32, 8, 128, 128, 64), (70, 5, 5, 64, 16, 32), (9, 12, 3, 128, 64, 16),
                                                 (700, 3, 1, 128, 128, 48)])
def test_append_rope(fm, T, Hq, Hkv, d, rot, page, e4m3, interleaved):
    g = torch.Generator().manual_seed(T)
    P = -(-T // page) + 2
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g).bfloat16()
    slots = torch.randperm(P * page, generator=g)[:T]
    pos = torch.randint(0, 10 ** 6, (T,), generator=g, dtype=torch.int32)
    if T > 5:
        slots[1], slots[4], pos[2] = -1, -7, -1
    on, stored = pos >= 0, (pos >= 0) & (slots >= 0)
    fill = torch.randint(0, 100, (P, Hkv, page, d), generator=g).to(torch.uint8 if e4m3 else torch.bfloat16)
    kc, vc = fill.cuda(), fill.cuda().clone()
    ds = [torch.tensor([x], device="cuda") for x in (0.0131, 0.0107)] if e4m3 else [None, None]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = qkv.cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    rot_ = fm.Rotary(rot, interleaved=interleaved, scaling="linear", factor=2.0)
    out = torch.full((T, Hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    fm.fm_paged_append_rope(q, k, v, slots.cuda(), pos.cuda(), rot_, kc, vc, status, q_out=out, k_descale=ds[0], v_descale=ds[1])
    assert int(status.item()) == 0 and torch.equal(x.cpu(), qkv)
    theta, m = ref.frequencies(rot, scaling="linear", factor=2.0)
    want, tol = ref.rope(qkv.double(), pos.clamp_min(0)[:, None], theta, m, interleaved)
    check(out, want[:, :Hq], tol[:, :Hq], on)
    assert (out[~on.cuda()] == 9).all()
    for cache, y, e, s in ((kc, want[:, Hq:Hq + Hkv], tol[:, Hq:Hq + Hkv], ds[0]), (vc, qkv[:, Hq + Hkv:].double(), torch.zeros(T, Hkv, d).double(), ds[1])):
        got = cache.cpu()
        at = slots[stored]
        new = got[at // page, :, at % page]
        if e4m3:
            f = float(s)
            new = new.view(torch.float8_e4m3fn).double()
            y, e = (y[stored] / f).clamp(-448, 448), e[stored] / f
            # half a step of the value, at least of the smallest step
            assert ((new - y).abs() <= e * (1 + 2.0 ** -4) + torch.maximum(y.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64)) + 2.0 ** -20 * y.abs()).all()
        else:
            y, e = y[stored], e[stored]
            assert ((new.double() - y).abs() <= e * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs()).all()
        left = fill.clone()
        left[at // page, :, at % page] = got[at // page, :, at % page]
        assert torch.equal(left, got)                                # every other slot as it was


def test_append_rope_is_rope_and_append(fm):
    """Bit for bit, over bf16 caches; in place; and over slots that are no slots."""
    g = torch.Generator().manual_seed(5)
    T, page, P = 40, 16, 5
    q, k, v = (torch.randn(T, h, 64, generator=g).bfloat16().cuda() for h in (6, 2, 2))
    slots, pos = torch.randperm(P * page, generator=g)[:T].cuda(), torch.randint(0, 9999, (T,), generator=g, dtype=torch.int32).cuda()
    rot = fm.Rotary(64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    caches = [[torch.zeros(P, 2, page, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    fm.fm_paged_append(fm.fm_rope(k, pos, rot), v, slots, *caches[0], status)
    want = fm.fm_rope(q, pos, rot)
    q2 = q.clone()
    assert fm.fm_paged_append_rope(q2, k, v, slots, pos, rot, *caches[1], status, q_out=q2) is q2
    assert torch.equal(q2, want) and all(torch.equal(a, b) for a, b in zip(*caches))
    bad = slots.clone()
    bad[7] = P * page
    before = [c.clone() for c in caches[1]]
    assert torch.equal(fm.fm_paged_append_rope(q, k, v, bad, pos, rot, *caches[1], status), want)
    assert int(status.item()) == fm.FM_ERR_PAGES and all(torch.equal(a, b) for a, b in zip(before, caches[1]))
