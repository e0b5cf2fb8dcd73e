"""Rotary positions with frequencies of the caller's own, as a model needs that was stretched in another way than the table's."""
import math

import pytest
import torch

import long_ref as ref
from long_context_fm_gb300 import build as fmbuild


@pytest.fixture(scope="module")
def fm():
    fmbuild.build()
    from long_context_fm_gb300 import fm as mod
    return mod


def by_index(rot, base=10000.0, factor=8.0, original=4096, slow=1.0, fast=32.0):
    """Frequencies whose ramp is linear in the pair's index, between the pairs that turn `fast` and `slow` times within `original`."""
    pair = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
    out = []
    for i in range(rot // 2):
        r, theta = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))), base ** (-2.0 * i / rot)
        out.append(theta / factor * r + theta * (1 - r))
    return out


@pytest.mark.parametrize("rot", [8, 64, 128])
def test_the_table(fm, rot):
    theta = by_index(rot)
    theta[1], theta[2] = 0.0, 6.28
    for given in (theta, tuple(theta), torch.tensor(theta, dtype=torch.float64)):
        r = fm.Rotary(rot, frequencies=given, device="cpu")
        assert r.magnitude == 1.0 and r.turns.shape == (rot // 2,)
        for t, f in zip(r.turns.tolist(), theta):
            # Two roundings of a double (2^-53 each), and what a whole number of 2^-64 turns leaves off, less than one of them.
            assert abs((t % 2 ** 64) * 2.0 ** -64 - f / (2 * math.pi)) <= 2.0 ** -52 * f + 2.0 ** -64
    assert fm.Rotary(rot, frequencies=theta, magnitude=1.5, device="cpu").magnitude == 1.5


def test_the_two_ramps_differ(fm):
    """The table's is linear in the turns within the trained length: at pair 36 of 64 the other frequency is 2.3 times as large or small."""
    mine, _ = ref.frequencies(128, scaling="yarn", factor=8.0)
    other = torch.tensor(by_index(128), dtype=torch.float64)
    ratio = torch.maximum(mine / other, other / mine)
    assert int(ratio.argmax()) == 36 and 2.30 < float(ratio.max()) < 2.31


@pytest.mark.parametrize("bad", [[1.0] * 31, [1.0] * 33, [[1.0] * 32], [1.0] * 31 + [math.nan], [1.0] * 31 + [math.inf], [1.0] * 31 + [-0.1], [1.0] * 31 + [2 * math.pi]])
def test_what_is_refused(fm, bad):
    with pytest.raises(ValueError):
        fm.Rotary(64, frequencies=bad, device="cpu")
    with pytest.raises(ValueError):
        fm.Rotary(64, frequencies=by_index(64), scaling="yarn", factor=8.0, device="cpu")


@pytest.mark.gpu
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_turned_by_them(fm, interleaved, inverse):
    m, N, d = 0.1 * math.log(8.0) + 1.0, 300, 128
    theta = by_index(d)
    rot = fm.Rotary(d, interleaved=interleaved, frequencies=theta, magnitude=m)
    g = torch.Generator().manual_seed(2)
    x, pos = torch.randn(1, 3, N, d, generator=g).bfloat16(), torch.randint(0, 1 << 24, (N,), generator=g).int()
    want, tol = ref.rope(x.double(), pos, torch.tensor(theta, dtype=torch.float64), rot.magnitude, interleaved, inverse)
    got = fm.fm_rope(x.cuda(), pos.cuda(), rot, inverse=inverse).double().cpu()
    assert ((got - want).abs() <= tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()).all()
