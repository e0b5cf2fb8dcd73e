"""The check of paged attention refuses a NaN wherever what a row attends is finite (no GPU is used)."""
import pytest
import torch

import paged_ref as ref
import paged_strict


def windowed(ctx, new, window, sink, page=16, Hq=2, Hkv=1, d=8):
    """Values behind every row's window are NaN; page numbers run through the requests."""
    g = torch.Generator().manual_seed(1)
    width = max(-(-(c + n) // page) for c, n in zip(ctx, new))
    table = [[r * width + b for b in range(width)] for r in range(len(ctx))]
    k, v = (torch.full((len(ctx) * width, Hkv, page, d), float("nan"), dtype=torch.float64) for _ in range(2))
    for r, (c, n) in enumerate(zip(ctx, new)):
        for j in range(c + n):
            if j > c - window or j < sink:
                for x in (k, v):
                    x[table[r][j // page], :, j % page] = torch.randn(Hkv, d, generator=g, dtype=torch.float64)
    q = torch.randn(sum(new), Hq, d, generator=g, dtype=torch.float64)
    return k, v, ref.attend(q, k, v, table, ctx, new, 0.3, window, sink)


@pytest.mark.parametrize("ctx,new,window,sink", [([500, 20, 131], [1, 1, 1], 100, 0), ([300, 40], [2, 3], 64, 10), ([200], [1], 1, 0)])
def test_a_nan_in_any_row_of_finite_keys_is_refused(ctx, new, window, sink):
    _, _, want = windowed(ctx, new, window, sink)
    assert torch.isfinite(want["o"]).all() and want["loose"].any()
    paged_strict.check_attention(want, new, want["o"].float(), want["lse"].float(), 8, 2.0 ** -16, False)
    for row in range(sum(new)):
        for head, col in ((0, 0), (1, 7)):
            o = want["o"].float()
            o[row, head, col] = float("nan")
            with pytest.raises(AssertionError):
                paged_strict.check_attention(want, new, o, want["lse"].float(), 8, 2.0 ** -16, False)


def test_a_nan_that_a_row_attends_excuses_its_column_in_the_request_alone():
    k, v, _ = windowed([40, 40], [2, 1], 100, 0)
    v[0, 0, 3, 5] = float("nan")
    g = torch.Generator().manual_seed(2)
    q = torch.randn(3, 2, 8, generator=g, dtype=torch.float64)
    want = ref.attend(q, k, v, [[0, 1, 2], [3, 4, 5]], [40, 40], [2, 1], 0.3, 100, 0)
    loose = paged_strict.attended_loose(want, [2, 1])
    assert loose[:2, :, 5].all() and int(loose.sum()) == 4
