"""Page numbers of a block table that no pool has, every one of them: attended ones read as zeros and
set the status, others are never looked at."""
import pytest
import torch

import paged_ref as ref

pytestmark = pytest.mark.gpu

PAGES = 6
OUTSIDE = [-1, -PAGES, -1 - PAGES, -2 - PAGES, PAGES, PAGES + 1, 2 ** 31 - 1, -2 ** 31]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def setting(fm, Hq, e4m3, ctx, new, table, window=0):
    g = torch.Generator(device="cuda").manual_seed(3)
    att = fm.PagedAttention(2, Hq, 2, 64, 16, PAGES, 3, 8, 4, window=window)
    kc, vc = (torch.randn(PAGES, 2, 16, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    one = torch.ones(1, device="cuda") if e4m3 else None
    if e4m3:
        kc, vc = (x.float().clamp(-400, 400).to(torch.float8_e4m3fn) for x in (kc, vc))
    q = torch.randn(sum(new), Hq, 64, generator=g, device="cuda").bfloat16()
    table = i32(table)
    att.plan(i32(ctx), i32(new), table)
    assert int(att.status.item()) == 0              # the bad pages hold no new token
    k0, v0 = (torch.cat([x.double(), torch.zeros_like(x[:1]).double()]).cpu() for x in (kc, vc))
    o, lse = att.attend(q, kc, vc, table, o_dtype=torch.float32, k_descale=one, v_descale=one)
    zeros = [[p if 0 <= p < PAGES else PAGES for p in row] for row in table.tolist()]
    want = ref.attend(q.double().cpu(), k0, v0, zeros, ctx, new, 0.125, window, 0)
    return att, o, lse, want


@pytest.mark.parametrize("page", OUTSIDE)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Hq", [4, 32])             # few rows; and many: 16 heads to a KV head, 4 tokens
def test_an_attended_page_outside_the_pool(Hq, e4m3, page):
    from long_context_fm_gb300 import fm
    att, o, lse, want = setting(fm, Hq, e4m3, [28, 20], [4, 1], [[page, 1, -1], [2, 3, -1]])
    assert int(att.status.item()) == fm.FM_ERR_PAGES
    ref.check_attention(want, o, lse, 64, 2.0 ** -22 if e4m3 else 2.0 ** -16, e4m3, e4m3 and Hq == 32)


@pytest.mark.parametrize("page", OUTSIDE)
@pytest.mark.parametrize("Hq", [4, 32])
def test_a_page_behind_the_window_may_be_anything(Hq, page):
    from long_context_fm_gb300 import fm
    att, o, lse, want = setting(fm, Hq, False, [28, 20], [4, 1], [[page, 1, page], [2, 3, page]], window=10)
    assert int(att.status.item()) == 0
    ref.check_attention(want, o, lse, 64, 2.0 ** -16, False)
