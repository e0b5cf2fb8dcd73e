"""Softmax weights far below a row's largest over e4m3 caches: one key some 18 nats above a long flat tail.

fp16 holds the weights as 2^7 exp(s - m), m a maximum in force that is the row's largest score or up to 2^8
below it: a weight is rounded to 11 bits a term, and by half a step of 2^-24 at least, which is 2^-32 of the row's
largest weight: n 2^-32 max|v| on an output.  The rest of the bound is paged_ref's.
"""
import math

import pytest
import torch

import paged_ref as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(o, lse, want, A, zlse, n, S, d, p_err, floor):
    w = (2 * d + 8) * 2.0 ** -24 * (S + 1) + 2.0 ** -21
    out = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[o.dtype]
    tol = ((2 * w + p_err + n * 2.0 ** -24) * A + n * floor) * (1 + out) + out * want.abs()
    err = (o.double().cpu() - want).abs()
    assert (err <= tol).all(), f"o: worst error / bound {float((err / tol).max()):.3f}"
    ltol = w + n[:, :, 0] * 2.0 ** -24 + 2.0 ** -22 * (zlse.abs() + 1)
    lerr = (lse.double().cpu() - zlse).abs()
    assert (lerr <= ltol).all(), f"lse: worst error / bound {float((lerr / ltol).max()):.3f}"


@pytest.mark.parametrize("nats", [9.0, 18.0])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("new", [1, 5, 20, 33])     # 8, 16 and 32 rows a unit, and the many-rows kernel
@pytest.mark.parametrize("d", [64, 128])
def test_one_key_above_a_long_tail(d, new, e4m3, o_dtype, nats):
    from long_context_fm_gb300 import fm
    page, heads, ctx = 128, 152, 100_000        # as many heads as the kernels have CTAs, so that no unit is cut into short parts
    g = torch.Generator().manual_seed(3)
    q = torch.zeros(new, heads, d)
    q[:, :, 5] = 16.0
    k = torch.zeros(2, heads, page, d)          # page 0: the key above the rest; page 1: all further pages
    k[0, :, 0, 5] = nats / 2
    tail = torch.randint(1, 9, (heads, d), generator=g) / 8.0 * (torch.randint(0, 2, (heads, d), generator=g) * 2 - 1)
    top = tail.roll(1, 1) * (torch.arange(d) % 2)               # zero in half the columns: the tail alone is left there
    v = tail[None, :, None].repeat(2, 1, page, 1)
    v[0, :, 0] = top
    to = (lambda x: x.to(torch.float8_e4m3fn).cuda()) if e4m3 else (lambda x: x.bfloat16().cuda())
    one = torch.ones(1, device="cuda") if e4m3 else None
    width = -(-(ctx + new) // page)
    table = torch.ones(1, width, dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    att = fm.PagedAttention(1, heads, heads, d, page, 2, width, new, new)
    att.plan(i32([ctx]), i32([new]), table)
    o, lse = att.attend(q.bfloat16().cuda(), to(k), to(v), table, scale=0.125, o_dtype=o_dtype, k_descale=one, v_descale=one)
    att.check_status()
    n = torch.arange(ctx + 1, ctx + new + 1, dtype=torch.float64)[:, None, None]
    total = math.exp(nats) + n - 1
    want = (math.exp(nats) * top.double() + (n - 1) * tail.double()) / total
    A = (math.exp(nats) * top.double().abs() + (n - 1) * tail.double().abs()) / total
    if e4m3:
        p_err = 2.0 ** -22 if o_dtype == torch.float32 or new <= 8 else 2.0 ** -11
    else:
        p_err = 2.0 ** -16 if o_dtype == torch.float32 or new <= 32 else 2.0 ** -8
    check(o, lse, want, A, total.log()[:, :, 0].expand(new, heads), n, nats, d, p_err, 2.0 ** -32 if e4m3 else 0.0)
