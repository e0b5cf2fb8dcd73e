"""Paged-cache operators on the GPU against 64-bit references (paged_ref states the bounds)."""
import numpy as np
import pytest
import torch

import paged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    from long_context_fm_gb300 import fm as mod
    return mod


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Batch:
    """Requests with cached tokens, their pages in random order, every place that no row attends filled with NaN."""

    def __init__(self, fm, ctx, new, Hq, Hkv, d, page, window=0, sink=0, e4m3=False, seed=0, layout="heads", q_max=None, spare=2,
                 q_scale=1.5, poison=True):
        many = max(new) * (Hq // Hkv) > 32
        g = torch.Generator().manual_seed(seed)
        self.fm, self.ctx, self.new, self.scale = fm, ctx, new, 1.0 / d ** 0.5
        self.Hq, self.Hkv, self.d, self.page, self.window, self.sink, self.e4m3 = Hq, Hkv, d, page, window, sink, e4m3
        R, T = len(ctx), sum(new)
        held = [-(-(c + n) // page) for c, n in zip(ctx, new)]
        P, self.max_pages = sum(held) + spare, max(max(held), 1) + 1
        order = torch.randperm(P, generator=g).tolist()
        self.table = [[-7] * self.max_pages for _ in range(R)]
        for r in range(R):
            for b in range(held[r]):
                self.table[r][b] = order.pop()
        k = torch.full((P, Hkv, page, d), float("nan"))
        v = k.clone()
        for r, (c, n) in enumerate(zip(ctx, new)):
            for j in range(c + n):
                b0 = j // page * page
                gone = b0 + page - 1 <= c - window and b0 >= sink if many else j <= c - window and j >= sink
                if window and n and poison and gone:
                    continue            # behind the window of every row (many rows: with its whole page)
                k[self.table[r][j // page], :, j % page] = torch.randn(Hkv, d, generator=g)
                v[self.table[r][j // page], :, j % page] = torch.randn(Hkv, d, generator=g)
        if window and poison:           # pages wholly behind the window may be gone
            for r, (c, n) in enumerate(zip(ctx, new)):
                for b in range(held[r]):
                    if (b + 1) * page - 1 <= c - window and b * page >= sink:
                        self.table[r][b] = -3
        self.kd = self.vd = None
        if e4m3:
            self.kd, self.vd = torch.tensor([0.0131], device="cuda"), torch.tensor([0.0109], device="cuda")
            to = lambda x, s: (x / s.cpu()).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
            kc, vc = to(k, self.kd), to(v, self.vd)
            self.k64, self.v64 = ref.e4m3_values(kc) * float(self.kd), ref.e4m3_values(vc) * float(self.vd)
        else:
            kc, vc = k.bfloat16(), v.bfloat16()
            self.k64, self.v64 = kc.double(), vc.double()
        if layout == "heads":
            self.k, self.v = kc.cuda(), vc.cuda()
        elif layout == "tokens":        # [P, page, Hkv, d] memory
            self.k, self.v = (x.cuda().transpose(1, 2).contiguous().transpose(1, 2) for x in (kc, vc))
        else:                           # keys and values of a token next to one another
            both = torch.stack([kc, vc], 3).cuda()
            self.k, self.v = both[:, :, :, 0], both[:, :, :, 1]
        wide = (torch.randn(max(T, 1), Hq + 3, d + 8, generator=g) * q_scale).bfloat16()
        self.q = wide.cuda()[:T, 1:Hq + 1, :d] if layout != "heads" else wide[:T, 1:Hq + 1, :d].contiguous().cuda()
        self.q64 = wide[:T, 1:Hq + 1, :d].double()
        self.att = fm.PagedAttention(R, Hq, Hkv, d, page, P, self.max_pages, max(T, 1) + 3, q_max or max(max(new), 1), window=window, sink=sink)
        self.dev_table = i32(self.table)
        self.att.plan(i32(ctx), i32(new), self.dev_table)

    def run(self, o_dtype, rows_behind=2):
        T = sum(self.new)
        q = torch.cat([self.q, torch.full((rows_behind, self.Hq, self.d), float("nan"), dtype=torch.bfloat16, device="cuda")]) if rows_behind else self.q
        o = torch.full((T + rows_behind, self.Hq, self.d), 77.0, dtype=o_dtype, device="cuda")
        lse = torch.full((T + rows_behind, self.Hq), 77.0, device="cuda")
        self.fm.fm_attn_paged(self.att.step, q, self.k, self.v, self.dev_table, self.att.plan_buffer, self.scale, o, lse, self.att.status,
                              self.kd, self.vd)
        torch.cuda.synchronize()
        self.att.check_status()
        assert (o[T:] == 77).all() and (lse[T:] == 77).all()
        return o[:T], lse[:T]

    def reference(self):
        return ref.attend(self.q64, self.k64, self.v64, self.table, self.ctx, self.new, self.scale, self.window, self.sink)

    def p_err(self, o_dtype, few=True):
        if self.e4m3:
            return 2.0 ** -11 if o_dtype == torch.bfloat16 else 2.0 ** -22
        return 2.0 ** -16 if few or o_dtype == torch.float32 else 2.0 ** -8

    def check(self, o_dtype, few=True):
        o, lse = self.run(o_dtype)
        return ref.check_attention(self.reference(), o, lse, self.d, self.p_err(o_dtype, few), self.e4m3, self.e4m3 and not few)


# ---- plan ---------------------------------------------------------------------------
PLANS = [
    dict(ctx=[0], new=[1], page=16), dict(ctx=[16], new=[1], page=16), dict(ctx=[15], new=[1], page=16), dict(ctx=[31, 32, 33], new=[0, 0, 0], page=32),
    dict(ctx=[0, 5, 0, 100, 16, 0], new=[7, 0, 0, 33, 16, 1], page=16), dict(ctx=[3] * 700, new=[1] * 700, page=32),
    dict(ctx=[0, 1000, 77], new=[5000, 1, 333], page=48), dict(ctx=[7, 2], new=[0, 9001], page=128), dict(ctx=list(range(1300)), new=[r % 9 for r in range(1300)], page=16),
]


@pytest.mark.parametrize("case", range(len(PLANS)))
@pytest.mark.parametrize("how", ["pool", "in place", "given"])
def test_plan(fm, case, how):
    c = PLANS[case]
    ctx, new, page = c["ctx"], c["new"], c["page"]
    R, T = len(ctx), sum(new)
    rng = np.random.default_rng(case)
    need = [-(-(a + b) // page) for a, b in zip(ctx, new)]
    have = [-(-a // page) for a in ctx]
    P, width = sum(need) + 5, max(need) + 2
    order = rng.permutation(P).tolist()
    table = [[-5] * width for _ in range(R)]
    for r in range(R):
        for b in range(have[r] if how != "given" else need[r]):
            table[r][b] = order.pop()
    free, head = [9999] * 3 + order, 3
    att = fm.PagedAttention(R, 8, 2, 64, page, P, width, max(T, 1) + 6, max(max(new), 1))
    d_ctx, d_table = i32(ctx), i32(table)
    if how == "given":
        att.plan(d_ctx, i32(new), d_table)
        want = ref.plan(ctx, new, table, page, P)
    else:
        d_head = i32([head])
        att.plan(d_ctx, i32(new), d_table, free_pages=i32(free), free_head=d_head, in_place=how == "in place")
        want = ref.plan(ctx, new, table, page, P, free, head)
        assert int((d_head if how == "in place" else att.free_next).item()) == want[5]
    att.check_status()
    assert d_table.tolist() == want[0]
    assert att.cu_q.tolist() == want[1]
    assert att.slots.tolist() == want[2] + [-1] * (att.slots.numel() - T)
    assert att.positions.tolist() == want[3] + [-1] * (att.slots.numel() - T)
    assert (d_ctx if how == "in place" else att.seq_lens).tolist() == want[4]
    if how != "in place":
        assert d_ctx.tolist() == ctx


@pytest.mark.parametrize("ctx,new,code", [([-1, 0], [1, 1], 10), ([0, 0], [1, -1], 10), ([0, 0], [9, 1], 10), ([0, 0], [8, 8], 10), ([60, 0], [5, 0], 10),
                                          ([0, 2 ** 31 - 1], [1, 8], 10), ([15, 16], [8, 7], 11)])
def test_plans_that_fail_hand_out_nothing(fm, ctx, new, code):
    att = fm.PagedAttention(2, 4, 4, 64, 16, 40, 4, 15, 8)       # 64 keys, 15 rows, chunks of 8
    table, before = i32([[1, 2, -1, -1], [3, 4, -1, -1]]), [[1, 2, -1, -1], [3, 4, -1, -1]]
    att.plan(i32(ctx), i32(new), table, free_pages=i32([7]), free_head=i32([0]))
    assert int(att.status.item()) == code
    assert table.tolist() == before and att.cu_q.tolist() == [0, 0, 0] and int(att.free_next.item()) == 0
    assert (att.slots == -1).all() and att.seq_lens.tolist() == ctx
    # The empty plan writes nothing.
    cache = torch.zeros(40, 4, 16, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.ones(15, 4, 64, dtype=torch.bfloat16, device="cuda")
    att.append(x, x, cache, cache)
    o, lse = torch.full_like(x, 5.0), torch.full((15, 4), 5.0, device="cuda")
    fm.fm_attn_paged(att.step, x, cache, cache, table, att.plan_buffer, 0.1, o, lse, att.status)
    assert (cache == 0).all() and (o == 5).all() and (lse == 5).all()


@pytest.mark.parametrize("head,n_free", [(-1, 4), (5, 4), (2, 2)])
def test_free_list_heads_out_of_range(fm, head, n_free):
    att = fm.PagedAttention(1, 4, 4, 64, 16, 40, 4, 8, 8)
    att.plan(i32([0]), i32([1]), i32([[-1] * 4]), free_pages=i32(list(range(n_free))), free_head=i32([head]))
    assert int(att.status.item()) == fm.FM_ERR_PAGES and int(att.free_next.item()) == head


def test_a_free_page_outside_the_pool(fm):
    att = fm.PagedAttention(2, 4, 4, 64, 16, 40, 4, 8, 8)
    table = i32([[-1] * 4, [-1] * 4])
    att.plan(i32([0, 0]), i32([2, 2]), table, free_pages=i32([40, 5]), free_head=i32([0]))
    assert int(att.status.item()) == fm.FM_ERR_PAGES
    assert att.slots.tolist() == [-1, -1, 80, 81] + [-1] * 4


@pytest.mark.parametrize("new,code", [([0, 3], 0), ([1, 0], 11)])
def test_an_empty_free_list(fm, new, code):
    """No page is left: steps that need none go on, others fail, whatever the table holds behind the tokens."""
    att = fm.PagedAttention(2, 4, 4, 64, 16, 40, 4, 8, 8)
    table = i32([[1, 2, 3, 4], [5, 6, 7, 8]])
    att.plan(i32([16, 10]), i32(new), table, free_pages=torch.empty(0, dtype=torch.int32, device="cuda"), free_head=i32([0]))
    assert int(att.status.item()) == code and int(att.free_next.item()) == 0
    assert att.slots.tolist() == ([90, 91, 92] + [-1] * 5 if code == 0 else [-1] * 8)


@pytest.mark.parametrize("pages,code", [(4090, 0), (4097, 10)])
def test_more_key_tiles_than_31_bits(fm, pages, code):
    """Tables may name a page again and again: 512 tiles of 128 keys a page, 1024 KV heads."""
    att = fm.PagedAttention(1, 1024, 1024, 64, 65536, 1, 4100, 1, 1)
    att.plan(i32([pages * 65536 - 1]), i32([1]), torch.zeros(1, 4100, dtype=torch.int32, device="cuda"))
    assert int(att.status.item()) == code
    header = att.plan_buffer[:256].view(torch.int32).tolist()      # the sizes of the step, then n_few, ctas_few, tiles (64 bits)
    assert header[12:14] == ([1, 152] if code == 0 else [0, 0])
    assert att.plan_buffer[:256].view(torch.int64)[7] == (pages * 512 * 1024 if code == 0 else 0)


# ---- append --------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("T", [1, 2, 77, 1500])
@pytest.mark.parametrize("e4m3", [False, True])
def test_append(fm, d, Hkv, T, e4m3):
    page, P = 48, 40
    g = torch.Generator(device="cuda").manual_seed(T)
    slots = torch.randperm(P * page, generator=g, device="cuda")[:T]
    slots[T // 2::7] = -1
    kv = torch.randn(T, 2 * Hkv + 1, d + 8, generator=g, device="cuda").bfloat16() * 3
    kv[0, 0, 0], kv[0, 0, 1] = 7000.0, -1e-4
    k, v = kv[:, :Hkv, :d], kv[:, Hkv:2 * Hkv, :d]
    shape = (P, Hkv, page, d)
    kc = torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8) if e4m3 else torch.randn(shape, generator=g, device="cuda").bfloat16()
    vc = kc.flip(0).transpose(1, 2).contiguous().transpose(1, 2)        # tokens before heads in memory
    want_k, want_v = kc.clone(), vc.clone()
    kd, vd = torch.tensor([0.02], device="cuda"), torch.tensor([0.7], device="cuda")
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            for c, x, ds in ((want_k, k, kd), (want_v, v, vd)):
                c[s // page, :, s % page] = (x[t].float() / ds).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else x[t]
    status = i32([0])
    fm.fm_paged_append(k, v, slots, kc, vc, status, kd if e4m3 else None, vd if e4m3 else None)
    assert int(status.item()) == 0
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


def test_append_slots_outside_the_pool(fm):
    kc = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc, x, status = torch.zeros_like(kc), torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda"), i32([0])
    fm.fm_paged_append(x, x, torch.tensor([48, 3, 2 ** 40], device="cuda"), kc, vc, status)
    assert int(status.item()) == fm.FM_ERR_PAGES
    assert float(kc.sum()) == 2 * 64 and (kc[0, :, 3] == 1).all() and float(vc.sum()) == 2 * 64


def test_append_writes_nan_and_infinity(fm):
    kc = torch.zeros(1, 1, 16, 64, dtype=torch.uint8, device="cuda")
    vc, status, one = torch.zeros_like(kc), i32([0]), torch.ones(1, device="cuda")
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 0], x[0, 0, 1], x[0, 0, 2] = float("nan"), float("inf"), -float("inf")
    fm.fm_paged_append(x, x, torch.tensor([5], device="cuda"), kc, vc, status, one, one)
    got = kc[0, 0, 5].view(torch.float8_e4m3fn).float()
    assert got[0].isnan() and got[1] == 448 and got[2] == -448


@pytest.mark.parametrize("descale", [1.0, 0.02, 0.0131, 1 / 3, 0.7, 448.0, 1.9999999, 3e-24, 5e-25, 1e-38, 7e23, 1e30, 1.17e-38])
def test_append_rounds_every_value_as_a_division_does(fm, descale):
    """All 65,536 bf16 values: the codes are those of the fp32 quotient, saturated."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).cuda().view(1024, 1, 64)
    kc = torch.zeros(64, 1, 16, 64, dtype=torch.uint8, device="cuda")
    vc, status, ds = torch.zeros_like(kc), i32([0]), torch.tensor([descale], device="cuda")
    fm.fm_paged_append(x, x, torch.arange(1024, device="cuda"), kc, vc, status, ds, ds)
    q = x.float() / ds
    want = q.clamp(-448, 448).to(torch.float8_e4m3fn)
    got = kc.view(1024, 64).view(torch.float8_e4m3fn)
    assert torch.equal(got.float().isnan(), q.view(1024, 64).isnan()) and torch.equal(kc, vc)
    fine = ~q.view(1024, 64).isnan()
    assert torch.equal(got.view(torch.uint8)[fine], want.view(1024, 64).view(torch.uint8)[fine])


# ---- attention of few rows --------------------------------------------------------------
FEW = [
    # ctx, new, Hq, Hkv, page, window, sink
    ([0], [1], 4, 4, 16, 0, 0),
    ([15, 16, 17, 0, 127, 128, 129], [1] * 7, 8, 2, 16, 0, 0),
    ([1000, 3, 517], [1, 0, 1], 12, 4, 48, 0, 0),
    ([700], [1], 16, 1, 32, 0, 0),
    ([2200], [1], 2, 2, 128, 0, 0),
    ([300, 44, 0, 1023, 9], [4, 1, 2, 3, 4], 12, 4, 32, 0, 0),
    ([250, 5], [8, 8], 8, 2, 16, 0, 0),
    ([130, 600, 2], [1, 1, 1], 28, 4, 64, 0, 0),
    ([640], [1], 32, 1, 16, 0, 0),
    ([500, 20, 131, 128], [1, 1, 1, 1], 8, 8, 16, 100, 0),
    ([1500, 40, 131, 60], [2, 3, 1, 5], 8, 4, 32, 64, 10),
    ([900, 900], [6, 1], 10, 2, 16, 1, 0),
    ([700, 700], [3, 1], 4, 4, 64, 130, 200),
    ([260], [1], 3, 3, 256, 200, 1000),
]


@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", range(len(FEW)))
def test_few_rows(fm, case, d, e4m3, o_dtype):
    ctx, new, Hq, Hkv, page, window, sink = FEW[case]
    b = Batch(fm, ctx, new, Hq, Hkv, d, page, window, sink, e4m3, seed=case, layout=["heads", "tokens", "pairs"][case % 3])
    b.check(o_dtype)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_long_request_is_split_over_all_ctas(fm, e4m3):
    b = Batch(fm, [40000, 1], [1, 2], 2, 1, 64, 64, e4m3=e4m3, seed=5)
    b.check(torch.float32)
    o, lse = b.run(torch.float32)
    again = b.run(torch.float32)
    for x, y in zip((o, lse), again):                   # the same bits, whichever CTA comes last
        assert torch.equal(x.view(torch.int32), y.view(torch.int32))


# ---- attention of many rows ----------------------------------------------------------------
MANY = [
    # ctx, new, Hq, Hkv, page, window, sink
    ([0], [33], 1, 1, 16, 0, 0),
    ([0], [128], 2, 2, 16, 0, 0),
    ([0, 0, 0], [127, 129, 256], 2, 1, 32, 0, 0),
    ([500, 3, 0, 1000], [40, 1, 0, 130], 8, 2, 16, 0, 0),
    ([77], [61], 28, 4, 64, 0, 0),
    ([300, 128, 9], [70, 2, 65], 6, 2, 48, 0, 0),
    ([1000], [64], 4, 4, 128, 200, 0),
    ([900, 20], [150, 100], 2, 2, 32, 64, 10),
    ([900, 400], [100, 37], 4, 2, 16, 300, 140),
    ([2500], [45], 2, 2, 256, 0, 0),
    ([640, 255], [3, 5], 32, 1, 16, 0, 0),
    ([100], [90], 5, 5, 16, 1, 0),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,q_max", [(64, 8), (128, 8), (128, 34), (64, 4), (128, 4)])
def test_requests_of_few_and_fewer_rows(fm, e4m3, o_dtype, d, q_max):
    """4 to 32 rows beside one another, each unit's keys over several CTAs: parts of a unit computed in different ways."""
    new = [1, 8, 2, 4, 0, 3, 1, 5, 1, 8] if q_max >= 8 else [1, 4, 2, 4, 0, 3, 1, 2, 1, 4]
    b = Batch(fm, [2100, 1777, 300, 1290, 50, 2047, 3, 900, 1600, 0], new, 12, 3, d, 16, e4m3=e4m3, seed=5, q_max=q_max)
    b.check(o_dtype)


@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_rows(fm, case, d, e4m3, o_dtype):
    ctx, new, Hq, Hkv, page, window, sink = MANY[case]
    b = Batch(fm, ctx, new, Hq, Hkv, d, page, window, sink, e4m3, seed=100 + case, layout=["heads", "tokens", "pairs"][case % 3])
    b.check(o_dtype, few=False)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_short_chunk_over_a_long_cache_is_split(fm, e4m3):
    b = Batch(fm, [9000, 700], [20, 17], 4, 2, 128, 32, e4m3=e4m3, seed=6)
    b.check(torch.float32, few=False)
    first, again = b.run(torch.float32), b.run(torch.float32)
    for x, y in zip(first, again):
        assert torch.equal(x.view(torch.int32), y.view(torch.int32))


def test_many_units_of_every_length(fm):
    """More units than CTAs, whole and uneven."""
    rng = np.random.default_rng(3)
    ctx, new = rng.integers(0, 300, 40).tolist(), rng.integers(0, 90, 40).tolist()
    Batch(fm, ctx, new, 8, 8, 64, 16, seed=7).check(torch.bfloat16, few=False)


def test_short_units_of_scaled_rows_over_e4m3(fm):
    """One or two tiles a unit, nine or so per CTA, every row of q at a power of two of its own."""
    rng = np.random.default_rng(8)
    b = Batch(fm, rng.integers(0, 150, 90).tolist(), rng.integers(9, 70, 90).tolist(), 32, 8, 128, 16, e4m3=True, seed=8)
    f = torch.exp2(torch.randint(-12, 3, b.q.shape[:2], generator=torch.Generator().manual_seed(8)).double())[..., None]
    b.q64 = b.q64 * f
    b.q = (b.q.double() * f.cuda()).bfloat16()
    for o_dtype in (torch.bfloat16, torch.float32):
        first = b.run(o_dtype)
        b.check(o_dtype, few=False)
        for _ in range(3):
            for x, y in zip(first, b.run(o_dtype)):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("new", [[1, 2, 0], [70, 1, 9]])
def test_a_sink_without_a_window_changes_nothing(fm, new):
    a, b = (Batch(fm, [300, 40, 5], new, 8, 2, 64, 16, sink=sink, seed=9) for sink in (0, 7))
    for x, y in zip(a.run(torch.float32), b.run(torch.float32)):
        assert torch.equal(x, y)
    b.check(torch.float32, few=max(new) * 4 <= 32)


def test_as_many_requests_as_there_may_be(fm):
    b = Batch(fm, [r % 37 for r in range(8192)], [int(r % 3 > 0) for r in range(8192)], 2, 1, 64, 16, seed=10)
    b.check(torch.bfloat16)


def test_more_chunks_than_are_sorted(fm):
    """The planner sorts up to 512 chunks by their keys; more keep the requests' order."""
    b = Batch(fm, [r % 50 for r in range(700)], [9 + r % 7 if r % 8 else 1 for r in range(700)], 4, 1, 64, 16, seed=11)
    b.check(torch.bfloat16, few=False)
