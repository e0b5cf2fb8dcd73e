"""Attention weight of cached keys on the GPU against a 64-bit reference (long_ref states the bound)."""
import pytest
import torch

import long_ref as ref
import test_gpu_paged as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    from long_context_fm_gb300 import fm as mod
    return mod


def pool_of(b, seed=3):
    """Weights from earlier steps; NaN where new tokens will be, a mark everywhere else."""
    g = torch.Generator().manual_seed(seed)
    P = b.k.shape[0]
    w = torch.rand(P, b.Hkv, b.page, generator=g)
    for r, (c, n) in enumerate(zip(b.ctx, b.new)):
        for j in range(c, c + n):
            w[b.table[r][j // b.page], :, j % b.page] = float("nan")
    return w


def check(fm, b, lse=None, twice=False):
    rows = sum(b.new)
    if lse is None:
        _, lse = b.run(torch.float32)
    before = pool_of(b)
    pool = before.clone().cuda()
    q = torch.cat([b.q, torch.full((2, b.Hq, b.d), float("nan"), dtype=torch.bfloat16, device="cuda")])    # a padded batch
    z = torch.cat([lse, torch.full((2, b.Hq), float("nan"), device="cuda")])
    fm.fm_paged_weights(b.att.step, q, z, b.k, b.dev_table, b.att.plan_buffer, b.scale, pool, b.att.status, b.kd)
    b.att.check_status()
    terms = [r for r, n in enumerate(b.new) if n * (b.Hq // b.Hkv) <= 32] if b.e4m3 else []
    want, tol = ref.weights(b.q64, b.k64, lse.double().cpu(), before.double(), b.table, b.ctx, b.new, b.scale, b.window, b.sink, terms)
    got = pool.double().cpu()
    same = (tol == 0)
    assert torch.equal(torch.nan_to_num(got[same], nan=7.0), torch.nan_to_num(before.double()[same], nan=7.0))     # what no row attends
    err, tol = (got - want).abs()[~same], tol[~same]
    assert (err <= tol).all(), f"worst error / bound {float((err / tol).max()):.3f}"
    return pool


CASES = [
    dict(ctx=[0], new=[1], Hq=1, Hkv=1, page=16), dict(ctx=[1], new=[1], Hq=4, Hkv=4, page=16), dict(ctx=[127, 128, 129, 0], new=[1, 1, 1, 2], Hq=8, Hkv=2, page=32),
    dict(ctx=[300, 5, 0, 1000, 77], new=[3, 0, 1, 8, 2], Hq=8, Hkv=2, page=16), dict(ctx=[700, 200], new=[1, 4], Hq=14, Hkv=2, page=48),
    dict(ctx=[513, 40], new=[2, 1], Hq=16, Hkv=1, page=128), dict(ctx=[260], new=[1], Hq=32, Hkv=1, page=64),
    dict(ctx=[60] * 9, new=[1] * 9, Hq=10, Hkv=5, page=16),
    # more than 32 rows of a request
    dict(ctx=[0], new=[33], Hq=1, Hkv=1, page=16), dict(ctx=[0, 130], new=[200, 65], Hq=4, Hkv=2, page=32), dict(ctx=[300, 50, 7, 129], new=[150, 1, 40, 0], Hq=8, Hkv=2, page=16),
    dict(ctx=[1000], new=[128], Hq=14, Hkv=2, page=128), dict(ctx=[64], new=[300], Hq=5, Hkv=1, page=48), dict(ctx=[3], new=[700], Hq=2, Hkv=2, page=64),
    dict(ctx=[500, 0], new=[257, 129], Hq=32, Hkv=1, page=16),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_weights(fm, case, d, e4m3):
    check(fm, base.Batch(fm, d=d, e4m3=e4m3, seed=case, **CASES[case]))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window,sink", [(1, 0), (1, 3), (40, 0), (128, 4), (200, 130), (129, 17), (5000, 1)])
@pytest.mark.parametrize("new", [[1, 1, 2], [3, 0, 1], [150, 1, 60]])
def test_windows(fm, new, window, sink, e4m3):
    """Keys behind the window, NaN in places that no row attends, keep what they had."""
    check(fm, base.Batch(fm, [700, 333, 64], new, 8, 2, 128, 16, window=window, sink=sink, e4m3=e4m3, seed=window))


@pytest.mark.parametrize("d,e4m3", [(128, False), (64, False), (128, True), (64, True)])
@pytest.mark.parametrize("new", [[1, 2, 1], [60, 1, 200]])
def test_long_walks(fm, new, d, e4m3):
    """Dozens of tiles for every block: every stage comes round many times."""
    check(fm, base.Batch(fm, [20000, 9000, 14001], new, 16, 8, d, 64, e4m3=e4m3, seed=12))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window,sink", [(0, 0), (300, 5), (40, 0)])
@pytest.mark.parametrize("d", [64, 128])
def test_few_heads_of_many_rows(fm, d, window, sink, e4m3):
    """Few pairs of key tiles against dozens of row tiles: cut along the rows, and added up again; next to requests that are not."""
    check(fm, base.Batch(fm, [100, 700, 64], [1500, 40, 2], 8, 1, d, 32, window=window, sink=sink, e4m3=e4m3, seed=7))


def test_more_requests_of_many_rows_than_a_warp(fm):
    check(fm, base.Batch(fm, [60 * (r % 7) for r in range(45)], [33 + 9 * (r % 40) for r in range(45)], 2, 2, 64, 16, seed=8))


@pytest.mark.parametrize("layout", ["tokens", "pairs"])
@pytest.mark.parametrize("new", [[2, 1], [90, 1]])
def test_strides(fm, layout, new):
    check(fm, base.Batch(fm, [200, 31], new, 6, 2, 64, 32, layout=layout, seed=4))


def test_steps_add_up(fm):
    """Two layers' worth of rows over one plan: the second call adds to cached keys and begins new ones again."""
    b = base.Batch(fm, [300, 20], [1, 2], 8, 2, 64, 16)
    _, lse = b.run(torch.float32)
    one = torch.zeros(b.k.shape[:3], device="cuda")
    b.att.weigh(b.q, lse, b.k, b.dev_table, one, b.scale)
    two = one.clone()
    b.att.weigh(b.q, lse, b.k, b.dev_table, two, b.scale)
    for r, (c, n) in enumerate(zip(b.ctx, b.new)):
        for j in range(c + n):
            at = (b.table[r][j // b.page], slice(None), j % b.page)
            assert torch.equal(two[at], one[at] * (2 if j < c else 1))
    # Every row gives a weight of one to each query head.
    for r in range(2):
        own = sum(one[b.table[r][j // 16], :, j % 16].double() for j in range(b.ctx[r] + b.new[r]))
        assert torch.allclose(own, torch.full_like(own, 4.0 * b.new[r]), rtol=1e-5)


def test_a_call_repeats_itself(fm):
    b = base.Batch(fm, [3000, 1200, 70], [1, 300, 40], 8, 2, 128, 16, seed=6)
    _, lse = b.run(torch.float32)
    pools = []
    for _ in range(3):
        pool = torch.ones(b.k.shape[:3], device="cuda")
        b.att.weigh(b.q, lse, b.k, b.dev_table, pool, b.scale)
        pools.append(pool)
    assert torch.equal(pools[0], pools[1]) and torch.equal(pools[0], pools[2])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("new,row", [([3, 1], 1), ([100, 2], 40), ([300, 1], 130)])
def test_a_row_that_is_no_number(fm, new, row, window, e4m3):
    """Its weights reach the keys that it attends and no others: neither those behind it nor those behind its window."""
    b = base.Batch(fm, [200, 30], new, 8, 2, 128, 16, window=window, e4m3=e4m3, seed=9, poison=False)
    _, lse = b.run(torch.float32)

    def weigh(z):
        pool = torch.zeros(b.k.shape[:3], device="cuda")
        b.att.weigh(b.q, z, b.k, b.dev_table, pool, b.scale, b.kd)
        b.att.check_status()
        return [torch.stack([pool[b.table[r][j // 16], :, j % 16] for j in range(c + n)]) for r, (c, n) in enumerate(zip(b.ctx, b.new))]

    want, at = weigh(lse), b.ctx[0] + row
    j = torch.arange(b.ctx[0] + new[0], device="cuda")
    attended = (j <= at) & (j > at - window if window else j >= 0)
    for value in (float("nan"), float("-inf"), float("inf")):
        z = lse.clone()
        z[row] = value
        got = weigh(z)
        assert torch.equal(got[1], want[1]) and torch.equal(got[0][~attended], want[0][~attended])
        if value != value:
            assert got[0][attended].isnan().all()


@pytest.mark.parametrize("new", [[1, 2], [100, 1]])
def test_pages_outside_the_pool(fm, new):
    b = base.Batch(fm, [300, 20], new, 8, 2, 64, 16)
    _, lse = b.run(torch.float32)
    want = torch.zeros(b.k.shape[:3], device="cuda")
    b.att.weigh(b.q, lse, b.k, b.dev_table, want, b.scale)
    for value in (-1, b.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        table = [list(r) for r in b.table]
        gone, table[0][3] = table[0][3], value
        pool = torch.zeros_like(want)
        b.att.weigh(b.q, lse, b.k, base.i32(table), pool, b.scale)
        assert int(b.att.status.item()) == fm.FM_ERR_PAGES
        b.att.status.zero_()
        keep = want.clone()
        keep[gone] = 0
        assert torch.equal(pool, keep)


def test_a_plan_that_is_not_the_calls(fm):
    b = base.Batch(fm, [30, 20], [1, 2], 8, 2, 64, 16)
    _, lse = b.run(torch.float32)
    pool = torch.zeros(b.k.shape[:3], device="cuda")
    other = fm.PagedStep(*[getattr(b.att.step, n) for n, _ in fm.PagedStep._fields_])
    other.window = 5
    fm.fm_paged_weights(other, b.q, lse, b.k, b.dev_table, b.att.plan_buffer, b.scale, pool, b.att.status)
    assert int(b.att.status.item()) == fm.FM_ERR_PLAN_MISMATCH and (pool == 0).all()
    b.att.status.zero_()
    fm.fm_paged_weights(b.att.step, b.q[:2], lse[:2], b.k, b.dev_table, b.att.plan_buffer, b.scale, pool, b.att.status)
    assert int(b.att.status.item()) == fm.FM_ERR_LENGTHS and (pool == 0).all()
