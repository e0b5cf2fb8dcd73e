"""Eviction and release on the GPU: whole numbers and moved bits, so equal to the reference (long_ref)."""
import numpy as np
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


class Pool:
    def __init__(self, lens, Hkv, d, page, e4m3=False, layout="heads", seed=0, values="spread"):
        rng = np.random.default_rng(seed)
        self.lens, self.Hkv, self.d, self.page = lens, Hkv, d, page
        need = [-(-n // page) for n in lens]
        P, width = sum(need) + 3, max(need) + 2
        order = rng.permutation(P).tolist()
        self.table = [[-9] * width for _ in lens]
        for r, n in enumerate(need):
            for b in range(n):
                self.table[r][b] = order.pop()
        shape = (P, Hkv, page, d)
        bits = lambda: torch.from_numpy(rng.integers(0, 256, (*shape, 1 if e4m3 else 2), dtype=np.uint8))  # noqa: E731
        kv = [bits()[..., 0] if e4m3 else bits().view(torch.bfloat16)[..., 0] for _ in range(2)]     # any bits, NaN among them
        if layout == "heads":
            self.k, self.v = (x.cuda() for x in kv)
        elif layout == "tokens":
            self.k, self.v = (x.cuda().transpose(1, 2).contiguous().transpose(1, 2) for x in kv)
        else:
            both = torch.stack(kv, 3).cuda()
            self.k, self.v = both[:, :, :, 0], both[:, :, :, 1]
        self.k0, self.v0 = kv
        w = np.exp(rng.normal(size=shape[:3]) * 2).astype(np.float32)
        if values == "ties":
            w = rng.integers(0, 3, shape[:3]).astype(np.float32)
        if values == "equal":
            w[:] = 0.25
        if values == "odd":
            w = rng.choice(np.array([0.0, -0.0, 1e-40, -1e-40, -3.0, 2.0, np.inf, -np.inf, np.nan, 3e38], np.float32), shape[:3])
        if values == "near":            # differ in the last bits alone
            w = (np.float32(1.0).view(np.uint32) + rng.integers(0, 300, shape[:3]).astype(np.uint32)).view(np.float32)
        self.w0 = torch.from_numpy(w)
        self.w = self.w0.cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def expect(self, budget, recent, sink):
        k, v, w = self.k0.clone(), self.v0.clone(), self.w0.clone()
        kept = torch.full((len(self.lens), self.Hkv, budget), -1, dtype=torch.int32)
        new = []
        for r, n in enumerate(self.lens):
            new.append(min(n, budget))
            if n <= budget:
                continue
            for h in range(self.Hkv):
                of = [float(self.w0[self.table[r][j // self.page], h, j % self.page]) for j in range(n)]
                places = ref.kept_places(of, n, budget, recent, sink)
                kept[r, h] = torch.tensor(places, dtype=torch.int32)
                for to, j in enumerate(places):
                    a, b = (self.table[r][to // self.page], h, to % self.page), (self.table[r][j // self.page], h, j % self.page)
                    k[a], v[a], w[a] = self.k0[b], self.v0[b], self.w0[b]
        return k, v, w, kept, new

    def run(self, fm, budget, recent, sink, **kw):
        kept = torch.full((len(self.lens), self.Hkv, budget), 5, dtype=torch.int32, device="cuda")
        new = fm.fm_paged_evict(i32(self.lens), i32(self.table), self.k, self.v, self.w, budget, self.status, recent, sink, kept=kept, **kw)
        return kept, new

    def check(self, fm, budget, recent=0, sink=0):
        k, v, w, kept, new = self.expect(budget, recent, sink)
        got, lens = self.run(fm, budget, recent, sink)
        assert int(self.status.item()) == 0
        assert lens.tolist() == new
        assert torch.equal(got.cpu(), kept)
        raw = lambda x: x.cpu().contiguous().view(torch.uint8)  # noqa: E731
        assert torch.equal(raw(self.k), raw(k)) and torch.equal(raw(self.v), raw(v)) and torch.equal(raw(self.w), raw(w))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,budget,recent,sink", [
    ([2], 1, 0, 0), ([2], 1, 1, 0), ([2], 1, 0, 1), ([17], 16, 3, 2), ([100, 0, 7, 64, 65], 64, 8, 4), ([300, 1000], 100, 0, 0), ([300, 31], 32, 16, 16),
    ([513, 600, 90], 200, 199, 1), ([2500], 2000, 100, 4), ([1500, 1300], 129, 0, 129), ([777], 700, 700, 0)])
def test_evict(fm, lens, budget, recent, sink, d, e4m3):
    Pool(lens, 3, d, 16, e4m3, seed=len(lens) + budget).check(fm, budget, recent, sink)


@pytest.mark.parametrize("values", ["ties", "equal", "odd", "near"])
@pytest.mark.parametrize("lens,budget,recent,sink", [([50], 20, 3, 2), ([1000, 40, 700], 333, 10, 1), ([2100], 64, 0, 0)])
def test_weights_that_are_equal_or_odd(fm, values, lens, budget, recent, sink):
    Pool(lens, 2, 64, 32, values=values, seed=8).check(fm, budget, recent, sink)


@pytest.mark.parametrize("values", ["spread", "ties"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("R", [8, 9, 32, 33, 152, 153])
def test_many_requests(fm, R, e4m3, values):
    """More and more (request, head) pairs: fewer and fewer blocks share one."""
    Pool([(37 * r) % 400 for r in range(R)], 2, 64, 16, e4m3, seed=R, values=values).check(fm, 90, 11, 3)


@pytest.mark.parametrize("layout", ["tokens", "pairs"])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_strides_and_pages(fm, layout, page):
    Pool([400, 129, 250], 2, 64, page, layout=layout, seed=1).check(fm, 130, 20, 4)


def test_evict_again(fm):
    """Down to the budget, and further down."""
    p = Pool([900], 2, 64, 16, seed=2)
    p.check(fm, 500, 50, 4)
    p.k0, p.v0, p.w0, p.lens = p.k.cpu(), p.v.cpu(), p.w.cpu(), [500]
    p.check(fm, 77, 7, 2)


def test_many_places(fm):
    """More than a cluster holds in shared memory, against a vectorised reference."""
    n, budget, recent, sink, page, Hkv = 120007, 30011, 1000, 4, 64, 2
    pages = -(-n // page)
    g = torch.Generator().manual_seed(3)
    table = torch.randperm(pages, generator=g).int()
    w0 = torch.randint(0, 20000, (pages, Hkv, page), generator=g).float()                # with ties
    k0 = torch.randint(0, 256, (pages, Hkv, page, 64), generator=g, dtype=torch.uint8)
    k, w = k0.cuda(), w0.cuda()
    v = k.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = torch.empty(1, Hkv, budget, dtype=torch.int32, device="cuda")
    fm.fm_paged_evict(i32([n]), table[None].cuda(), k, v, w, budget, status, recent, sink, kept=kept)
    assert int(status.item()) == 0
    line = w0[table.long()].transpose(0, 1).reshape(Hkv, -1)
    for h in range(Hkv):
        best = torch.sort(line[h, sink:n - recent], descending=True, stable=True).indices[:budget - sink - recent] + sink
        places = torch.cat([torch.arange(sink), best.sort().values, torch.arange(n - recent, n)])
        assert torch.equal(kept[0, h].cpu().long(), places)
        for x, x0 in ((k, k0), (v, k0), (w, w0)):
            assert torch.equal(x.cpu()[table.long()][:, h].flatten(0, 1)[:budget], x0[table.long()][:, h].flatten(0, 1)[places])


def test_long_slices_are_read_again(fm):
    """One head of 300,000 tokens: a CTA's slice is longer than what it keeps in shared memory."""
    n, budget, page = 300001, 1000, 128
    pages = -(-n // page)
    g = torch.Generator().manual_seed(4)
    w0 = torch.rand(pages, 1, page, generator=g)
    k = torch.zeros(pages, 1, page, 64, dtype=torch.uint8, device="cuda")
    v, w = k.clone(), w0.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = torch.empty(1, 1, budget, dtype=torch.int32, device="cuda")
    fm.fm_paged_evict(i32([n]), torch.arange(pages, dtype=torch.int32, device="cuda")[None], k, v, w, budget, status, kept=kept)
    best = torch.sort(w0.flatten()[:n], descending=True, stable=True).indices[:budget].sort().values
    assert torch.equal(kept[0, 0].cpu().long(), best) and torch.equal(w.cpu().flatten()[:budget], w0.flatten()[best])


def test_requests_that_are_left_alone(fm):
    """A length or a page out of range: its request alone is left."""
    for bad in ("length", "long", "page", "last page"):
        p = Pool([200, 180, 150], 2, 64, 16, seed=6)
        lens, code = list(p.lens), fm.FM_ERR_LENGTHS
        k, v, w, kept, new = p.expect(64, 8, 2)
        if bad == "length":
            lens[1] = -1
        elif bad == "long":
            lens[1] = len(p.table[0]) * 16 + 1
        else:
            p.table[1][2 if bad == "page" else 180 // 16] = -1 if bad == "page" else p.k.shape[0]
            code = fm.FM_ERR_PAGES
        got = torch.zeros_like(kept).cuda()
        after = fm.fm_paged_evict(i32(lens), i32(p.table), p.k, p.v, p.w, 64, p.status, 8, 2, kept=got)
        assert int(p.status.item()) == code
        assert after.tolist() == [64, lens[1], 64]
        assert (got[1] == -1).all() and torch.equal(got.cpu()[[0, 2]], kept[[0, 2]])
        others = [x for r in (0, 2) for x in p.table[r][:-(-p.lens[r] // 16)]]
        mine = [x for x in range(p.k.shape[0]) if x not in others]
        assert torch.equal(p.w.cpu()[others], w[others]) and torch.equal(p.w.cpu()[mine], p.w0[mine])
        assert torch.equal(p.k.cpu()[others].view(torch.uint8), k[others].view(torch.uint8))
        assert torch.equal(p.k.cpu()[mine].view(torch.uint8), p.k0[mine].view(torch.uint8))


# ---- release -------------------------------------------------------------------------------
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("held,lens,page", [
    ([1], [0], 16), ([16, 17, 0], [16, 16, 0], 16), ([100, 50, 33, 1], [1, 50, 0, 1], 16), ([5000, 7], [4096, 7], 64), ([96] * 700, [33] * 700, 32),
    (list(range(1300)), [x // 2 for x in range(1300)], 16), ([70000], [3], 16)])
def test_release(fm, held, lens, page, in_place):
    rng = np.random.default_rng(len(held))
    need = [-(-n // page) for n in held]
    P, width = sum(need) + 4, max(need) + 1
    order = rng.permutation(P).tolist()
    free, head = list(order), sum(need)
    table, at = [[-3] * width for _ in held], 0
    for r, n in enumerate(need):
        table[r][:n] = order[at:at + n]
        at += n
    want, after = ref.released(held, lens, table, page, free, head)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d_held, d_free, d_head, d_table = i32(held), i32(free), i32([head]), i32(table)
    seq, nxt = fm.fm_paged_release(d_held, i32(lens), d_table, page, P, d_free, d_head, status, *((d_head, d_held) if in_place else ()))
    assert int(status.item()) == 0 and seq.tolist() == lens and nxt.tolist() == [after] and d_free.tolist() == want
    assert d_table.tolist() == table
    if not in_place:
        assert d_held.tolist() == held and d_head.tolist() == [head]


@pytest.mark.parametrize("held,lens,head,change,code", [
    ([40, 20], [41, 0], 4, None, 10), ([40, 20], [-1, 0], 4, None, 10), ([200, 20], [1, 0], 4, None, 10), ([-1, 20], [0, 0], 4, None, 10),
    ([40, 20], [0, 0], 4, None, 11), ([40, 20], [0, 0], -1, None, 11), ([40, 20], [0, 0], 10, None, 11), ([40, 20], [0, 0], 5, -1, 11),
    ([40, 20], [0, 0], 5, 9, 11)])
def test_releases_that_fail_give_nothing_back(fm, held, lens, head, change, code):
    table = [[0, 1, 2, -1], [3, 4, -1, -1]]
    if change is not None:
        table[1][1] = change
    free = i32([7] * 9)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seq, nxt = fm.fm_paged_release(i32(held), i32(lens), i32(table), 16, 9, free, i32([head]), status)
    assert int(status.item()) == code and seq.tolist() == held and nxt.tolist() == [head] and (free == 7).all()


def test_lengths_alone(fm):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seq, nxt = fm.fm_paged_release(i32([40, 20]), i32([3, 20]), i32([[-1] * 4] * 2), 16, 9, None, None, status)
    assert int(status.item()) == 0 and seq.tolist() == [3, 20] and nxt is None


def test_what_is_given_back_is_taken_again(fm):
    """Plan, release, plan: the pages come back in the order in which they were given."""
    att = fm.PagedAttention(2, 4, 4, 64, 16, 20, 8, 128, 100)
    lens, table, free, head = i32([0, 0]), i32([[-1] * 8] * 2), i32(list(range(20))), i32([0])
    att.plan(lens, i32([70, 40]), table, free_pages=free, free_head=head, in_place=True)
    assert table.tolist() == [[0, 1, 2, 3, 4, -1, -1, -1], [5, 6, 7, -1, -1, -1, -1, -1]] and head.tolist() == [8]
    att.release(lens, i32([20, 40]), table, free, head, in_place=True)
    assert lens.tolist() == [20, 40] and head.tolist() == [5] and free.tolist()[5:9] == [2, 3, 4, 8]
    att.plan(lens, i32([1, 60]), table, free_pages=free, free_head=head, in_place=True)
    att.check_status()
    assert table.tolist()[1] == [5, 6, 7, 2, 3, 4, 8, -1] and lens.tolist() == [21, 100] and head.tolist() == [9]
