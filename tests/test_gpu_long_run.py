"""Rotary, weights, eviction, verification and release as they are used together: a serving loop whose caches stay bounded,
checked against 64 bits step by step; captured and replayed; on another stream; past 32-bit offsets."""
import pytest
import torch

import long_ref
import paged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    from long_context_fm_gb300 import fm as mod
    return mod


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """Two layers, three requests; tokens drafted ahead, caches cut down to a budget."""

    def __init__(self, fm, e4m3, d=64, budget=70, max_q=100):
        self.fm, self.R, self.Hq, self.Hkv, self.d, self.page, self.P, self.width, self.V = fm, 3, 6, 2, d, 16, 40, 14, 50
        self.e4m3, self.budget, self.recent, self.sink = e4m3, budget, 20, 3
        self.g = torch.Generator().manual_seed(21)
        shape = (self.P, self.Hkv, self.page, d)
        self.caches = [[torch.full(shape, 127, dtype=torch.uint8, device="cuda") if e4m3 else torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
                        for _ in range(2)] for _ in range(2)]
        self.weights = [torch.full(shape[:3], float("nan"), device="cuda") for _ in range(2)]
        self.ds = torch.tensor([0.017], device="cuda") if e4m3 else None
        self.rot = fm.Rotary(d, scaling="yarn", factor=4.0)
        self.att = fm.PagedAttention(self.R, self.Hq, self.Hkv, d, self.page, self.P, self.width, 160, max_q)
        self.free, self.head = i32(torch.randperm(self.P, generator=self.g).tolist()), i32([0])
        self.lens, self.table = i32([0] * self.R), i32([[-1] * self.width] * self.R)
        self.cut_lens = i32([0] * self.R)
        self.past = [0] * self.R                    # tokens of each conversation, evicted ones among them
        self.said = [[] for _ in range(self.R)]

    def inputs(self, new):
        T, g = sum(new), self.g
        xs = [[torch.randn(T, h, self.d, generator=g).bfloat16() for h in (self.Hq, self.Hkv, self.Hkv)] for _ in range(2)]
        p = torch.softmax(torch.randn(T, self.V, generator=g), 1)
        q = torch.softmax(p.log() + 0.5 * torch.randn(T, self.V, generator=g), 1)
        tokens = torch.multinomial(q, 1, generator=g)[:, 0].roll(1).int()
        return xs, p, q, tokens, torch.rand(T, generator=g), torch.rand(self.R, generator=g)

    def held(self, layer, r, n):
        """Cached keys, values (double) and weights of request r, [Hkv, n, ...]."""
        pages = self.table[r, :-(-n // self.page)].long()
        out = []
        for c in (*self.caches[layer], self.weights[layer]):
            x = c[pages].transpose(0, 1).flatten(1, 2)[:, :n].cpu()
            out.append(ref.e4m3_values(x) * float(self.ds) if x.dtype == torch.uint8 else x.double())
        return out

    def step(self, new, drafts):
        """new[r] rows of each request; with drafts all but the first of them are drafted."""
        fm, att, page = self.fm, self.att, self.page
        xs, p, q, tokens, ua, us = self.inputs(new)
        ctx = self.lens.tolist()
        before = [[self.held(layer, r, ctx[r]) for r in range(self.R)] for layer in range(2)]
        positions = [self.past[r] + i for r, n in enumerate(new) for i in range(n)]
        att.plan(self.lens, i32(new), self.table, free_pages=self.free, free_head=self.head, in_place=True)
        theta, m = long_ref.frequencies(self.d, scaling="yarn", factor=4.0)
        seq = self.lens.tolist()
        assert seq == [c + n for c, n in zip(ctx, new)]
        for layer, (qx, k, v) in enumerate(xs):
            kc, vc = self.caches[layer]
            turned = att.append_rope(qx.cuda(), k.cuda(), v.cuda(), self.rot, kc, vc, positions=i32(positions), k_descale=self.ds, v_descale=self.ds)
            o, lse = att.attend(turned, kc, vc, self.table, o_dtype=torch.float32, k_descale=self.ds, v_descale=self.ds)
            att.weigh(turned, lse, kc, self.table, self.weights[layer], k_descale=self.ds)
            att.check_status()
            # What was held is as it was; new keys are the turned ones; attention and weights are those over what is held.
            want_k, tol = long_ref.rope(k.double(), torch.tensor(positions)[:, None], theta, m, False)
            half = 2.0 ** -4 if self.e4m3 else 2.0 ** -8
            t0 = 0
            for r, n in enumerate(new):
                hk, hv, hw = self.held(layer, r, seq[r])
                for x, y in zip((hk, hv), before[layer][r]):
                    assert torch.equal(x[:, :ctx[r]], y)
                for x, y, e in ((hk, want_k, tol), (hv, v.double(), torch.zeros_like(tol))):
                    y, e = y[t0:t0 + n].transpose(0, 1), e[t0:t0 + n].transpose(0, 1)
                    step = 2.0 ** -9 * float(self.ds) if self.e4m3 else 0.0
                    assert ((x[:, ctx[r]:] - y).abs() <= e * (1 + half) + half * y.abs() * (1 + 2.0 ** -20) + step).all()
                if n:
                    line = [x.transpose(0, 1)[:, :, None] for x in (hk, hv)]      # a page per key
                    qq = turned[t0:t0 + n].double().cpu()
                    want = ref.attend(qq, *line, [list(range(seq[r]))], [ctx[r]], [n], self.d ** -0.5)
                    many = n * 3 > 32
                    ref.check_attention(want, o[t0:t0 + n], lse[t0:t0 + n], self.d, 2.0 ** -22 if self.e4m3 else 2.0 ** -16, self.e4m3, self.e4m3 and many)
                    old = torch.nan_to_num(before[layer][r][2]).transpose(0, 1)[:, :, None]
                    old = torch.cat([old, torch.zeros(n, self.Hkv, 1)])
                    w, e = long_ref.weights(qq, line[0], lse[t0:t0 + n].double().cpu(), old, [list(range(seq[r]))], [ctx[r]], [n], self.d ** -0.5,
                                            q_terms=[0] if self.e4m3 and not many else ())
                    assert ((hw.transpose(0, 1)[:, :, None] - w).abs() <= e).all()
                t0 += n
        if drafts:
            cu = att.cu_q.tolist()
            out, n_out, kept = att.verify(p.cuda(), q.cuda(), tokens.cuda(), ua.cuda(), us.cuda(), seq_lens=self.lens)
            want, count = long_ref.verify(p.double(), q.double(), tokens.tolist(), ua.double().tolist(), us.double().tolist(), cu)
            assert out.tolist() == want and n_out.tolist() == count
            self.give_back(kept, [s - n + c for s, n, c in zip(seq, new, count)])
            for r, c in enumerate(count):
                self.past[r] += c
                self.said[r] += want[cu[r]:cu[r] + c]
        else:
            self.past = [a + n for a, n in zip(self.past, new)]
        self.evict()

    def evict(self):
        lens = self.lens.tolist()
        if max(lens) <= self.budget:
            return
        want = [min(n, self.budget) for n in lens]
        for layer in range(2):
            before = [self.held(layer, r, lens[r]) for r in range(self.R)]
            kept = torch.empty(self.R, self.Hkv, self.budget, dtype=torch.int32, device="cuda")
            self.att.evict(self.lens, self.table, *self.caches[layer], self.weights[layer], self.budget, self.recent, self.sink, kept=kept, new_lens=self.cut_lens)
            for r in range(self.R):
                after = self.held(layer, r, want[r])
                for h in range(self.Hkv):
                    places = long_ref.kept_places(before[r][2][h].tolist(), lens[r], self.budget, self.recent, self.sink) if lens[r] > self.budget else list(range(lens[r]))
                    assert all(torch.equal(x[h], y[h, places]) for x, y in zip(after, before[r]))
                    assert lens[r] <= self.budget or kept[r, h].tolist() == places
        self.give_back(self.cut_lens, want)

    def give_back(self, lens, want):
        held, free, head = self.lens.tolist(), self.free.tolist(), int(self.head)
        expect, at = long_ref.released(held, want, self.table.tolist(), self.page, free, head)
        self.att.release(self.lens, lens, self.table, self.free, self.head, in_place=True)
        self.att.check_status()
        assert self.lens.tolist() == want and self.free.tolist() == expect and self.head.tolist() == [at]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_a_bounded_conversation(fm, d, e4m3):
    s = Server(fm, e4m3, d)
    s.step([60, 0, 5], False)
    s.step([1, 90, 100 - 60], False)        # two prompts past the budget
    for new in ([3, 2, 1], [4, 4, 4], [1, 0, 5], [5, 5, 5], [2, 30, 2], [3, 3, 3]):
        s.step(new, True)
    assert all(len(x) > 2 for x in s.said) and max(s.lens.tolist()) <= s.budget < max(s.past)


def test_captured_and_on_another_stream(fm):
    """A whole step (plan, append, attention, weights, verification, eviction, releases) captured once and replayed gives the bits of the
    calls made one by one, on a stream of its own."""
    def build():
        s = Server(fm, False)
        s.xs = [[torch.zeros(12, h, 64, dtype=torch.bfloat16, device="cuda") for h in (6, 2, 2)] for _ in range(2)]
        s.p, s.q = torch.zeros(12, 50, device="cuda"), torch.zeros(12, 50, device="cuda")
        s.tokens, s.ua, s.us, s.kept = i32([0] * 12), torch.zeros(12, device="cuda"), torch.zeros(3, device="cuda"), i32([0] * 3)
        s.new, s.positions = i32([4] * 3), i32([0] * 12)
        s.weights = [torch.zeros_like(w) for w in s.weights]
        return s

    def fill(s, seed):
        s.g = torch.Generator().manual_seed(seed)
        xs, p, q, tokens, ua, us = s.inputs([4] * 3)
        for a, b in zip([*s.xs[0], *s.xs[1], s.p, s.q, s.tokens, s.ua, s.us], [*xs[0], *xs[1], p, q, tokens, ua, us]):
            a.copy_(b)
        s.positions.copy_(torch.arange(12, dtype=torch.int32) + 37 * seed)

    def step(s):
        s.att.plan(s.lens, s.new, s.table, free_pages=s.free, free_head=s.head, in_place=True)
        outs = []
        for (q, k, v), (kc, vc), w in zip(s.xs, s.caches, s.weights):
            t = s.att.append_rope(q, k, v, s.rot, kc, vc, positions=s.positions)
            o, lse = s.att.attend(t, kc, vc, s.table)
            s.att.weigh(t, lse, kc, s.table, w)
            outs += [t, o, lse]
        got = s.att.verify(s.p, s.q, s.tokens, s.ua, s.us, seq_lens=s.lens, new_lens=s.kept)
        s.att.release(s.lens, s.kept, s.table, s.free, s.head, in_place=True)
        for (kc, vc), w in zip(s.caches, s.weights):
            s.att.evict(s.lens, s.table, kc, vc, w, 30, 9, 2, new_lens=s.cut_lens)
        s.att.release(s.lens, s.cut_lens, s.table, s.free, s.head, in_place=True)
        return [*outs, *got]

    def state(s):
        return [s.lens, s.table, s.free, s.head, *s.weights, *(c for pair in s.caches for c in pair)]

    one, two = build(), build()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    fill(two, 0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        kept = [x.clone() for x in state(two)]
        step(two)                            # once before the capture
        for x, y in zip(state(two), kept):
            x.copy_(y)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            outs = step(two)
    for seed in range(12):
        fill(one, seed)
        fill(two, seed)
        want = step(one)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        one.att.check_status()
        two.att.check_status()
        for a, b in zip([*want, *state(one)], [*outs, *state(two)]):
            assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))
    assert max(one.lens.tolist()) == 30      # the budget was met


def test_a_cache_past_32_bits(fm):
    """Pages whose offsets pass 2^32 bytes, keys and values and weights: rows go there, are weighed and moved there."""
    P, Hkv, page, d, new = 40000, 4, 128, 128, 400           # 5.2 GB of keys
    kc, vc = (torch.empty(P, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    weights = torch.zeros(P, Hkv, page, device="cuda")
    g = torch.Generator().manual_seed(2)
    ids = [P - 1, 3, P - 5, P - 9]
    att = fm.PagedAttention(1, 8, Hkv, d, page, P, 5, new, new)
    table = i32([ids + [-1]])
    att.plan(i32([0]), i32([new]), table)
    q, k, v = (torch.randn(new, h, d, generator=g).bfloat16().cuda() for h in (8, Hkv, Hkv))
    rot = fm.Rotary(d)
    turned = att.append_rope(q, k, v, rot, kc, vc)
    line = lambda x: x[ids].transpose(0, 1).flatten(1, 2)[:, :new].clone()  # noqa: E731
    keys, values = line(kc), line(vc)
    assert torch.equal(values.transpose(0, 1), v) and torch.equal(keys.transpose(0, 1), fm.fm_rope(k, att.positions[:new], rot))
    o, lse = att.attend(turned, kc, vc, table)
    att.weigh(turned, lse, kc, table, weights)
    att.check_status()
    want, tol = long_ref.weights(turned.double().cpu(), kc[ids].double().cpu(), lse.double().cpu(), torch.zeros(4, Hkv, page, dtype=torch.float64), [[0, 1, 2, 3]],
                                 [0], [new], d ** -0.5)
    assert ((weights[ids].double().cpu() - want).abs() <= tol).all()
    heavy = line(weights).cpu()
    after = att.evict(i32([new]), table, kc, vc, weights, 150, 20, 4)
    att.check_status()
    assert after.tolist() == [150]
    for h in range(Hkv):
        places = long_ref.kept_places(heavy[h].tolist(), new, 150, 20, 4)
        assert torch.equal(line(kc)[h, :150], keys[h, places]) and torch.equal(line(vc)[h, :150], values[h, places])
        assert torch.equal(line(weights)[h, :150].cpu(), heavy[h, places])


def test_results_of_a_call_on_a_given_stream(fm):
    """They are of that stream's memory: what the current stream frees and asks for is never theirs."""
    side = torch.cuda.Stream()
    rot = fm.Rotary(64)
    lens, new, table = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([40], [20], [[0, 1, 2]]))
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    pool, status, x = torch.zeros(3, 2, 16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(20, 2, 64, dtype=torch.bfloat16, device="cuda")
    places, slots, v = torch.arange(20, dtype=torch.int32, device="cuda"), torch.arange(20, device="cuda"), torch.zeros_like(k)
    p, u = torch.full((2, 100), 0.01, device="cuda"), torch.full((2,), 0.5, device="cuda")
    tokens, cu = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    calls = [lambda s: fm.fm_rope(x, places, rot, stream=s),
             lambda s: fm.fm_paged_append_rope(x, x, x, slots, places, rot, k, v, status, stream=s),
             lambda s: fm.fm_paged_evict(lens, table, k, v, pool, 30, status, stream=s),
             lambda s: fm.fm_paged_release(lens, new, table, 16, 3, None, None, status, stream=s)[0],
             lambda s: fm.fm_verify_drafts(p, None, tokens, u, u[:1], cu, lens, status, stream=s)[0]]
    for call in calls:
        for stream in (side, side.cuda_stream):
            got = call(stream)
            torch.cuda.synchronize()
            at, like = got.data_ptr(), (got.shape, got.dtype)
            del got
            mine = [torch.empty(like[0], dtype=like[1], device="cuda") for _ in range(50)]
            assert all(m.data_ptr() != at for m in mine)
    assert int(status) == 0
