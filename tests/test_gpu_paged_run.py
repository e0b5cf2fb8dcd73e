"""The paged operators as they are used: prompts in chunks, then tokens, through plan, append and
attention; captured and replayed; on other streams; with caches beyond 32-bit offsets."""
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


class Server:
    """Two layers, three requests; what was appended is kept in 64 bits for the reference."""

    def __init__(self, fm, e4m3, window=0, sink=0, max_tokens=160, max_q=130):
        self.R, self.Hq, self.Hkv, self.d, self.page, self.P, self.width = 3, 6, 2, 64, 16, 90, 28
        self.window, self.sink, self.e4m3 = window, sink, e4m3
        self.g = torch.Generator().manual_seed(9)
        shape = (self.P, self.Hkv, self.page, self.d)
        self.caches = [[torch.full(shape, 127, dtype=torch.uint8, device="cuda") if e4m3 else
                        torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
        self.ds = torch.tensor([0.017], device="cuda") if e4m3 else None
        self.att = fm.PagedAttention(self.R, self.Hq, self.Hkv, self.d, self.page, self.P, self.width, max_tokens, max_q, window=window, sink=sink)
        self.free = i32(torch.randperm(self.P, generator=self.g).tolist())
        self.head, self.lens = i32([0]), i32([0] * self.R)
        self.table = i32([[-1] * self.width] * self.R)
        self.history = [[[torch.zeros(0, self.Hkv, self.d, dtype=torch.float64) for _ in range(2)] for _ in range(self.R)] for _ in range(2)]

    def inputs(self, new):
        """q, k, v of both layers for the step's rows."""
        T = sum(new)
        return [[torch.randn(T, h, self.d, generator=self.g).bfloat16() for h in (self.Hq, self.Hkv, self.Hkv)] for _ in range(2)]

    def remember(self, new, xs):
        for layer, (_, k, v) in enumerate(xs):
            t = 0
            for r, n in enumerate(new):
                for i, x in enumerate((k, v)):
                    y = x[t:t + n].double()
                    if self.e4m3:
                        s = self.ds.cpu()
                        y = (x[t:t + n].float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).double() * float(s)
                    self.history[layer][r][i] = torch.cat([self.history[layer][r][i], y])
                t += n

    def expected(self, layer, new, q):
        """The reference over the remembered keys, one page each."""
        k = [torch.cat([self.history[layer][r][i] for r in range(self.R)]) for i in range(2)]
        lens = [self.history[layer][r][0].shape[0] for r in range(self.R)]
        first = np.concatenate([[0], np.cumsum(lens)])
        table = [list(range(first[r], first[r + 1])) + [0] for r in range(self.R)]
        caches = [x[:, :, None, :] for x in k]
        return ref.attend(q.double(), caches[0], caches[1], table, [n - m for n, m in zip(lens, new)], new, 1 / 8.0, self.window, self.sink)

    def run(self, xs):
        out = []
        for (kc, vc), (q, k, v) in zip(self.caches, xs):
            self.att.append(k, v, kc, vc, self.ds, self.ds)
            out.append(self.att.attend(q, kc, vc, self.table, o_dtype=torch.float32, k_descale=self.ds, v_descale=self.ds))
        return out

    def step(self, new):
        xs = self.inputs(new)
        self.att.plan(self.lens, i32(new), self.table, free_pages=self.free, free_head=self.head, in_place=True)
        out = self.run([[x.cuda() for x in layer] for layer in xs])
        self.att.check_status()
        self.remember(new, xs)
        self.check(new, xs, out)

    def check(self, new, xs, out):
        few = max(new) * 3 <= 32
        for layer in range(2):
            o, lse = out[layer]
            p = (2.0 ** -22 if self.e4m3 else 2.0 ** -16)
            ref.check_attention(self.expected(layer, new, xs[layer][0]), o, lse, self.d, p, self.e4m3, self.e4m3 and not few)


@pytest.mark.parametrize("window,sink", [(0, 0), (40, 5)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_prompts_in_chunks_then_tokens(fm, e4m3, window, sink):
    s = Server(fm, e4m3, window, sink)
    steps = ([130, 0, 7], [1, 100, 1], [0, 0, 0], [20, 1, 0], [1, 1, 1], [1, 0, 1], [4, 2, 3], [1, 1, 1])
    for new in steps:
        if sum(new):
            s.step(new)
        else:
            s.att.plan(s.lens, i32(new), s.table, free_pages=s.free, free_head=s.head, in_place=True)
    total = [sum(x) for x in zip(*steps)]
    assert s.lens.tolist() == total
    held = [-(-n // 16) for n in total]
    assert int(s.head.item()) == sum(held)
    pages = [s.table[r, :held[r]].tolist() for r in range(3)]
    assert sorted(sum(pages, [])) == sorted(s.free[:sum(held)].tolist())


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_captured_decoding_step_replays(fm, e4m3):
    s = Server(fm, e4m3, max_tokens=3, max_q=1)
    long = Server(fm, e4m3)             # the same pool of work, for the prompt
    s.caches, s.table, s.free, s.head, s.lens, s.history = long.caches, long.table, long.free, long.head, long.lens, long.history
    long.step([90, 30, 15])
    new = [1, 1, 1]
    one, xs = i32(new), s.inputs(new)
    dev = [[x.cuda() for x in layer] for layer in xs]
    lens, head = s.lens.clone(), s.head.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):       # warm-up, then undone
        s.att.plan(s.lens, one, s.table, free_pages=s.free, free_head=s.head, in_place=True)
        s.run(dev)
        s.lens.copy_(lens)
        s.head.copy_(head)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.att.plan(s.lens, one, s.table, free_pages=s.free, free_head=s.head, in_place=True)
        out = s.run(dev)
    for _ in range(6):
        xs = s.inputs(new)
        for a, b in zip(dev, xs):
            for x, y in zip(a, b):
                x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        s.att.check_status()
        s.remember(new, xs)
        s.check(new, xs, out)
    assert s.lens.tolist() == [96, 36, 21]


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_captured_mixed_batch_replays_to_the_same_bits(fm, e4m3):
    """Chunks, split chunks and single tokens in one captured step: the two attention kernels overlap."""
    g = torch.Generator(device="cuda").manual_seed(8)
    ctx, new, page, P, width = [3000, 40, 700, 9, 2500], [30, 1, 100, 2, 0], 32, 240, 96
    att = fm.PagedAttention(5, 8, 2, 128, page, P, width, 140, 100)
    table = torch.full((5, width), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    for r, (c, n) in enumerate(zip(ctx, new)):
        held = -(-(c + n) // page)
        table[r, :held], order = order[:held], order[held:]
    kc, vc = (torch.randn(P, 2, page, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    ds = torch.tensor([0.013], device="cuda") if e4m3 else None
    if e4m3:
        kc, vc = ((x.float() / ds).clamp(-448, 448).to(torch.float8_e4m3fn) for x in (kc, vc))
    q = torch.randn(133, 8, 128, generator=g, device="cuda").bfloat16()
    lens, fresh = i32(ctx), i32(new)
    att.plan(lens, fresh, table)
    want = att.attend(q, kc, vc, table, k_descale=ds, v_descale=ds)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att.plan(lens, fresh, table)
        first = att.attend(q, kc, vc, table, k_descale=ds, v_descale=ds)
        second = att.attend(q, kc, vc, table, k_descale=ds, v_descale=ds)       # another layer on the same plan
    for _ in range(4):
        for x in first + second:
            x.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        att.check_status()
        for got in (first, second):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_side_streams_and_both_ways_of_marshalling_agree(fm):
    """The current stream through the extension, a stream argument through ctypes: the same bits."""
    g = torch.Generator(device="cuda").manual_seed(1)
    R, page, P, width = 5, 32, 80, 16
    att = fm.PagedAttention(R, 8, 2, 128, page, P, width, 60, 30)
    lens, new = i32([100, 0, 33, 480, 7]), i32([1, 30, 4, 1, 12])
    table = torch.randperm(P, generator=g, device="cuda")[:R * width].to(torch.int32).view(R, width)
    kc, vc = (torch.randn(P, 2, page, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    q, k, v = (torch.randn(48, h, 128, generator=g, device="cuda").bfloat16() for h in (8, 2, 2))
    got = []
    for way in range(3):
        kk, vv = kc.clone(), vc.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        if way == 0:
            att.plan(lens, new, table)
            att.append(k, v, kk, vv)
            o, lse = att.attend(q, kk, vv, table)
        elif way == 1:
            with torch.cuda.stream(side):
                att.plan(lens, new, table)
                att.append(k, v, kk, vv)
                o, lse = att.attend(q, kk, vv, table)
        else:
            o, lse = torch.empty_like(q), torch.empty(48, 8, device="cuda")
            fm.fm_paged_plan(att.step, lens, new, table, att.seq_lens, att.cu_q, att.slots, att.positions, att.plan_buffer, att.status, stream=side)
            fm.fm_paged_append(k, v, att.slots, kk, vv, att.status, stream=side)
            fm.fm_attn_paged(att.step, q, kk, vv, table, att.plan_buffer, 128 ** -0.5, o, lse, att.status, stream=side)
        torch.cuda.synchronize()
        att.check_status()
        got.append((kk, vv, o, lse, att.slots.clone(), att.positions.clone()))
    for other in got[1:]:
        for x, y in zip(got[0], other):
            assert torch.equal(x, y)


@pytest.mark.parametrize("new", [[1, 2], [40, 1]])
def test_pages_beyond_four_gigabytes(fm, new):
    P, page, d = 1_150_000, 16, 128                 # 4.7 GB a pool
    kc, vc = (torch.empty(P, 1, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ctx, g = [37, 18], torch.Generator().manual_seed(2)
    table = [[P - 1, 3, P - 7, 1_060_000, P - 5], [P - 2, P - 3, 1_050_001, P - 9, 2]]
    T = sum(new)
    att = fm.PagedAttention(2, 2, 1, d, page, P, 5, T, max(new))
    dt = i32(table)
    hist = [[torch.randn(c + n, 1, d, generator=g).bfloat16() for c, n in zip(ctx, new)] for _ in range(2)]
    for r in range(2):
        for j in range(ctx[r]):
            for pool, h in zip((kc, vc), hist):
                pool[table[r][j // page], 0, j % page] = h[r][j, 0].cuda()
    k, v = (torch.cat([h[r][ctx[r]:] for r in range(2)]).cuda() for h in hist)
    q = torch.randn(T, 2, d, generator=g).bfloat16()
    att.plan(i32(ctx), i32(new), dt)
    att.append(k, v, kc, vc)
    o, lse = att.attend(q.cuda(), kc, vc, dt, o_dtype=torch.float32)
    att.check_status()
    small = [torch.zeros(10, 1, page, d, dtype=torch.float64) for _ in range(2)]
    for r in range(2):
        for j in range(ctx[r] + new[r]):
            for pool, h in zip(small, hist):
                pool[r * 5 + j // page, 0, j % page] = h[r][j, 0].double()
    want = ref.attend(q.double(), small[0], small[1], [[0, 1, 2, 3, 4], [5, 6, 7, 8, 9]], ctx, new, d ** -0.5)
    ref.check_attention(want, o, lse, d, 2.0 ** -16, False)


def test_slots_beyond_32_bits(fm):
    att = fm.PagedAttention(1, 2, 1, 64, 16, 2 ** 31 - 1, 4, 4, 4)
    att.plan(i32([14]), i32([4]), i32([[2 ** 31 - 2, 2 ** 30, -1, -1]]))
    att.check_status()
    a, b = (2 ** 31 - 2) * 16, 2 ** 30 * 16
    assert att.slots.tolist() == [a + 14, a + 15, b, b + 1]


def test_pages_shared_by_requests(fm):
    """A common prefix: two block tables name the same pages."""
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(8, 2, 16, 64, generator=g).bfloat16() for _ in range(2))
    table, ctx, new = [[3, 1, 5], [3, 1, 2], [3, 1, 5]], [40, 33, 40], [1, 3, 1]
    q = torch.randn(5, 4, 64, generator=g).bfloat16()
    att = fm.PagedAttention(3, 4, 2, 64, 16, 8, 3, 5, 3)
    att.plan(i32(ctx), i32(new), i32(table))
    o, lse = att.attend(q.cuda(), k.cuda(), v.cuda(), i32(table), o_dtype=torch.float32)
    att.check_status()
    ref.check_attention(ref.attend(q.double(), k.double(), v.double(), table, ctx, new, 0.125), o, lse, 64, 2.0 ** -16, False)


# ---- calls that are refused, or end with a status ------------------------------------------------
def small(fm, **kw):
    d = dict(requests=2, Hq=4, Hkv=2, d=64, page_size=16, num_pages=6, max_pages=3, max_tokens=8, max_q=4)
    d.update(kw)
    return fm.PagedAttention(**d)


def test_attention_with_fewer_rows_than_the_plan(fm):
    for max_q, Hq in ((4, 4), (4, 32)):             # both kernels
        att = small(fm, max_q=max_q, Hq=Hq)
        table = i32([[0, 1, -1], [2, 3, -1]])
        att.plan(i32([3, 3]), i32([4, 4]), table)
        kc = torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
        q = torch.zeros(7, Hq, 64, dtype=torch.bfloat16, device="cuda")
        o, lse = torch.full_like(q, 3.0), torch.full((7, Hq), 3.0, device="cuda")
        fm.fm_attn_paged(att.step, q, kc, kc, table, att.plan_buffer, 0.1, o, lse, att.status)
        assert int(att.status.item()) == fm.FM_ERR_LENGTHS and (o == 3).all() and (lse == 3).all()


@pytest.mark.parametrize("field,value", [("requests", 1), ("window", 9), ("max_q", 3), ("max_pages", 2), ("num_pages", 5)])
def test_a_plan_of_another_step(fm, field, value):
    att = small(fm)
    att.plan(i32([3, 3]), i32([1, 1]), i32([[0, 1, -1], [2, 3, -1]]))
    other = small(fm, **{field: value})
    kc = torch.zeros(other.step.num_pages, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.full_like(q, 3.0), torch.full((2, 4), 3.0, device="cuda")
    table = i32([[0, 1, -1], [2, 3, -1]])[:other.step.requests, :other.step.max_pages].contiguous()
    fm.fm_attn_paged(other.step, q, kc, kc, table, att.plan_buffer, 0.1, o, lse, att.status)
    assert int(att.status.item()) == fm.FM_ERR_PLAN_MISMATCH and (o == 3).all()


@pytest.mark.parametrize("Hq", [4, 32])
def test_a_page_number_outside_the_pool_reads_as_zeros(fm, Hq):
    att = small(fm, Hq=Hq)
    g = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.randn(6, 2, 16, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(5, Hq, 64, generator=g, device="cuda").bfloat16()
    new, ctx = [4, 1], [28, 20]
    table = i32([[6, 1, -1], [2, 3, -1]])
    att.plan(i32(ctx), i32(new), table)
    assert int(att.status.item()) == 0              # the bad page holds no new token
    o, lse = att.attend(q, kc, vc, table, o_dtype=torch.float32)
    assert int(att.status.item()) == fm.FM_ERR_PAGES
    k0, v0 = (torch.cat([x, torch.zeros_like(x[:1])]).double().cpu() for x in (kc, vc))
    want = ref.attend(q.double().cpu(), k0, v0, table.tolist(), ctx, new, 0.125)
    ref.check_attention(want, o, lse, 64, 2.0 ** -16, False)


def test_python_refusals(fm):
    att = small(fm)
    kc = torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    q, table = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), i32([[0, 1, -1], [2, 3, -1]])
    att.plan(i32([3, 3]), i32([1, 1]), table)
    for bad in (lambda: att.attend(q.float(), kc, kc, table), lambda: att.attend(q, kc.half(), kc.half(), table),
                lambda: att.attend(q, kc, kc, table.long()), lambda: att.attend(q.cpu(), kc, kc, table),
                lambda: att.attend(q, kc, kc, table, o_dtype=torch.float16), lambda: att.attend(q, kc, kc.cpu(), table)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: att.attend(q[:, :3], kc, kc, table), lambda: att.attend(q, kc, kc[:5], table),
                lambda: att.attend(q, kc.view(torch.uint8)[..., :64], kc.view(torch.uint8)[..., :64], table), lambda: att.attend(q, kc, kc, table[:1]),
                lambda: att.attend(q.transpose(1, 2).contiguous().transpose(1, 2), kc, kc, table),
                lambda: att.append(q[:, :2], q[:, :2], kc[..., :32], kc[..., :32]), lambda: att.plan(i32([1]), i32([1]), table),
                lambda: att.plan(i32([1, 1]), i32([1, 1]), table, free_pages=i32([1, 2]))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fm.FmError) as e:            # the library's own refusal: rows that do not begin on 16 bytes
        wide = torch.zeros(2, 4, 65, dtype=torch.bfloat16, device="cuda")
        att.attend(wide[:, :, :64], kc, kc, table)
    assert e.value.code == fm.FM_ERR_INVALID_ARG
    with pytest.raises(fm.FmError):
        att.attend(q, kc, kc, table, scale=float("nan"))
    empty = att.attend(q[:0], kc, kc, table)
    assert empty[0].shape == (0, 4, 64) and int(att.status.item()) == 0
