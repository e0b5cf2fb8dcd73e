"""Verification of drafted tokens on the GPU: whole numbers, equal to the reference's (long_ref)."""
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


def rows_of(new, V, dtype, greedy, seed, noise=0.7, width=None):
    """Probabilities, drafted tokens and random numbers of requests with new[r] rows."""
    g = torch.Generator().manual_seed(seed)
    T = sum(new)
    x = torch.randn(T, V, generator=g) * 2
    p, q = torch.softmax(x, 1), torch.softmax(x + noise * torch.randn(T, V, generator=g), 1)
    drawn = q.argmax(1) if greedy else torch.multinomial(q, 1, generator=g)[:, 0]
    tokens = torch.cat([torch.zeros(1, dtype=torch.int64), drawn[:-1]]).int()
    u, s = torch.rand(T, generator=g), torch.rand(len(new), generator=g)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return p.to(dtype), None if greedy else q.to(dtype), tokens, u, s, cu


def check(fm, p, q, tokens, u, s, cu, code=0, behind=2):
    R, T = len(cu) - 1, cu[-1]
    pad = lambda t, x: torch.cat([t, torch.full((behind, *t.shape[1:]), x, dtype=t.dtype)])  # noqa: E731
    dev = lambda t, x: None if t is None else pad(t, x).cuda()  # noqa: E731
    out = torch.full((T + behind,), 77, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seq = i32([1000 + 7 * r for r in range(R)])
    got = fm.fm_verify_drafts(dev(p, float("nan")), dev(q, float("nan")), dev(tokens, -5), dev(u, 0.5), s.cuda(), i32(cu), seq, status, out=out)
    want, n_out = ref.verify(p.double(), None if q is None else q.double(), tokens.tolist(), u.double().tolist(), s.double().tolist(), cu)
    assert int(status.item()) == code
    assert got[0].tolist() == want + [77] * behind
    assert got[1].tolist() == n_out
    assert got[2].tolist() == [1000 + 7 * r - (cu[r + 1] - cu[r]) + n_out[r] for r in range(R)]
    return want, n_out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("new,V", [([1], 1), ([1, 2], 2), ([3, 0, 1, 5], 17), ([2] * 40, 1000), ([4, 9, 1], 2049), ([5, 5, 2, 1], 32001), ([70, 33], 100),
                                   ([3, 4], 16385), ([2, 5], 131072)])
def test_verify(fm, new, V, greedy, dtype):
    check(fm, *rows_of(new, V, dtype, greedy, seed=V + len(new)))


@pytest.mark.parametrize("noise", [0.0, 0.05, 5.0])
def test_drafts_near_and_far(fm, noise):
    """The same distribution keeps every draft; a far one next to none."""
    _, n_out = check(fm, *rows_of([6] * 30, 500, torch.float32, False, 9, noise))
    if noise == 0.0:
        assert n_out == [6] * 30


@pytest.mark.parametrize("u", [0.0, 1.0 - 2.0 ** -24])
def test_the_ends_of_the_random_numbers(fm, u):
    p, q, tokens, a, s, cu = rows_of([3] * 20, 3001, torch.float32, False, 3)
    check(fm, p, q, tokens, torch.full_like(a, u), torch.full_like(s, u), cu)


def test_borders(fm):
    """Sums that are exact in any order, random numbers on their borders: the next token, never one without weight."""
    V = 4096
    p = torch.zeros(9, V)
    p[:, ::2] = 2.0 ** -11                       # the even tokens
    s = torch.tensor([0.0, 2.0 ** -11, 0.25, 0.5, 0.625, 1 - 2.0 ** -11, 1 - 2.0 ** -24, 3 * 2.0 ** -11, 0.125])
    got, _ = check(fm, p, None, torch.zeros(9, dtype=torch.int32), torch.zeros(9), s, list(range(10)))
    assert got == [0, 2, 1024, 2048, 2560, 4094, 4094, 6, 512]


def test_weights_that_are_all_zero(fm):
    """p = q refused by p(t) = 0 (u = 0 times anything is not below zero): the draw is p's; q above p everywhere as well."""
    p = torch.tensor([[0.5, 0.5, 0.0, 0.0], [0.25, 0.25, 0.25, 0.25]])
    check(fm, p, p.clone(), torch.tensor([0, 2], dtype=torch.int32), torch.zeros(2), torch.tensor([0.6]), [0, 2])
    check(fm, p, p * 1.5, torch.tensor([0, 3], dtype=torch.int32), torch.full((2,), 0.99), torch.tensor([0.4]), [0, 2])
    check(fm, torch.tensor([[0.0, 1.0], [0.5, 0.5]]), None, torch.tensor([0, 0], dtype=torch.int32), torch.zeros(2), torch.tensor([0.3]), [0, 2])


def test_a_draft_without_probability(fm):
    """q(t) = 0: kept if the target gives it anything."""
    p, q = torch.tensor([[0.1, 0.9], [0.5, 0.5]]), torch.tensor([[0.0, 1.0], [0.5, 0.5]])
    got, n_out = check(fm, p, q, torch.tensor([1, 0], dtype=torch.int32), torch.tensor([0.999, 0.0]), torch.tensor([0.7]), [0, 2])
    assert got == [0, 1] and n_out == [2]


@pytest.mark.parametrize("V", [5, 9000])
@pytest.mark.parametrize("bad", [0.0, float("nan"), float("inf")])
def test_rows_that_cannot_be_drawn_from(fm, V, bad):
    p = torch.full((3, V), 1.0 / V)
    p[1] = bad if bad == 0.0 else p[1]
    p[1, V // 2] = bad
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, n_out, lens = fm.fm_verify_drafts(p.cuda(), None, i32([0, 0, 0]), torch.zeros(3, device="cuda"), torch.full((3,), 0.5, device="cuda"),
                                           i32([0, 1, 2, 3]), i32([9, 9, 9]), status)
    assert int(status.item()) == fm.FM_ERR_PROBS
    assert out.tolist()[1] == -1 and out.tolist()[0] == out.tolist()[2] >= 0 and n_out.tolist() == [1, 1, 1] and lens.tolist() == [9, 9, 9]


@pytest.mark.parametrize("token", [-1, 100, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("greedy", [False, True])
def test_drafts_outside_the_vocabulary(fm, token, greedy):
    p, q, tokens, u, s, cu = rows_of([3, 2], 100, torch.float32, greedy, 5)
    tokens[1] = token
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, n_out, _ = fm.fm_verify_drafts(p.cuda(), None if greedy else q.cuda(), tokens.cuda(), u.cuda(), s.cuda(), i32(cu), i32([9, 9]), status)
    assert int(status.item()) == fm.FM_ERR_PROBS and n_out.tolist()[0] == 1 and 0 <= out.tolist()[0] < 100 and out.tolist()[1:3] == [-1, -1]
    # A token behind the first refusal is not looked at.
    tokens[1], tokens[2] = (0 if float(p[0, 0]) < 0.5 else 1), token
    u[0] = 1.0 - 2.0 ** -24
    status.zero_()
    p[0, int(tokens[1])] = 0.0
    fm.fm_verify_drafts(p.cuda(), None if greedy else q.cuda(), tokens.cuda(), u.cuda(), s.cuda(), i32(cu), i32([9, 9]), status)
    assert int(status.item()) == 0


@pytest.mark.parametrize("cu", [[0, 2, 5], [0, -1, 4], [-2, 2, 4], [0, 3, 2]])
def test_rows_out_of_range(fm, cu):
    p, q, tokens, u, s, _ = rows_of([2, 2], 50, torch.float32, False, 6)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    _, n_out, lens = fm.fm_verify_drafts(p.cuda(), q.cuda(), tokens.cuda(), u.cuda(), s.cuda(), i32(cu), i32([9, 8]), status, out=out)
    assert int(status.item()) == fm.FM_ERR_LENGTHS
    for r in range(2):
        if not 0 <= cu[r] <= cu[r + 1] <= 4:
            assert n_out.tolist()[r] == 0 and lens.tolist()[r] == [9, 8][r]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_at_any_stride(fm, dtype):
    """Rows inside wider ones, off 16 bytes."""
    p, q, tokens, u, s, cu = rows_of([4, 3], 4999, dtype, False, 8)
    a, b = torch.full((7, 5011), float("nan"), dtype=dtype), torch.full((7, 5003), float("nan"), dtype=dtype)
    a[:, 3:5002], b[:, 1:5000] = p, q
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (tokens.cuda(), u.cuda(), s.cuda(), i32(cu), i32([50, 50]), status)
    one = fm.fm_verify_drafts(p.cuda(), q.cuda(), *args)
    two = fm.fm_verify_drafts(a.cuda()[:, 3:5002], b.cuda()[:, 1:5000], *args)
    assert all(torch.equal(x, y) for x, y in zip(one, two)) and int(status.item()) == 0
    assert one[0].tolist() == ref.verify(p.double(), q.double(), tokens.tolist(), u.double().tolist(), s.double().tolist(), cu)[0]


def test_tokens_come_out_as_the_targets(fm):
    """30,000 single drafts of 5 tokens: the first token's frequencies are p's, each within six standard deviations."""
    g = torch.Generator().manual_seed(11)
    n = 30000
    p, q = torch.tensor([0.4, 0.3, 0.2, 0.1, 0.0]), torch.tensor([0.1, 0.2, 0.3, 0.2, 0.2])
    tokens = torch.zeros(2 * n, dtype=torch.int32)
    tokens[1::2] = torch.multinomial(q, n, replacement=True, generator=g).int()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    freq = torch.zeros(5)
    for i in range(0, n, 5000):
        rows = slice(2 * i, 2 * i + 10000)
        out, _, _ = fm.fm_verify_drafts(p.expand(10000, 5).contiguous().cuda(), q.expand(10000, 5).contiguous().cuda(), tokens[rows].cuda(),
                                        torch.rand(10000, generator=g).cuda(), torch.rand(5000, generator=g).cuda(),
                                        torch.arange(0, 10001, 2, dtype=torch.int32, device="cuda"), i32([9] * 5000), status)
        freq += torch.bincount(out[::2].long().cpu(), minlength=5).float()
    assert int(status.item()) == 0
    assert ((freq / n - p).abs() <= 6 * (p * (1 - p) / n).sqrt()).all()


def test_a_step_without_rows(fm):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    p = torch.empty(0, 50, device="cuda")
    for draft in (None, p):
        out, n_out, lens = fm.fm_verify_drafts(p, draft, none, none.float(), torch.zeros(2, device="cuda"), i32([0, 0, 0]), i32([5, 0]), status)
        assert out.shape == (0,) and n_out.tolist() == [0, 0] and lens.tolist() == [5, 0] and int(status.item()) == 0


def test_lengths_in_place(fm):
    p, q, tokens, u, s, cu = rows_of([3, 1], 40, torch.float32, False, 5)
    status, seq = torch.zeros(1, dtype=torch.int32, device="cuda"), i32([30, 20])
    args = (p.cuda(), q.cuda(), tokens.cuda(), u.cuda(), s.cuda(), i32(cu), seq, status)
    want = fm.fm_verify_drafts(*args)[2].tolist()
    got = fm.fm_verify_drafts(*args, new_lens=seq)[2]
    assert got.data_ptr() == seq.data_ptr() and seq.tolist() == want
