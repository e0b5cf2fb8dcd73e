"""Operators around the attention of long conversations, in plain torch and through the package.

Rotary positions (of a training batch with the backward pass, and of a serving step's rows as they are appended to the
paged cache), the attention weight that every cached key receives, the eviction of the lightest keys down to a budget, and
the verification of drafted tokens; the last two with the pages that they give back.  With ``own`` false they are computed
by elementary torch operations; with ``own`` true by the calls a user makes.
"""
import math
import random

import torch

own = False

_DEV = "cuda"


def listed():
    def rope(name, **kw):
        return dict(dict(op="rope", name=name, d=128, rot=128, pairs="halves", scaling="none", factor=1.0, inverse=False), **kw)

    def append(name, **kw):
        return dict(dict(op="append", name=name, Hq=32, Hkv=8, d=128, rot=128, pairs="halves", scaling="none", factor=1.0, page=64,
                         cache="bf16", ctx_max=8192), **kw)

    def weigh(name, **kw):
        return dict(dict(op="weigh", name=name, Hq=32, Hkv=8, d=128, page=64, window=0, sink=0, cache="bf16"), **kw)

    def evict(name, **kw):
        return dict(dict(op="evict", name=name, Hkv=8, d=128, page=64, cache="bf16", sink=4), **kw)

    def verify(name, **kw):
        return dict(dict(op="verify", name=name, probs="f32", greedy=False, page=64, ctx_max=8192), **kw)

    return [
        # The queries of a 128K-token packed training sequence, positions beginning again with every document, stretched.
        rope("rope_train_128k", B=1, H=8, N=131072, lens=1, x="bf16", out="bf16", scaling="yarn", factor=8.0),
        # The backward pass: fp32 gradients of the attention to 16 bits, half of the head rotated, neighbours paired.
        rope("rope_grad", B=2, H=8, N=8192, lens=2, x="f32", out="bf16", rot=64, pairs="neighbours", inverse=True),
        # The new tokens of a small decoding batch: all latency.
        append("append_decode", R=33, q_max=1, lens=3),
        # Prompt chunks into an e4m3 cache of small pages, positions stretched linearly.
        append("append_chunks_e4m3", R=12, q_max=4096, ctx_max=16384, page=16, cache="e4m3", scaling="linear", factor=4.0, lens=4),
        # Two short chats: the smallest call.
        weigh("weigh_small", R=2, q_max=1, ctx_max=500, d=64, page=16, lens=5),
        # A decoding batch of ragged lengths: reads every key once.
        weigh("weigh_batch", R=96, q_max=1, ctx_max=16000, lens=7),
        # The same kind of batch over an e4m3 cache with small pages, up to three tokens a request.
        weigh("weigh_batch_e4m3", R=64, q_max=3, ctx_max=16000, page=16, cache="e4m3", lens=8),
        # Two long prompts' chunks after a cached prefix: matrix work.
        weigh("weigh_chunk", R=2, q_max=4096, ctx_max=12000, lens=9),
        # A batch of conversations, the longer ones cut down to 4,096 tokens.
        evict("evict_batch", R=32, ctx_max=12000, budget=4096, recent=512, lens=10),
        # One conversation of 128K tokens cut down to 16K, e4m3 cache.
        evict("evict_128k", R=1, ctx_max=131072, budget=16384, recent=2048, cache="e4m3", lens=11),
        # Two requests with a drafted token or two, the drafts taken as the likeliest ones, 16-bit probabilities.
        verify("verify_small", R=2, q_max=3, V=32000, probs="bf16", greedy=True, lens=12),
        # A serving batch with four drafted tokens a request and a large vocabulary.
        verify("verify_batch", R=64, q_max=5, V=131072, lens=13),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    lens = rng.randrange(1 << 30)
    op = rng.choice(["rope", "append", "weigh", "weigh", "evict", "verify"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "e4m3"])
    turn = dict(rot=rng.choice([d, d, d // 2, 8 * rng.randrange(2, d // 8)]), pairs=rng.choice(["halves", "neighbours"]),
                scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=rng.choice([1.5, 4.0, 16.0]))
    if op == "rope":
        B, H = rng.choice([1, 1, 2, 3]), rng.choice([1, 5, 8, 16])
        N = min(_log(rng, 1, 131072), 134_000_000 // (B * H * d))
        return dict(op=op, B=B, H=H, N=N, d=d, lens=lens, x=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "bf16", "f32"]),
                    inverse=rng.choice([False, True]), **turn)
    if op == "append":
        Hq, Hkv = rng.choice([(8, 8), (32, 8), (12, 4), (16, 1), (5, 5)])
        R, q_max = _log(rng, 1, 128), _log(rng, 1, 4096)
        q_max = max(1, min(q_max, 32768 // R))
        return dict(op=op, R=R, q_max=q_max, ctx_max=_log(rng, 1, 8192), Hq=Hq, Hkv=Hkv, d=d, page=page, cache=cache, lens=lens, **turn)
    if op == "weigh":
        Hq, Hkv = rng.choice([(8, 8), (16, 16), (32, 8), (12, 4), (28, 4), (10, 2), (16, 1), (5, 5)])
        q_max = rng.choice([1, 1, _log(rng, 2, 8), _log(rng, 9, 3000)])
        ctx_max = _log(rng, 1, 100000 if q_max == 1 else 16000)
        R = _log(rng, 1, 96)
        keys = ctx_max + q_max
        R = max(1, min(R, 1_000_000_000 // (keys * Hkv * d), 2_000_000_000 // (Hq * q_max * keys)))
        window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        return dict(op=op, R=R, q_max=q_max, ctx_max=ctx_max, Hq=Hq, Hkv=Hkv, d=d, page=page, window=window,
                    sink=rng.choice([0, 4, 10]) if window else 0, cache=cache, lens=lens)
    if op == "evict":
        R, Hkv = _log(rng, 1, 64), rng.choice([1, 2, 5, 8])
        ctx_max = min(_log(rng, 20, 131072), 250_000_000 // (R * Hkv * d))
        budget = _log(rng, max(2, ctx_max // 64), ctx_max)
        sink = min(rng.choice([0, 4]), budget)
        return dict(op=op, R=R, ctx_max=ctx_max, budget=budget, recent=rng.randrange(budget - sink + 1), sink=sink, Hkv=Hkv, d=d, page=page,
                    cache=cache, lens=lens)
    q_max = rng.choice([1, 2, 3, 5, 9])
    V = _log(rng, 500, 131072)
    return dict(op=op, R=min(_log(rng, 1, 128), 64 * 5 * 131072 // (q_max * V)), q_max=q_max, V=V, probs=rng.choice(["f32", "bf16"]),
                greedy=rng.choice([False, False, True]), page=page, ctx_max=_log(rng, 1, 8192), lens=lens)


def _lens(case):
    """Cached and new tokens of every request: request 0 has the largest of both, the others are spread below."""
    rng, q = random.Random(case["lens"]), case.get("q_max", 1)
    ctx = [case["ctx_max"]] + [_log(rng, max(1, case["ctx_max"] // 16), case["ctx_max"]) for _ in range(case["R"] - 1)]
    new = [q] + [_log(rng, max(1, q // 512), q) for _ in range(case["R"] - 1)]
    return ctx, new


def _pages(tokens, page):
    return -(-tokens // page)


def _rotary(case):
    """Frequencies of the pairs (float64, radians per position) and the factor on sine and cosine."""
    rot, s = case["rot"], case["factor"]
    base = 10000.0
    if case["scaling"] == "ntk" and rot > 2:
        base *= s ** (rot / (rot - 2))
    theta = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["scaling"] == "linear":
        theta = theta / s
    if case["scaling"] == "yarn":
        g = ((4096 * theta / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return theta * (g + (1 - g) / s), 0.1 * math.log(s) + 1.0
    return theta, 1.0


def prepare(case, seed):
    g = torch.Generator(device=_DEV).manual_seed(seed)
    s = dict(case=case)
    normal = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device=_DEV).normal_(generator=g)  # noqa: E731
    if "rot" in case:
        theta, s["magnitude"] = _rotary(case)
        s["theta"] = theta.to(_DEV)
        if own:
            from long_context_fm_gb300 import fm
            s["rotary"] = fm.Rotary(case["rot"], interleaved=case["pairs"] == "neighbours", scaling=case["scaling"], factor=case["factor"],
                                    original=4096)
    if case["op"] == "rope":
        rng, at = random.Random(case["lens"]), torch.arange(case["N"], dtype=torch.int32)
        begin = 0
        while begin < case["N"]:            # documents of a packed batch
            n = _log(rng, 256, 32768)
            at[begin:begin + n] -= begin
            begin += n
        s["positions"] = at.to(_DEV)
        s["x"] = normal(case["B"], case["H"], case["N"], case["d"], dtype=_type(case["x"]))
        return s
    page = case["page"]
    ctx, new = _lens(case)
    if case["op"] == "evict":
        new = [0] * len(ctx)
    R, T, full = case["R"], sum(new), [_pages(c + n, page) for c, n in zip(ctx, new)]
    num_pages = sum(full) + 3
    s.update(page=page, T=T, num_pages=num_pages, max_pages=max(full) + 1, q_max=max(new), k_max=max(c + n for c, n in zip(ctx, new)))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=_DEV)  # noqa: E731
    s["ctx"], s["new"], s["seq"] = i32(ctx), i32(new), i32([c + n for c, n in zip(ctx, new)])
    s["cu_q"] = torch.cat([i32([0]), s["new"].cumsum(0).int()])
    # Pages of the pool in the order in which a server that has run for a while has them: any order.
    order = torch.randperm(num_pages, generator=g, device=_DEV).to(torch.int32)
    s["table"] = torch.full((R, s["max_pages"]), -1, dtype=torch.int32, device=_DEV)
    s["table"][torch.arange(s["max_pages"], device=_DEV)[None, :] < i32(full)[:, None]] = order[:sum(full)]
    # The pages that requests hold were taken from the front of the free list.
    s["free"], s["head"] = order, i32([sum(full)])
    if case["op"] == "verify":
        V = case["V"]
        x = normal(T, V, dtype=torch.float32).mul_(2.0)
        s["target"] = torch.softmax(x, 1)
        q = torch.softmax(x.add_(normal(T, V, dtype=torch.float32).mul_(0.7)), 1)
        last = s["cu_q"][1:].long() - 1
        drawn = q.argmax(1) if case["greedy"] else q.cumsum(1, dtype=torch.float64).lt_(torch.rand(T, 1, generator=g, device=_DEV)).sum(1).clamp_max(V - 1)
        s["tokens"] = torch.cat([i32([0]), drawn.int()[:-1]])   # row i + 1 feeds what was drafted at row i
        s["tokens"][(last + 1)[:-1]] = 0
        s["target"] = s["target"].to(_type(case["probs"]))
        s["draft"] = None if case["greedy"] else q.to(_type(case["probs"]))
        s["u_accept"] = torch.rand(T, generator=g, device=_DEV)
        s["u_sample"] = torch.rand(R, generator=g, device=_DEV)
        if own:
            s["status"] = torch.zeros(1, dtype=torch.int32, device=_DEV)
        return s
    Hkv, d = case["Hkv"], case["d"]
    e4m3 = case["cache"] == "e4m3"
    if e4m3:
        s["k_descale"] = torch.tensor([4.0 / 448.0 * 1.5], device=_DEV)
        s["v_descale"] = torch.tensor([4.0 / 448.0 * 1.25], device=_DEV)
    for n in ("k", "v"):
        x = normal(num_pages, Hkv, page, d)
        s[n + "_cache"] = (x / s[n + "_descale"].to(torch.bfloat16)).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else x
    if case["op"] == "append":
        Hq = case["Hq"]
        qkv = normal(T, Hq + 2 * Hkv, d)        # one projection's output
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        row = torch.repeat_interleave(torch.arange(R, device=_DEV), s["new"].long(), output_size=T)
        at = torch.arange(T, device=_DEV) - s["cu_q"][row] + s["ctx"][row]
        s["slots"] = s["table"][row, at // page].long() * page + at % page
        # Requests of which much was evicted: the positions run ahead of the cached lengths.
        s["positions"] = (at + torch.randint(0, 100000, (R,), generator=g, device=_DEV)[row]).int()
        if own:
            s["status"] = torch.zeros(1, dtype=torch.int32, device=_DEV)
        return s
    # A few keys take most of the weight, most keys next to none, some none at all.
    w = normal(num_pages, Hkv, page, dtype=torch.float32).mul_(2.0).exp_()
    s["weights"] = torch.where(w < 0.04, 0.0, w)
    if case["op"] == "evict":
        if own:
            s["status"] = torch.zeros(1, dtype=torch.int32, device=_DEV)
            s["kept"] = torch.empty(R, Hkv, case["budget"], dtype=torch.int32, device=_DEV)
        return s
    s["weights"].mul_(2.0 ** -10)                           # of the order of what one step adds
    s["q"] = normal(T, case["Hq"], d).mul_(1.5)
    s["scale"] = 1.0 / math.sqrt(d)
    s["lse"] = _lse(s)
    if own:
        from long_context_fm_gb300 import fm
        s["step"] = fm.PagedAttention(R, case["Hq"], Hkv, d, page, num_pages, s["max_pages"], T, s["q_max"], window=case["window"], sink=case["sink"])
        s["step"].plan(s["ctx"], s["new"], s["table"])
    return s


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


# ---- rotary positions -----------------------------------------------------------

def _rotate(s, x, positions, inverse=False):
    """x: [..., d] with the rows' positions [...] broadcast over it, in 32 bits; angles in 64."""
    rot = s["case"]["rot"]
    angle = positions.double()[..., None] * s["theta"]
    cos, sin = (angle.cos() * s["magnitude"]).float(), (angle.sin() * s["magnitude"]).float()
    if inverse:
        sin = -sin
    x = x.float()
    y = x.clone()
    if s["case"]["pairs"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _rope(s):
    return dict(y=_rotate(s, s["x"], s["positions"], s["case"]["inverse"]).to(_type(s["case"]["out"])))


def _append(s):
    page, slots, at = s["page"], s["slots"], s["positions"][:, None]
    where = (slots // page, slice(None), slots % page)
    for n, x in (("k", _rotate(s, s["k"], at)), ("v", s["v"].float())):
        if n + "_descale" in s:
            x = (x / s[n + "_descale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            x = x.to(torch.bfloat16)
        s[n + "_cache"][where] = x
    return dict(q=_rotate(s, s["q"], at).to(torch.bfloat16), **_caches(s))


def _caches(s):
    """Both caches; codes as the values they stand for (in units of the descale)."""
    if "k_descale" in s:
        return {n: s[n + "_cache"].view(torch.float8_e4m3fn) for n in ("k", "v")}
    return {n: s[n + "_cache"] for n in ("k", "v")}


# ---- attention weight of the cached keys ----------------------------------------------

def _scores(s):
    """Scaled scores [R, Hkv, G, q_max, k_max], -inf where the mask or a ragged end hides the pair; rows of q [R, q_max], which exist, pages."""
    case, page, q_max, k_max = s["case"], s["page"], s["q_max"], s["k_max"]
    R, Hq, Hkv, d = case["R"], case["Hq"], case["Hkv"], case["d"]
    G = Hq // Hkv
    ctx, new = s["ctx"].long(), s["new"].long()
    key = torch.arange(k_max, device=_DEV)
    pages = s["table"].long()[:, key // page].clamp_min(0)  # [R, k_max]
    k = s["k_cache"][pages, :, key % page]                  # [R, k_max, Hkv, d]
    k = k.view(torch.float8_e4m3fn).float() * s["k_descale"] if "k_descale" in s else k.float()
    i = torch.arange(q_max, device=_DEV)
    valid = i[None, :] < new[:, None]
    tok = torch.where(valid, (new.cumsum(0) - new)[:, None] + i[None, :], 0)  # [R, q_max]
    q = s["q"][tok].float().view(R, q_max, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(R, Hkv, G * q_max, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(R, Hkv, G, q_max, k_max)
    pos = ctx[:, None] + i[None, :]
    see = valid[:, :, None] & (key[None, None, :] <= pos[:, :, None])
    if case["window"]:
        see = see & ((key[None, None, :] > pos[:, :, None] - case["window"]) | (key[None, None, :] < case["sink"]))
    return x.masked_fill_(~see[:, None, None], -math.inf), tok, valid, pages


def _lse(s):
    """Log-sum-exp of every row's scores [T, Hq]: what the attention gives."""
    x, _, valid, _ = _scores(s)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    z = m.squeeze(-1) + x.sub_(m).exp_().sum(-1).log()      # [R, Hkv, G, q_max]
    return z.permute(0, 3, 1, 2).reshape(*valid.shape, -1)[valid]


def _weigh(s):
    case, page = s["case"], s["page"]
    x, tok, valid, pages = _scores(s)
    R, Hkv, G, q_max, k_max = x.shape
    z = s["lse"][tok].view(R, q_max, Hkv, G).permute(0, 2, 3, 1)
    w = x.sub_(z[..., None]).exp_().sum((2, 3))             # [R, Hkv, k_max]
    key = torch.arange(k_max, device=_DEV)
    # Keys of this step begin at zero; places behind a request's end go to a page that no request holds.
    inside, fresh = key < s["seq"][:, None], key >= s["ctx"][:, None]
    pages = torch.where(inside, pages, s["free"][-1].long())
    old = s["weights"][pages, :, key % page].transpose(1, 2)
    w = torch.where(inside[:, None], torch.where(fresh[:, None], w, old + w), old)
    s["weights"][pages, :, key % page] = w.transpose(1, 2)
    return dict(weights=s["weights"])


# ---- eviction ----------------------------------------------------------------------------

def _evict(s):
    case, page, k_max = s["case"], s["page"], s["k_max"]
    R, Hkv = case["R"], case["Hkv"]
    budget, recent, sink = case["budget"], case["recent"], case["sink"]
    lens = s["ctx"].long()
    key = torch.arange(max(k_max, budget), device=_DEV)
    pages = torch.where(key < lens[:, None], s["table"].long()[:, (key // page).clamp_max(s["max_pages"] - 1)], s["free"][-1].long())
    w = s["weights"][pages, :, key % page].transpose(1, 2)  # [R, Hkv, k_max]
    sure = (key < sink) | (key >= lens[:, None] - recent)
    w = torch.where(sure[:, None], math.inf, w).masked_fill((key >= lens[:, None])[:, None], -math.inf)
    kept = w.sort(dim=2, descending=True, stable=True).indices[:, :, :budget].sort(dim=2).values
    cut = (lens > budget)[:, None, None]
    to = torch.arange(budget, device=_DEV)
    kept = torch.where(cut, kept, to)                       # what is not cut stays where it is
    head = torch.arange(Hkv, device=_DEV)[None, :, None]
    src, dst = pages[:, None].expand(R, Hkv, -1).gather(2, kept), pages[:, None, :budget].expand(R, Hkv, -1)
    for x in (s["k_cache"], s["v_cache"], s["weights"]):
        x[dst, head, to % page] = x[src, head, kept % page]
    new = lens.clamp_max(budget)
    return dict(kept=torch.where(cut, kept, -1).int(), new_lens=new.int(), weights=s["weights"], **_caches(s), **_release(s, s["ctx"], new))


def _release(s, held, lens):
    """Pages behind `lens` go back in front of the free list's head, in the order of the requests and of their places."""
    page, free, head = s["page"], s["free"], s["head"].long()
    want, have = (lens.long() + page - 1) // page, (held.long() + page - 1) // page
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device=_DEV), (have - want).cumsum(0)])
    col = torch.arange(s["max_pages"], device=_DEV)[None, :]
    back = (col >= want[:, None]) & (col < have[:, None])
    at = torch.where(back, head - off[-1] + off[:-1, None] + col - want[:, None], len(free))
    more = torch.cat([free, free[:1]])
    more[at] = s["table"]
    return dict(free=more[:-1], free_next=(head - off[-1]).int(), seq_lens=lens.int())


# ---- verification of drafted tokens ---------------------------------------------------------

def _verify(s):
    R, q_max, T, V = s["case"]["R"], s["q_max"], s["T"], s["case"]["V"]
    cu, new = s["cu_q"].long(), s["new"].long()
    i = torch.arange(q_max, device=_DEV)
    rows = (cu[:-1, None] + i).clamp_max(T - 1)             # [R, q_max]
    drafted = s["tokens"].long()[(rows + 1).clamp_max(T - 1)]
    p = s["target"][rows, drafted].double()
    q = 1.0 if s["draft"] is None else s["draft"][rows, drafted].double()
    ok = (s["u_accept"][rows].double() * q < p) & (i < new[:, None] - 1)
    taken = ok.long().cumprod(1).sum(1)                     # accepted drafts: up to the first refusal
    row = cu[:-1] + taken
    p = s["target"][row].double()
    hot = torch.arange(V, device=_DEV) == s["tokens"].long()[(row + 1).clamp_max(T - 1), None]
    q = hot.double() if s["draft"] is None else s["draft"][row].double()
    r = torch.where((taken < new - 1)[:, None], (p - q if s["draft"] is not None else torch.where(hot, 0.0, p)).clamp_min(0.0), p)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p)
    c = r.cumsum(1)
    x = ((c > s["u_sample"].double()[:, None] * c[:, -1:]) & (r > 0)).int().argmax(1)
    out = torch.full((T,), -1, dtype=torch.int32, device=_DEV)
    mine = torch.repeat_interleave(torch.arange(R, device=_DEV), new, output_size=T)
    at = torch.arange(T, device=_DEV) - cu[mine]
    feed = s["tokens"][(torch.arange(T, device=_DEV) + 1).clamp_max(T - 1)]
    out = torch.where(at < taken[mine], feed, torch.where(at == taken[mine], x[mine].int(), out))
    lens = s["seq"].long() - new + taken + 1
    return dict(out=out, n_out=(taken + 1).int(), new_lens=lens.int(), **_release(s, s["seq"], lens))


def run(state):
    s = state
    case = s["case"]
    op = case["op"]
    if not own:
        return dict(rope=_rope, append=_append, weigh=_weigh, evict=_evict, verify=_verify)[op](s)
    from long_context_fm_gb300 import fm
    if op == "rope":
        return dict(y=fm.fm_rope(s["x"], s["positions"], s["rotary"], out_dtype=_type(case["out"]), inverse=case["inverse"]))
    if op == "append":
        q = fm.fm_paged_append_rope(s["q"], s["k"], s["v"], s["slots"], s["positions"], s["rotary"], s["k_cache"], s["v_cache"], s["status"],
                                    k_descale=s.get("k_descale"), v_descale=s.get("v_descale"))
        return dict(q=q, **_caches(s))
    if op == "weigh":
        s["step"].weigh(s["q"], s["lse"], s["k_cache"], s["table"], s["weights"], s["scale"], k_descale=s.get("k_descale"))
        return dict(weights=s["weights"])
    if op == "evict":
        new_lens = fm.fm_paged_evict(s["ctx"], s["table"], s["k_cache"], s["v_cache"], s["weights"], case["budget"], s["status"],
                                     recent=case["recent"], sink=case["sink"], kept=s["kept"])
        seq, after = fm.fm_paged_release(s["ctx"], new_lens, s["table"], s["page"], s["num_pages"], s["free"], s["head"], s["status"])
        return dict(kept=s["kept"], new_lens=new_lens, weights=s["weights"], free=s["free"], free_next=after, seq_lens=seq, **_caches(s))
    out, n_out, new_lens = fm.fm_verify_drafts(s["target"], s["draft"], s["tokens"], s["u_accept"], s["u_sample"], s["cu_q"], s["seq"], s["status"])
    seq, after = fm.fm_paged_release(s["seq"], new_lens, s["table"], s["page"], s["num_pages"], s["free"], s["head"], s["status"])
    return dict(out=out, n_out=n_out, new_lens=new_lens, free=s["free"], free_next=after, seq_lens=seq)


def work(case):
    size = {"bf16": 2, "f32": 4, "e4m3": 1}
    if case["op"] == "rope":
        n = case["B"] * case["H"] * case["N"] * case["d"]
        return dict(bytes=n * (size[case["x"]] + size[case["out"]]) + 4 * case["N"], flops=3 * n * case["rot"] // case["d"])
    ctx, new = _lens(case)
    T, R, page = sum(new), case["R"], case["page"]
    if case["op"] == "verify":
        # One row of both distributions per request (of the target's alone where every draft is accepted).
        return dict(bytes=R * case["V"] * size[case["probs"]] * (1 if case["greedy"] else 2) + 16 * T + 24 * R, flops=2 * R * case["V"])
    Hkv, d, esz = case["Hkv"], case["d"], size[case["cache"]]
    if case["op"] == "append":
        return dict(bytes=T * d * (4 * case["Hq"] + 2 * Hkv * (2 + esz)) + 12 * T, flops=3 * T * (case["Hq"] + Hkv) * case["rot"])
    if case["op"] == "evict":
        # The weights that are chosen among, and key, value and weight of all that is kept but the first ones, read and written.
        long = [c for c in ctx if c > case["budget"]]
        moved = len(long) * (case["budget"] - case["sink"]) * Hkv
        return dict(bytes=4 * Hkv * sum(c - case["sink"] - case["recent"] for c in long) + moved * (4 * d * esz + 8) +
                    4 * len(long) * Hkv * case["budget"] + 8 * R + 4 * sum(_pages(c, page) for c in long), flops=0)
    pairs, keys = _pairs(ctx, new, case["window"], case["sink"])
    Hq = case["Hq"]
    return dict(bytes=keys * Hkv * (d * esz + 8) + T * Hq * (2 * d + 4) + 4 * sum(_pages(c + n, page) for c, n in zip(ctx, new)),
                flops=2 * d * Hq * pairs)


def _pairs(ctx, new, window, sink):
    """Attended (row, key) pairs of one head, and the keys that some row attends."""
    if not window:
        return sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new)), sum(c + n for c, n in zip(ctx, new))
    pairs = sum(min(p + 1, window + min(sink, max(0, p + 1 - window))) for c, n in zip(ctx, new) for p in range(c, c + n))
    return pairs, sum(min(c + n, n + window - 1 + sink) for c, n in zip(ctx, new))


# ---- 64-bit values ------------------------------------------------------------------

def _nearest_e4m3(x):
    """The e4m3 value nearest to x (ties to the even code), in 64 bits."""
    x = x.clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _turned(case, x, positions, inverse=False):
    """x double [..., d] as complex numbers times a power of e."""
    theta, m = _rotary(case)
    rot = case["rot"]
    angle = positions.double()[..., None] * theta.to(x.device)
    z = torch.polar(torch.full_like(angle, m), -angle if inverse else angle)
    if case["pairs"] == "halves":
        y = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z
        return torch.cat([y.real, y.imag, x[..., rot:]], -1)
    y = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * z
    return torch.cat([torch.view_as_real(y).reshape(*x.shape[:-1], rot), x[..., rot:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        y = torch.empty(s["x"].shape, dtype=torch.float64, device=_DEV)
        for h in range(case["H"]):
            y[:, h] = _turned(case, s["x"][:, h].double(), s["positions"], case["inverse"])
        return dict(y=y)
    ctx, new = _lens(case)
    page = case["page"]
    if op == "append":
        found = dict(q=_turned(case, s["q"].double(), s["positions"][:, None]))
        k = _turned(case, s["k"].double(), s["positions"][:, None])
        for n, x in (("k", k), ("v", s["v"].double())):
            c = s[n + "_cache"]
            if case["cache"] == "e4m3":
                c = c.view(torch.float8_e4m3fn)
                x = _nearest_e4m3(x / float(s[n + "_descale"]))
            c = c.double()
            c[torch.div(s["slots"], page, rounding_mode="floor"), :, s["slots"] % page] = x
            found[n] = c
        return found
    table = s["table"].tolist()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731

    def released(held, lens):
        free, head = s["free"].tolist(), int(s["head"])
        back = [table[r][b] for r in range(len(lens)) for b in range(_pages(lens[r], page), _pages(held[r], page))]
        free[head - len(back):head] = back
        return dict(free=i32(free), free_next=i32([head - len(back)]), seq_lens=i32(lens))

    if op == "verify":
        out, n_out, lens, t0 = [], [], [], 0
        tokens, ua, us = s["tokens"].tolist(), s["u_accept"].double().tolist(), s["u_sample"].double().tolist()
        for r, n in enumerate(new):
            a = 0
            while a < n - 1:
                t = tokens[t0 + a + 1]
                if not ua[t0 + a] * (1.0 if case["greedy"] else float(s["draft"][t0 + a, t])) < float(s["target"][t0 + a, t]):
                    break
                a += 1
            w = s["target"][t0 + a].double()
            if a < n - 1 and case["greedy"]:
                w[tokens[t0 + a + 1]] = 0.0
            elif a < n - 1:
                w = (w - s["draft"][t0 + a].double()).clamp_min(0.0)
            c = w.cpu().numpy().cumsum()
            out += tokens[t0 + 1:t0 + 1 + a] + [int((c <= us[r] * c[-1]).sum())] + [-1] * (n - 1 - a)
            n_out.append(a + 1)
            lens.append(ctx[r] + a + 1)
            t0 += n
        return dict(out=i32(out), n_out=i32(n_out), new_lens=i32(lens), **released([c + n for c, n in zip(ctx, new)], lens))
    Hkv = case["Hkv"]
    if op == "evict":
        budget, recent, sink = case["budget"], case["recent"], case["sink"]
        c = {n: x.double().clone() for n, x in _caches(s).items()}
        c["weights"] = s["weights"].double()
        kept = torch.full((case["R"], Hkv, budget), -1, dtype=torch.int32)
        for r, n in enumerate(ctx):
            if n <= budget:
                continue
            ids = s["table"][r, :_pages(n, page)].long()
            for h in range(Hkv):
                w = c["weights"][ids, h].reshape(-1)[sink:n - recent].cpu()
                best = sorted(range(len(w)), key=lambda j, v=w.tolist(): (-v[j], j))[:budget - sink - recent]
                kept[r, h] = torch.tensor(list(range(sink)) + sorted(j + sink for j in best) + list(range(n - recent, n)), dtype=torch.int32)
                src = kept[r, h].long().to(_DEV)
                to = torch.arange(budget, device=_DEV)
                for x in c.values():
                    x[ids[to // page], h, to % page] = x[ids[src // page], h, src % page]
        return dict(kept=kept, new_lens=i32([min(n, budget) for n in ctx]), **c, **released(ctx, [min(n, budget) for n in ctx]))
    Hq, d = case["Hq"], case["d"]
    G = Hq // Hkv
    if 2 * d * Hq * sum(n * (c + n) for c, n in zip(ctx, new)) > 3e12:
        return None
    weights = s["weights"].double()
    t0 = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        L = c + n
        ids = s["table"][r, :_pages(L, page)].long()
        p, j = torch.arange(c, L, device=_DEV)[:, None], torch.arange(L, device=_DEV)
        hidden = (j > p) | ((j <= p - case["window"]) & (j >= case["sink"]) if case["window"] else torch.zeros_like(j > p))
        for h in range(Hkv):
            k = s["k_cache"][ids, h].reshape(-1, d)[:L]
            k = k.view(torch.float8_e4m3fn).double() * float(s["k_descale"]) if case["cache"] == "e4m3" else k.double()
            w = torch.zeros(L, dtype=torch.float64, device=_DEV)
            for g in range(G):
                x = s["q"][t0:t0 + n, h * G + g].double() @ k.T / math.sqrt(d) - s["lse"][t0:t0 + n, h * G + g, None].double()
                w += torch.exp(x).masked_fill(hidden, 0.0).sum(0)
            old = weights[ids, h].reshape(-1)
            old[:L] = torch.where(j < c, old[:L], 0.0) + w
            weights[ids, h] = old.view(len(ids), page)
        t0 += n
    return dict(weights=weights)
