"""Operators of serving over a paged key/value cache, in plain torch and through the package.

Three operators: the step's plan (block tables, slot map, positions from request lengths), the append of new keys and
values to the cache's pages, and the attention of every request's new tokens over its cached keys.  With ``own`` false
they are computed by elementary torch operations in 32 bits; with ``own`` true by the calls a user makes.
"""
import math
import random

import torch

own = False

_DEV = "cuda"


def listed():
    def plan(name, **kw):
        return dict(dict(op="plan", name=name, ctx_max=8192, Hq=32, Hkv=8, d=128, page=64, window=0, sink=0, lens=1), **kw)

    def append(name, **kw):
        return dict(dict(op="append", name=name, ctx_max=8192, Hkv=8, d=128, page=64, cache="bf16", lens=1), **kw)

    def attend(name, **kw):
        return dict(dict(op="attend", name=name, Hq=32, Hkv=8, d=128, page=64, window=0, sink=0, cache="bf16", out="bf16",
                         lens=1), **kw)

    return [
        # One decoding step of 256 requests: every request gets one slot, a few get a new page.
        plan("plan_decode", R=256, q_max=1),
        # A step of ragged prompt chunks: tens of thousands of slots and hundreds of new pages.
        plan("plan_prompts", R=48, q_max=2048, ctx_max=32768, page=16, lens=2),
        # The new tokens of a small decoding batch: 33 rows, all latency.
        append("append_decode", R=33, q_max=1),
        # Prompt chunks written as bf16.
        append("append_prompts", R=12, q_max=4096, ctx_max=16384, lens=3),
        # Prompt chunks quantised to e4m3 as they are written, 16-token pages.
        append("append_prompts_e4m3", R=12, q_max=4096, ctx_max=16384, page=16, cache="e4m3", lens=4),
        # Two short chats: the smallest call.
        attend("decode_small", R=2, q_max=1, ctx_max=500, d=64, page=16, lens=5),
        # One request of 128K tokens, 8 heads of its own keys each: split over the long axis.
        attend("decode_128k", R=1, q_max=1, ctx_max=131071, Hq=8, Hkv=8, out="f32", lens=6),
        # A serving batch: 96 requests of ragged lengths, 4 query heads to a key head.
        attend("decode_batch", R=96, q_max=1, ctx_max=16000, lens=7),
        # The same kind of batch on an e4m3 cache with small pages, two tokens a request (one guessed ahead).
        attend("decode_batch_e4m3", R=64, q_max=2, ctx_max=16000, page=16, cache="e4m3", lens=8),
        # Two long prompts' chunks after a cached prefix: matrix work.
        attend("chunk_long", R=2, q_max=4096, ctx_max=12000, lens=9),
        # Chunks of every size next to single tokens, e4m3 cache, 7 query heads to a key head.
        attend("chunk_mixed_e4m3", R=8, q_max=512, ctx_max=7500, Hq=28, Hkv=4, page=32, cache="e4m3", lens=10),
        # A streaming chunk with a window of 1024 and 10 kept first tokens, 16 heads of 32K tokens.
        attend("chunk_window", R=1, q_max=2048, ctx_max=30700, Hq=16, Hkv=16, page=128, window=1024, sink=10, lens=11),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    lens = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128])
    d = rng.choice([64, 128])
    op = rng.choice(["plan", "append", "attend", "attend", "attend"])
    if op == "plan":
        Hq, Hkv = rng.choice([(8, 8), (32, 8), (12, 4), (16, 1)])
        R, q_max = _log(rng, 1, 512), _log(rng, 1, 2048)
        q_max = max(1, min(q_max, 98304 // R))
        return dict(op=op, R=R, q_max=q_max, ctx_max=_log(rng, 1, 65536), Hq=Hq, Hkv=Hkv, d=d, page=page,
                    window=rng.choice([0, 0, 512]), sink=rng.choice([0, 4]), lens=lens)
    if op == "append":
        R, q_max = _log(rng, 1, 128), _log(rng, 1, 4096)
        q_max = max(1, min(q_max, 49152 // R))
        return dict(op=op, R=R, q_max=q_max, ctx_max=_log(rng, 1, 8192), Hkv=rng.choice([1, 2, 5, 8]), d=d, page=page,
                    cache=rng.choice(["bf16", "e4m3"]), lens=lens)
    Hq, Hkv = rng.choice([(8, 8), (16, 16), (32, 8), (12, 4), (28, 4), (10, 2), (16, 1), (5, 5)])
    q_max = rng.choice([1, 1, _log(rng, 2, 8), _log(rng, 9, 3000)])
    ctx_max = _log(rng, 1, 100000 if q_max == 1 else 16000)
    R = _log(rng, 1, 96)
    keys = ctx_max + q_max
    R = max(1, min(R, 1_000_000_000 // (keys * Hkv * d), 2_000_000_000 // (Hq * q_max * keys)))
    window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    return dict(op=op, R=R, q_max=q_max, ctx_max=ctx_max, Hq=Hq, Hkv=Hkv, d=d, page=page, window=window,
                sink=rng.choice([0, 4, 10]) if window else 0, cache=rng.choice(["bf16", "bf16", "e4m3"]),
                out=rng.choice(["bf16", "bf16", "f32"]), lens=lens)


def _lens(case):
    """Cached and new tokens of every request: request 0 has the largest of both, the others are spread below."""
    rng = random.Random(case["lens"])
    ctx = [case["ctx_max"]] + [_log(rng, max(1, case["ctx_max"] // 16), case["ctx_max"]) for _ in range(case["R"] - 1)]
    new = [case["q_max"]] + [_log(rng, max(1, case["q_max"] // 512), case["q_max"]) for _ in range(case["R"] - 1)]
    return ctx, new


def _pages(tokens, page):
    return -(-tokens // page)


def prepare(case, seed):
    g = torch.Generator(device=_DEV).manual_seed(seed)
    R, page, Hkv, d = case["R"], case["page"], case["Hkv"], case["d"]
    ctx, new = _lens(case)
    T, full = sum(new), [_pages(c + n, page) for c, n in zip(ctx, new)]
    num_pages = sum(full) + 3
    s = dict(case=case, page=page, T=T, num_pages=num_pages, max_pages=max(full) + 1, q_max=max(new),
             k_max=max(c + n for c, n in zip(ctx, new)))
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=_DEV)
    s["new"] = torch.tensor(new, dtype=torch.int32, device=_DEV)
    # Pages of the pool in the order in which a server that has run for a while has them: any order.
    order = torch.randperm(num_pages, generator=g, device=_DEV).to(torch.int32)
    held = full if case["op"] != "plan" else [_pages(c, page) for c in ctx]
    table = torch.full((R, s["max_pages"]), -1, dtype=torch.int32, device=_DEV)
    col = torch.arange(s["max_pages"], device=_DEV)[None, :]
    has = col < torch.tensor(held, device=_DEV)[:, None]
    table[has] = order[: sum(held)]
    s["table"] = table
    if case["op"] == "plan":
        s["free"] = torch.cat([order[sum(held):], order[: sum(held)]])  # what is held is not looked at
        s["head"] = torch.zeros(1, dtype=torch.int32, device=_DEV)
        if own:
            from long_context_fm_gb300 import fm
            s["step"] = fm.PagedAttention(R, case["Hq"], Hkv, d, page, num_pages, s["max_pages"], T, s["q_max"],
                                          window=case["window"], sink=case["sink"])
        return s
    shape = (num_pages, Hkv, page, d)
    e4m3 = case["cache"] == "e4m3"
    if e4m3:
        s["k_descale"] = torch.tensor([4.0 / 448.0 * 1.5], device=_DEV)
        s["v_descale"] = torch.tensor([4.0 / 448.0 * 1.25], device=_DEV)
    for n in ("k", "v"):
        x = torch.empty(shape, dtype=torch.bfloat16, device=_DEV).normal_(generator=g)
        s[n + "_cache"] = (x / s[n + "_descale"].to(torch.bfloat16)).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else x
    if case["op"] == "append":
        # One projection's output holds the keys and the values: rows of 2 Hkv heads.
        kv = torch.empty(T, 2 * Hkv, d, dtype=torch.bfloat16, device=_DEV).normal_(generator=g)
        s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
        s["slots"] = _plan(s)["slots"]
        if own:
            s["status"] = torch.zeros(1, dtype=torch.int32, device=_DEV)
        return s
    s["q"] = torch.empty(T, case["Hq"], d, dtype=torch.bfloat16, device=_DEV).normal_(generator=g).mul_(1.5)
    s["out"] = torch.float32 if case["out"] == "f32" else torch.bfloat16
    s["scale"] = 1.0 / math.sqrt(d)
    if own:
        # The step's plan serves every layer of the model.
        from long_context_fm_gb300 import fm
        s["step"] = fm.PagedAttention(R, case["Hq"], Hkv, d, page, num_pages, s["max_pages"], T, s["q_max"],
                                      window=case["window"], sink=case["sink"])
        s["step"].plan(s["ctx"], s["new"], s["table"])
    return s


def _plan(s):
    """Plain form of the plan: pages from the free list (where there is one), slots and positions."""
    page, T, ctx, new = s["page"], s["T"], s["ctx"].long(), s["new"].long()
    zero = torch.zeros(1, dtype=torch.int64, device=_DEV)
    have, want = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    cu = torch.cat([zero, new.cumsum(0)])
    off = torch.cat([zero, (want - have).cumsum(0)])
    table = s["table"]
    if "free" in s:
        col = torch.arange(table.shape[1], device=_DEV)[None, :]
        at = s["head"].long() + off[:-1, None] + col - have[:, None]
        table = torch.where((col >= have[:, None]) & (col < want[:, None]), s["free"][at.clamp(0, s["num_pages"] - 1)], table)
    row = torch.repeat_interleave(torch.arange(len(ctx), device=_DEV), new, output_size=T)
    pos = torch.arange(T, device=_DEV) - cu[row] + ctx[row]
    slots = table[row, pos // page].long() * page + pos % page
    r = dict(table=table, cu_q=cu.int(), slots=slots, positions=pos.int(), seq_lens=(ctx + new).int())
    if "free" in s:
        r["free_next"] = s["head"] + off[-1:].int()
    return r


def _append(s):
    page, slots = s["page"], s["slots"]
    at = (slots // page, slice(None), slots % page)
    for n in ("k", "v"):
        x = s[n]
        if n + "_descale" in s:
            x = (x.float() / s[n + "_descale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        s[n + "_cache"][at] = x
    return _caches(s)


def _caches(s):
    """Both caches; codes as the values they stand for (in units of the descale)."""
    if "k_descale" in s:
        return {n: s[n + "_cache"].view(torch.float8_e4m3fn) for n in ("k", "v")}
    return {n: s[n + "_cache"] for n in ("k", "v")}


def _attend(s):
    case, page, q_max, k_max, T = s["case"], s["page"], s["q_max"], s["k_max"], s["T"]
    R, Hq, Hkv, d = case["R"], case["Hq"], case["Hkv"], case["d"]
    G = Hq // Hkv
    ctx, new = s["ctx"].long(), s["new"].long()
    key = torch.arange(k_max, device=_DEV)
    pages = s["table"].long()[:, key // page].clamp_min(0)  # [R, k_max]
    inside = key[None, :] < (ctx + new)[:, None]
    k, v = ((_values(s, n)[pages, :, key % page]).transpose(1, 2) for n in ("k", "v"))  # [R, Hkv, k_max, d]
    v = torch.where(inside[:, None, :, None], v, 0.0)
    i = torch.arange(q_max, device=_DEV)
    first = new.cumsum(0) - new
    valid = i[None, :] < new[:, None]
    tok = torch.where(valid, first[:, None] + i[None, :], 0)  # [R, q_max]
    q = s["q"][tok].float().view(R, q_max, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(R, Hkv, G * q_max, d)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    pos = ctx[:, None] + i[None, :]
    see = key[None, None, :] <= pos[:, :, None]
    if case["window"]:
        see = see & ((key[None, None, :] > pos[:, :, None] - case["window"]) | (key[None, None, :] < case["sink"]))
    x = x.view(R, Hkv, G, q_max, k_max).masked_fill_(~(see & inside[:, None, :])[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(R, Hkv, G * q_max, k_max), v).view(R, Hkv, G, q_max, d) / total
    lse = (m + total.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(R, q_max, Hq, d)[valid]
    lse = lse.permute(0, 3, 1, 2).reshape(R, q_max, Hq)[valid]
    return dict(o=o.to(s["out"]), lse=lse)


def _values(s, n):
    x = s[n + "_cache"]
    return x.view(torch.float8_e4m3fn).float() * s[n + "_descale"] if n + "_descale" in s else x.float()


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return dict(plan=_plan, append=_append, attend=_attend)[op](s)
    if op == "plan":
        p = s["step"]
        p.plan(s["ctx"], s["new"], s["table"], free_pages=s["free"], free_head=s["head"])
        return dict(table=s["table"], cu_q=p.cu_q, slots=p.slots, positions=p.positions, seq_lens=p.seq_lens,
                    free_next=p.free_next)
    if op == "append":
        from long_context_fm_gb300 import fm
        fm.fm_paged_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["status"],
                           k_descale=s.get("k_descale"), v_descale=s.get("v_descale"))
        return _caches(s)
    o, lse = s["step"].attend(s["q"], s["k_cache"], s["v_cache"], s["table"], s["scale"], o_dtype=s["out"],
                              k_descale=s.get("k_descale"), v_descale=s.get("v_descale"))
    return dict(o=o, lse=lse)


def _pairs(ctx, new, window, sink):
    """Attended (row, key) pairs of one head, and the keys that some row attends."""
    if not window:
        return sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new)), sum(c + n for c, n in zip(ctx, new))
    pairs = sum(min(p + 1, window + min(sink, max(0, p + 1 - window))) for c, n in zip(ctx, new) for p in range(c, c + n))
    return pairs, sum(min(c + n, n + window - 1 + sink) for c, n in zip(ctx, new))


def work(case):
    ctx, new = _lens(case)
    T, R, page, Hkv, d = sum(new), case["R"], case["page"], case["Hkv"], case["d"]
    if case["op"] == "plan":
        fresh = sum(_pages(c + n, page) - _pages(c, page) for c, n in zip(ctx, new))
        return dict(bytes=8 * R + 4 * R + 8 * fresh + 12 * T + 4 * (2 * R + 1) + 8, flops=0)
    esz = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        return dict(bytes=2 * T * Hkv * d * (2 + esz) + 8 * T, flops=0)
    pairs, keys = _pairs(ctx, new, case["window"], case["sink"])
    Hq = case["Hq"]
    osz = 4 if case["out"] == "f32" else 2
    return dict(bytes=2 * keys * Hkv * d * esz + T * Hq * (d * (2 + osz) + 4) + 4 * sum(_pages(c + n, page) for c, n in zip(ctx, new)),
                flops=4 * d * Hq * pairs)


def _nearest_e4m3(x):
    """The e4m3 value nearest to x (ties to the even code), in 64 bits."""
    x = x.clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    ctx, new = _lens(case)
    page, table = case["page"], s["table"].tolist()
    if case["op"] == "plan":
        free, at, t = s["free"].tolist(), 0, 0
        slots, positions, cu = [], [], [0]
        for r, (c, n) in enumerate(zip(ctx, new)):
            for b in range(_pages(c, page), _pages(c + n, page)):
                table[r][b] = free[at]
                at += 1
            positions += range(c, c + n)
            slots += [table[r][p // page] * page + p % page for p in range(c, c + n)]
            t += n
            cu.append(t)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
        return dict(table=i32(table), cu_q=i32(cu), slots=torch.tensor(slots), positions=i32(positions),
                    seq_lens=i32([c + n for c, n in zip(ctx, new)]), free_next=i32([at]))
    if case["op"] == "append":
        found = {}
        slots = s["slots"].cpu()
        for n in ("k", "v"):
            c, x = s[n + "_cache"].cpu(), s[n].cpu().double()
            if case["cache"] == "e4m3":
                c = c.view(torch.float8_e4m3fn)
                x = _nearest_e4m3(x / float(s[n + "_descale"]))
            c = c.double()
            c[torch.div(slots, page, rounding_mode="floor"), :, slots % page] = x
            found[n] = c
        return found
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    G = Hq // Hkv
    if 4 * d * Hq * sum(n * (c + n) for c, n in zip(ctx, new)) > 6e12:
        return None
    o = torch.empty(s["T"], Hq, d, dtype=torch.float64, device=_DEV)
    lse = torch.empty(s["T"], Hq, dtype=torch.float64, device=_DEV)
    t0 = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        L = c + n
        ids = s["table"][r, : _pages(L, page)].long()
        p = torch.arange(c, L, device=_DEV)[:, None]
        j = torch.arange(L, device=_DEV)[None, :]
        hidden = (j > p) | ((j <= p - case["window"]) & (j >= case["sink"]) if case["window"] else torch.zeros_like(j > p))
        for h in range(Hkv):
            k, v = (s[x + "_cache"][ids, h].reshape(-1, d)[:L] for x in ("k", "v"))
            if case["cache"] == "e4m3":
                k, v = (x.view(torch.float8_e4m3fn).double() * float(s[y]) for x, y in ((k, "k_descale"), (v, "v_descale")))
            k, v = k.double(), v.double()
            for g in range(G):
                x = s["q"][t0:t0 + n, h * G + g].double() @ k.T / math.sqrt(d)
                x[hidden] = -math.inf
                z = torch.logsumexp(x, 1)
                lse[t0:t0 + n, h * G + g] = z
                o[t0:t0 + n, h * G + g] = torch.exp(x - z[:, None]) @ v
        t0 += n
    return dict(o=o, lse=lse)
