"""Plain 64-bit references of the operators around the attention of long conversations, and the tolerances that their
tests use.

Rotary: an angle is held to 2^-32 turns and rounded to fp32 within [-1/2, 1/2) turns (2^-26 turns; 2^-28 where the nearest
quarter is taken off first), so off by at most 2 pi (2^-32 + 2^-26) = 9.6e-8 rad; the frequency is a double after four roundings on either side: 2^-50 p theta rad
more; sine and cosine of it are within two units of the last place (2^-23), and times m rounded (2^-24): 2^-21 m in all.  Two
products and a sum in fp32: 3 x 2^-24 m (|a| + |b|).  The result is rounded once.
  bound = m (|a| + |b|) (2^-21 + 2^-22 + 2^-50 p theta) + half a step of the result.
Weights: a score is a sum of d exact products in fp32: within w = (2 d + 8) 2^-24 (S + 1) + 2^-21 (paged_ref), the log-sum-exp is
scaled in fp32 and subtracted (2^-22 (|lse| + 1)), and a sum of n positive terms in any order is within n 2^-24 of itself:
  bound = sum p (w + 2^-22 (|lse| + 1) + n 2^-24) + 2^-23 (old + sum);
q as two e4m3 terms: 2^-17 scale max|q| sum|k| on a score more.
"""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.uint8: 2.0 ** -4}


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=4096, slow=1.0, fast=32.0):
    out = []
    b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" else base
    for i in range(rot // 2):
        t = b ** (-2.0 * i / rot)
        if scaling == "linear":
            t /= factor
        if scaling == "yarn":
            g = min(1.0, max(0.0, (original * t / (2 * math.pi) - slow) / (fast - slow)))
            t *= g + (1 - g) / factor
        out.append(t)
    return torch.tensor(out, dtype=torch.float64), (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def rope(x, positions, theta, m, interleaved, inverse=False):
    """x double [..., d], positions [...] broadcast against it; the turned x and the bound without the last rounding."""
    rot = 2 * len(theta)
    angle = positions.double()[..., None] * theta
    c, s = angle.cos() * m, angle.sin() * m * (-1 if inverse else 1)
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., first], x[..., second]
    y, tol = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    e = abs(m) * (a.abs() + b.abs()) * (2.0 ** -21 + 2.0 ** -22 + 2.0 ** -50 * angle.abs())
    tol[..., first], tol[..., second] = e, e
    return y, tol


def weights(q, k_cache, lse, old, table, ctx, new, scale, window=0, sink=0, q_terms=()):
    """New pool of weights [P, Hkv, page] (double) and the bound of every entry; q double [T, Hq, d], caches double,
    lse double [T, Hq]; q_terms: requests whose q enters as two e4m3 terms."""
    T, Hq, d = q.shape
    P, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    out, tol = old.clone(), torch.zeros_like(old)
    t0 = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        if n == 0:
            continue
        j, p = torch.arange(c + n), torch.arange(c, c + n)[:, None]
        see = (j <= p) & ((j > p - window) | (j < sink) if window else torch.ones_like(j <= p))
        keys = torch.nonzero(see.any(0))[:, 0]
        pg, off = torch.tensor([int(table[r][int(x) // page]) for x in keys]), keys % page
        for h in range(Hkv):
            k = k_cache[pg, h, off]
            w, e = torch.zeros(len(keys), dtype=torch.float64), torch.zeros(len(keys), dtype=torch.float64)
            for g in range(h * G, (h + 1) * G):
                qq, z = q[t0:t0 + n, g], lse[t0:t0 + n, g, None]
                x = torch.exp(scale * qq @ k.T - z) * see[:, keys]
                rel = (2 * d + 8) * 2.0 ** -24 * (scale * qq.abs() @ k.abs().T + 1) + 2.0 ** -21 + 2.0 ** -22 * (z.abs() + 1) + n * G * 2.0 ** -24
                if r in q_terms:
                    rel = rel + 2.0 ** -17 * scale * qq.abs().amax(1, keepdim=True) * k.abs().sum(1)
                w += x.sum(0)
                e += (x * rel).sum(0)
            fresh = keys >= c
            before = torch.where(fresh, 0.0, out[pg, h, off])
            out[pg, h, off] = before + w
            tol[pg, h, off] += e + 2.0 ** -23 * (before.abs() + w)
        t0 += n
    return out, tol


def kept_places(w, length, budget, recent, sink):
    """Places that one head of one request keeps; w: its weights, a list."""
    rank = lambda x: math.inf if x != x else x  # noqa: E731
    # NaN counts as the largest, above infinity.
    order = sorted(range(sink, length - recent), key=lambda j: (0 if w[j] != w[j] else 1, -rank(w[j]), j))
    return sorted(list(range(sink)) + order[:budget - sink - recent] + list(range(length - recent, length)))


def released(held, lens, table, page, free, head):
    back = [table[r][b] for r in range(len(lens)) for b in range(-(-lens[r] // page), -(-held[r] // page))]
    free = list(free)
    free[head - len(back):head] = back
    return free, head - len(back)


def verify(target, draft, tokens, u_accept, u_sample, cu):
    """(out, n_out) by plain loops; probabilities double [T, V]."""
    out, n_out = [], []
    for r in range(len(cu) - 1):
        b, n = cu[r], cu[r + 1] - cu[r]
        if n == 0:
            n_out.append(0)
            continue
        a = 0
        while a < n - 1:
            t = tokens[b + a + 1]
            q = 1.0 if draft is None else float(draft[b + a, t])
            if not u_accept[b + a] * q < float(target[b + a, t]):
                break
            a += 1
        p = target[b + a].clamp_min(0.0)
        w = p.clone()
        if a < n - 1:
            if draft is None:
                w[tokens[b + a + 1]] = 0.0
            else:
                w = (target[b + a] - draft[b + a]).clamp_min(0.0)
            if float(w.sum()) == 0.0:
                w = p
        total = math.fsum(w.tolist())
        run, x = 0.0, -1
        for i, y in enumerate(w.tolist()):
            run += y
            if y > 0 and run > u_sample[r] * total:
                x = i
                break
        out += [tokens[b + 1 + i] for i in range(a)] + [x] + [-1] * (n - 1 - a)
        n_out.append(a + 1)
    return out, n_out
