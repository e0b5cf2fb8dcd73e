"""Plain 64-bit references of the paged-cache operators, and the tolerances that their tests use.

Error of an attention output against the reference (element by element).  Let
p_j be the softmax weights, A = sum_j p_j |v_j| and S the largest
scale * sum_i |q_i k_i| over the attended keys.
  * A score is a sum of d exact products accumulated in fp32 (d 2^-24 S and the
    same again for an order of summation that is not fixed), scaled and shifted
    in fp32 (2 roundings of at most S + max each), and exponentiated by ex2
    (2^-22 relative): every weight is within w = (2 d + 8) 2^-24 (S + 1) + 2^-21
    of its value, relatively, and so is their sum: 2 w A on the output.
  * many rows over an e4m3 cache: q as two e4m3 terms, after a scale that puts the
    row's largest element in [128, 256).  A term keeps four bits, so the two hold
    bf16's eight while the last of them is at least 2^-9, that is for elements of 2^-9
    of the largest or more; a smaller one is off by at most 2^-10, or 2^-17 of
    the largest: 2^-17 scale max|q| max_j sum_i |k_ji| on a score, on top of w.
  * P enters the second product rounded: one bf16 term eps/2 = 2^-8, two terms
    2^-16, one fp16 term 2^-11, two fp16 terms 2^-22, all relative; fp16 below
    2^-14 of the row's largest weight is fixed point with steps of 2^-24, half a
    step per key: n 2^-25 max|v|.  fp32 accumulation over n keys: its error
    grows like n 2^-24 A at most.
  * the result is rounded once: bf16 2^-8, fp32 2^-24 of the value.
lse: w + n 2^-24, and 2^-22 (|lse| + 1) for the logarithm and its scaling.
"""
import numpy as np
import torch


def plan(ctx, new, table, page, num_pages, free=None, head=0):
    """(table, cu, slots, positions, seq, next head) by plain loops."""
    table = [list(r) for r in table]
    cu, slots, pos = [0], [], []
    for r, (c, n) in enumerate(zip(ctx, new)):
        if free is not None:
            for b in range(-(-c // page), -(-(c + n) // page)):
                table[r][b] = int(free[head])
                head += 1
        for p in range(c, c + n):
            pg = table[r][p // page]
            slots.append(pg * page + p % page if 0 <= pg < num_pages else -1)
            pos.append(p)
        cu.append(cu[-1] + n)
    return table, cu, slots, pos, [c + n for c, n in zip(ctx, new)], head


def e4m3_values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def attend(q, k_cache, v_cache, table, ctx, new, scale, window=0, sink=0):
    """q double [T, Hq, d], caches double [P, Hkv, page, d]; returns o, lse, A, S, n per row."""
    T, Hq, d = q.shape
    _, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    o = torch.zeros(T, Hq, d, dtype=torch.float64)
    A = torch.zeros_like(o)
    lse = torch.full((T, Hq), -np.inf, dtype=torch.float64)
    S = torch.zeros(T, Hq, dtype=torch.float64)
    cnt = torch.zeros(T, 1, dtype=torch.float64)
    vmax = torch.zeros_like(o)
    QK = torch.zeros(T, Hq, dtype=torch.float64)
    loose = torch.zeros(T, Hq, d, dtype=torch.bool)
    t0 = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        L = c + n
        if n:       # columns of the request that hold a value that is not finite in some held page's token
            own = [(int(table[r][j // page]), j % page) for j in range(L) if int(table[r][j // page]) >= 0]
            pg, off = torch.tensor(own).T
            bad_k = (~torch.isfinite(k_cache[pg, :, off])).any(2).any(0)
            bad = (~torch.isfinite(v_cache[pg, :, off])).any(0) | bad_k[:, None]
            loose[t0:t0 + n] = bad.repeat_interleave(G, 0)
        for i in range(n):
            p = c + i
            j = np.arange(L)
            keep = j[(j <= p) & ((window == 0) | (j > p - window) | (j < sink))]
            pg = torch.tensor([int(table[r][x // page]) for x in keep])
            off = torch.tensor(keep % page)
            for h in range(Hkv):
                k, v = k_cache[pg, h, off], v_cache[pg, h, off]
                qq = q[t0 + i, h * G:(h + 1) * G]
                x = scale * qq @ k.T
                z = torch.logsumexp(x, 1)
                w = torch.exp(x - z[:, None])
                sl = slice(h * G, (h + 1) * G)
                o[t0 + i, sl] = w @ v
                A[t0 + i, sl] = w @ v.abs()
                lse[t0 + i, sl] = z
                S[t0 + i, sl] = scale * (qq.abs() @ k.abs().T).amax(1)
                QK[t0 + i, sl] = scale * qq.abs().amax(1) * k.abs().sum(1).max()
                vmax[t0 + i, sl] = v.abs().amax(0)
            cnt[t0 + i] = len(keep)
        t0 += n
    return dict(o=o, lse=lse, A=A, S=S, n=cnt, vmax=vmax, loose=loose, QK=QK)


def check_attention(ref, o, lse, d, p_err, fp16, q_terms=False):
    """Every element of o and lse (device tensors, rows of the step) within the bounds above."""
    got = o.double().cpu()
    # A value that is not finite (an e4m3 cast of torch's gives NaN above 464)
    # reaches every row that attends it; rows of the same request that do not may
    # have it too (the contract), so nothing is asked of those columns there.
    fin, loose = torch.isfinite(ref["o"]), ref["loose"]
    assert (torch.isfinite(got) == fin)[~loose].all() and not torch.isfinite(got)[~fin].any()
    fin = fin & torch.isfinite(got)
    w = (2 * d + 8) * 2.0 ** -24 * (ref["S"] + 1) + 2.0 ** -21
    if q_terms:
        w = w + 2.0 ** -17 * ref["QK"]
    out = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[o.dtype]
    tol = (2 * w + p_err + ref["n"] * 2.0 ** -24)[..., None] * ref["A"]
    if fp16:
        tol = tol + ref["n"][..., None] * 2.0 ** -25 * ref["vmax"]
    tol = tol * (1 + out) + out * ref["o"].abs() + 1e-30
    err = (got - ref["o"]).abs()
    err, tol = err[fin], tol[fin]
    assert (err <= tol).all(), f"o: worst error / bound {float((err / tol).max()):.3f}"
    ltol = w + ref["n"] * 2.0 ** -24 + 2.0 ** -22 * (ref["lse"].abs() + 1)
    lerr = (lse.double().cpu() - ref["lse"]).abs()
    assert (lerr <= ltol).all(), f"lse: worst error / bound {float((lerr / ltol).max()):.3f}"
    return float((err / tol).max())
