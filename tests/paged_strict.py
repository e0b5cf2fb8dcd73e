"""The element-by-element check of paged_ref, asking for a finite value wherever what is attended is finite.

paged_ref.attend excuses a column for a whole request as soon as one of its held tokens is not finite there,
attended or not.  Excused here are only columns in which a key that some row of the request attends is not finite: those alone may
spread to rows of the same request that do not attend it."""
import torch

import paged_ref as ref


def attended_loose(want, new):
    """[T, Hq, d]: columns in which some row of the same request has a reference that is not finite."""
    loose = torch.zeros_like(want["o"], dtype=torch.bool)
    t0 = 0
    for n in new:
        if n:
            loose[t0:t0 + n] = (~torch.isfinite(want["o"][t0:t0 + n])).any(0)
        t0 += n
    return loose


def check_attention(want, new, o, lse, d, p_err, fp16=False, q_terms=False):
    """paged_ref.check_attention with those columns excused, and with fp16 weights held to half a step of 2^-31 of the row's
    largest (they are lifted by 2^7) in place of 2^-24."""
    worst = ref.check_attention({**want, "loose": attended_loose(want, new)}, o, lse, d, p_err, fp16, q_terms)
    if not fp16:
        return worst
    w = (2 * d + 8) * 2.0 ** -24 * (want["S"] + 1) + 2.0 ** -21
    if q_terms:
        w = w + 2.0 ** -17 * want["QK"]
    out = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[o.dtype]
    tol = (2 * w + p_err + want["n"] * 2.0 ** -24)[..., None] * want["A"] + want["n"][..., None] * 2.0 ** -32 * want["vmax"]
    tol = tol * (1 + out) + out * want["o"].abs() + 1e-30
    got = o.double().cpu()
    fin = torch.isfinite(want["o"]) & torch.isfinite(got)
    part = ((got - want["o"]).abs() / tol)[fin]
    assert (part <= 1).all(), f"o: worst error / bound {float(part.max()):.3f}"
    return float(part.max())
