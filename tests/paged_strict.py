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


def check_attention(want, new, o, lse, *args):
    return ref.check_attention({**want, "loose": attended_loose(want, new)}, o, lse, *args)
