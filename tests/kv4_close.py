"""How near attention over the 4-bit cache has to be to 64 bits, tight enough
that a lost key shows among thousands.

For logits up to X in magnitude (natural units, before the softmax):

lse, fp32, row by row.  A logit's products are exact and its fp32 sums take at
most D/32 + D/G + 4 <= 20 roundings of partial sums up to about X, and the exp2
of it one more of X log2 e; errors of the keys are averaged, not added.  With
the sum's and the logarithm's own: 2^-24 (32 X + 8 (|lse| + 1)).

out.  e, what is off before the one rounding, is at most twice the logits' share
2^-24 32 X, and the two fp16 terms' 2^-22 of p s times codes up to 15, fp32 sums
of p s n and p lo of up to 31 s: with X <= 8 and s below |out|, 2^-15 of |out|.
Over values that lie anyhow between two numbers of the type, rounding x + e and
rounding x differ by |e| in the mean, by whole steps seldom rather than by e
always: so what is compared are outputs with the rounded reference, summed over
a call, with four steps of the largest for the chance of single ones.
"""
from __future__ import annotations

import numpy as np

STEP = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10}
MOST = 8.0  # X


def rounded(x, dt):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).to({"bf16": torch.bfloat16, "f16": torch.float16}[dt])
    return t.double().numpy()


def lse_off(got, want):
    """The largest error of lse as a share of what it may be; empty rows have to be empty."""
    empty = np.isneginf(want)
    if not np.array_equal(np.isneginf(got), empty):
        return np.inf
    off = np.abs(got[~empty] - want[~empty]) / (2.0 ** -24 * (32 * MOST + 8 * (np.abs(want[~empty]) + 1)))
    return float(off.max()) if off.size else 0.0


def out_off(got, want, dt):
    """The outputs' summed difference from the rounded reference as a share of what it may be."""
    near = rounded(want, dt)
    if not np.isfinite(got).all():
        return np.inf
    return float(np.abs(got - near).sum() / max(2.0 ** -15 * np.abs(want).sum() + 4 * STEP[dt] * np.abs(want).max(), 1e-30))


def inputs(shape_kv, shape_q, dt, seed):
    """k, v and q (torch, on the host) with logits |q.k| D^-1/2 up to about 5 and outputs that do not vanish."""
    import torch
    g = torch.Generator().manual_seed(seed)
    t = {"bf16": torch.bfloat16, "f16": torch.float16}[dt]
    k, v = torch.randn(shape_kv, generator=g), 0.5 * torch.randn(shape_kv, generator=g)
    mean = torch.rand(shape_kv[1:], generator=g) * 0.5 + 0.5
    v += torch.where(torch.rand(shape_kv[1:], generator=g) < 0.5, -mean, mean)
    return k.to(t), v.to(t), torch.randn(shape_q, generator=g).to(t)
