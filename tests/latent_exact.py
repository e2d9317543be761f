"""Chunks over a latent cache whose logits are exact in 32 bits, so that a result shows how its probabilities were rounded.

Queries and cached values are small whole numbers and the softmax scale is a power of two: a logit is a sum of r + 64
products under 2^12 in size, exact in any order, and few base-2 units from the others.  What is left of the error is the
result's rounding and P's."""

from __future__ import annotations

import math

import torch

import latent_ref as R

SCALE = 2.0 ** -7
CASES = [  # H, r, lens, new: up to 32 rows (both values in one operand), 33 to 64 (two operands), more (two CTAs)
    (1, 512, [6], [1]), (5, 256, [3], [1]), (16, 512, [20, 7], [1, 1]), (32, 512, [5], [1]), (32, 256, [17], [1]),
    (10, 512, [9], [3]), (33, 512, [9], [1]), (48, 256, [20], [1]), (64, 512, [3, 13], [1, 1]), (20, 512, [18], [3]),
    (65, 256, [11], [1]), (128, 512, [20], [1]), (16, 512, [70, 200], [1, 2]), (64, 256, [130, 300], [1, 1]),
]


def chunk(H, r, lens, new, dt):
    c = R.Latent(H, r, 16, dt, lens, new, seed=H + r)
    g = torch.Generator().manual_seed(H * r + lens[0])
    c.q_lat = torch.randint(-2, 3, c.q_lat.shape, generator=g).to(c.q_lat.dtype)
    live = ~torch.isnan(c.pool)
    c.pool = torch.where(live, torch.randint(-3, 4, c.pool.shape, generator=g).to(c.pool.dtype), c.pool)
    c.scale = SCALE
    return c


def rows(c):
    """Per row t: (t, base-2 logits [H][tokens seen], values [tokens seen][r]), in 64 bits."""
    for b, L in enumerate(c.lens):
        kv = c.tokens(b)
        for i in range(c.new[b]):
            t, seen = c.starts[b] + i, L - c.new[b] + i + 1
            yield t, c.q_lat[t].to(R.F64) @ kv[:seen].T * (SCALE / math.log(2.0)), kv[:seen, : c.r]


def attention(c, parts):
    """o_lat and how far a result may be from it.

    TOLERANCES.  e = eps / 2 of the type, p the normalised probabilities, A = sum p |c|, F a row's largest base-2 logit in
    size.  The result's rounding: e |o| (fp16: and 2^-25).  P's: e^2 A with two values, e A with one (fp16 holds p, of
    which a row's largest is 2^7, with a half step of 2^-25 at least: 2^-32 sum |c|).  A base-2 logit is an exact number
    times a rounded constant, rounded (2^-24 F each); the running maximum taken from it is another 2^-24 (F + 7), the
    difference 2^-24 (2 F + 7); exp2 is good to 2^-22, and so are the weights of parts that are joined: every p is off by
    dz = 2^-21 + 2^-24 (4 F + 10) of itself, which moves o by at most 2 dz A.  No maximum is raised after its first step
    (asserted: the logits are within 8 of that step's largest).  Sums of L terms, twice with two values: (2 L + 16) 2^-24 A."""
    e = torch.finfo(R.DT[c.dt]).eps / 2
    out = torch.zeros((c.T, c.H, c.r), dtype=R.F64)
    tol = torch.zeros_like(out)
    for t, f, v in rows(c):
        assert bool((f.amax(dim=1) - f[:, :64].amax(dim=1) < 7.9).all())
        p = torch.softmax(f * math.log(2.0), dim=1)
        o, A = p @ v, p @ v.abs()
        dz = 2.0 ** -21 + 2.0 ** -24 * (4 * f.abs().amax(dim=1, keepdim=True) + 10)
        x = e * o.abs() + (e * e if parts == 2 else e) * A + 2 * dz * A + (2 * len(v) + 16) * 2.0 ** -24 * A
        if c.dt == "f16":
            x = x + 2.0 ** -32 * v.abs().sum(dim=0) + 2.0 ** -25
        out[t], tol[t] = o, 1.01 * x
    return out, tol


def modelled(c, weights):
    """The operator with P as weights(hi, lo) of its two 16-bit values, all else exact but the result's rounding."""
    dt = R.DT[c.dt]
    out = torch.zeros((c.T, c.H, c.r), dtype=R.F64)
    for t, f, v in rows(c):
        p = torch.exp2(f - f.amax(dim=1, keepdim=True) + 7)
        hi = p.to(dt).to(R.F64)
        lo = (p - hi).to(dt).to(R.F64)
        out[t] = ((weights(hi, lo) @ v) / p.sum(dim=1, keepdim=True)).to(dt).to(R.F64)
    return out
