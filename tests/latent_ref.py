"""Plain 64-bit forms of the latent-cache operators, and seeded inputs for
their tests.  Everything runs on the CPU in float64 from the definitions."""

from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from paged_ref import DT, F64, rope_freqs, rotate, rotate_tol


@dataclass
class Latent:
    """A ragged chunk over a paged cache of latent vectors; tensors live on the CPU."""

    H: int
    r: int
    S: int
    dt: str
    lens: list
    new: list
    dn: int = 128
    dv: int = 128
    pad_rows: int = 0
    extra_pages: int = 0
    mp: int = 0
    seed: int = 0
    poison: float = float("nan")
    dr: int = 64

    def __post_init__(self):
        g = torch.Generator().manual_seed(self.seed + 29)
        B, S = len(self.lens), self.S
        pages = [-(-L // S) for L in self.lens]
        self.mp = max(self.mp, max(pages + [1]))
        self.n_phys = sum(pages) + self.extra_pages + 1
        perm = torch.randperm(self.n_phys, generator=g)
        self.page_table = torch.full((B, self.mp), -1, dtype=torch.int32)
        at = 0
        live = torch.zeros((self.n_phys, S), dtype=torch.bool)
        for b, L in enumerate(self.lens):
            self.page_table[b, : pages[b]] = perm[at : at + pages[b]].int()
            at += pages[b]
            for t0 in range(0, L, S):
                live[int(self.page_table[b, t0 // S]), : min(S, L - t0)] = True
        self.starts = [0]
        for n in self.new:
            self.starts.append(self.starts[-1] + n)
        self.T = self.starts[-1] + self.pad_rows
        self.q_start = torch.tensor(self.starts, dtype=torch.int32)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32)
        dt = DT[self.dt]
        rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.pool = rand(self.n_phys, S, self.r + self.dr).to(dt)
        # slots that hold no token: whatever the pool holds must not matter
        self.pool[~live] = self.poison
        self.q_lat = rand(self.T, self.H, self.r + self.dr).to(dt)
        self.q = rand(self.T, self.H, self.dn + self.dr).to(dt)
        self.kv = rand(self.T, self.r + self.dr).to(dt)  # the down-projection's output
        self.w_kv = (rand(self.H, self.dn + self.dv, self.r) / math.sqrt(self.r)).to(dt)
        self.norm = (1.0 + 0.1 * rand(self.r)).to(dt)
        self.scale = 1.0 / math.sqrt(self.dn + self.dr)

    def params(self, spg, **kw):
        a = dict(batch=len(self.lens), num_heads=self.H, latent_dim=self.r, rope_dim=self.dr, nope_dim=self.dn,
                 v_dim=self.dv, page_size=self.S, num_phys_pages=self.n_phys, max_pages_per_seq=self.mp, dtype=self.dt)
        a.update(kw)
        return spg.make_latent_params(**a)

    def tokens(self, b):
        L = self.lens[b]
        return self.pool[self.page_table[b, : -(-L // self.S)].long()].reshape(-1, self.r + self.dr)[:L].to(F64)


def attention(c: Latent, drop=(), parts=2):
    """o_lat, lse and how far a 16-bit result may be from them.

    drop: (b, page) pairs whose tokens take no part.

    TOLERANCES.  e = eps / 2 of the type, p the normalised probabilities, A = sum p |c|.  Rounding the result costs
    e |o|; p enters as two values, so its rounding costs e^2 A (one value: e A).  A logit is a sum of r + dr products in
    32 bits, off by at most (r + dr) 2^-24 sum |q k| scale; the exponent's argument adds a few 2^-24 |z| and 2^-22 of
    exp2 itself; a relative error dz of every p moves o by at most 2 dz A.  O is a sum of L terms (twice with two
    values) in 32 bits.  fp16 holds the unnormalised p, of which a row's largest is at least 2^7, with an absolute half
    step of 2^-25, and the result with one of 2^-25."""
    H, r = c.H, c.r
    out = torch.zeros((c.T, H, r), dtype=F64)
    tol = torch.zeros_like(out)
    lse = torch.full((c.T, H), -math.inf, dtype=F64)
    lse_tol = torch.zeros_like(lse)
    e = torch.finfo(DT[c.dt]).eps / 2
    for b, L in enumerate(c.lens):
        lo, n = c.starts[b], c.new[b]
        if n == 0:
            continue
        kv = c.tokens(b)
        gone = torch.zeros(L, dtype=torch.bool)
        for bb, pg in drop:
            if bb == b:
                gone[pg * c.S : (pg + 1) * c.S] = True
        kv = kv.masked_fill(gone[:, None], 0.0)
        q = c.q_lat[lo : lo + n].to(F64)
        z = torch.einsum("nhc,tc->nht", q, kv) * c.scale
        size = torch.einsum("nhc,tc->nht", q.abs(), kv.abs()) * c.scale
        hidden = torch.arange(L)[None] > torch.arange(L - n, L)[:, None]
        z = z.masked_fill((hidden | gone[None])[:, None], -math.inf)
        ls = torch.logsumexp(z, dim=2)
        fin = torch.isfinite(ls)
        p = torch.exp(z - torch.where(fin, ls, 0.0)[..., None])
        p = torch.where(torch.isfinite(z), p, torch.zeros_like(p))
        v = kv[:, :r]
        o, A = p @ v, p @ v.abs()
        zmax = z.masked_fill(~torch.isfinite(z), 0.0).abs().amax(dim=2)
        dz = (r + c.dr) * 2.0 ** -24 * size.amax(dim=2) + 8 * 2.0 ** -24 * (zmax + 1) + 2.0 ** -22
        t = e * o.abs() + (e * e if parts == 2 else e) * A + 2 * dz[..., None] * A + (2 * L + 8) * 2.0 ** -24 * A
        if c.dt == "f16":
            t = t + 2.0 ** -32 * v.abs().sum(dim=0) + 2.0 ** -25
        out[lo : lo + n], tol[lo : lo + n], lse[lo : lo + n] = o, 1.01 * t, ls
        lse_tol[lo : lo + n] = dz + (L + 8) * 2.0 ** -24 + 8 * 2.0 ** -24 * (1 + torch.where(fin, ls.abs(), 0.0))
    return out, tol, lse, lse_tol


def rounded(y, size, k, dt):
    """How far a sum of k products of total size `size` in 32 bits, rounded to dt, may be from y.  (A product unit may
    cut its sums instead of rounding them: 2^-23 of them each.)"""
    e = torch.finfo(DT[dt]).eps / 2
    t = e * y.abs() + 1.01 * k * 2.0 ** -23 * size
    return t + (2.0 ** -25 if dt == "f16" else 0.0)


def absorb(c: Latent):
    q, w = c.q[..., : c.dn].to(F64), c.w_kv[:, : c.dn].to(F64)
    y = torch.einsum("thd,hdc->thc", q, w)
    return y, rounded(y, torch.einsum("thd,hdc->thc", q.abs(), w.abs()), c.dn, c.dt)


def project(c: Latent, o_lat):
    o, w = o_lat.to(F64), c.w_kv[:, c.dn :].to(F64)
    y = torch.einsum("thc,hvc->thv", o, w)
    return y, rounded(y, torch.einsum("thc,hvc->thv", o.abs(), w.abs()), c.r, c.dt)


def append(c: Latent, rot, layout, inv, m, eps, norm=True, positions=None):
    """Pool rows [T][r + dr] and rotated queries [T][H][dr] of the rows that belong to a sequence, with tolerances: a
    mean of r squares in 32 bits and an inverse root good to 2^-22 (half of the former's error), three products; the turn
    as in paged_ref.  Rows of no sequence are NaN."""
    e = torch.finfo(DT[c.dt]).eps / 2
    row = torch.full((c.T, c.r + c.dr), math.nan, dtype=F64)
    row_tol = torch.zeros_like(row)
    q = torch.full((c.T, c.H, c.dr), math.nan, dtype=F64)
    q_tol = torch.zeros_like(q)
    tiny = 2.0 ** -25 if c.dt == "f16" else 0.0
    for b, L in enumerate(c.lens):
        lo, n = c.starts[b], c.new[b]
        pos = torch.arange(L - n, L) if positions is None else positions[lo : lo + n].long()
        x = c.kv[lo : lo + n, : c.r].to(F64)
        rel = 0.0
        if norm:
            x = x / torch.sqrt(x.square().mean(dim=1, keepdim=True) + eps) * c.norm.to(F64)
            rel = (c.r / 2 + 4) * 2.0 ** -24 + 2.0 ** -22 + 3 * 2.0 ** -24
        row[lo : lo + n, : c.r] = x
        row_tol[lo : lo + n, : c.r] = (e * 1.01 + rel) * x.abs() + tiny
        for src, dst, tol in ((c.kv[lo : lo + n, None, c.r :], row[lo : lo + n, None, c.r :], row_tol[lo : lo + n, None, c.r :]),
                              (c.q[lo : lo + n, :, c.dn :], q[lo : lo + n], q_tol[lo : lo + n])):
            y = rotate(src, pos, rot, layout, inv, m)
            dst.copy_(y)
            tol.copy_(1.01 * e * y.abs() + 1.01 * rotate_tol(src, rot, layout, m) + tiny)
    return row, row_tol, q, q_tol


__all__ = ["DT", "F64", "Latent", "absorb", "append", "attention", "project", "rope_freqs", "rounded"]
