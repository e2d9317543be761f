"""Plain 64-bit forms of the paged-chunk operators, and seeded inputs for
their tests.  Everything runs on the CPU in float64 from the definitions."""

from __future__ import annotations

import math
from dataclasses import dataclass

import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}
F64 = torch.float64


@dataclass
class Chunk:
    """A ragged chunk over a paged cache; tensors live on the CPU."""

    hq: int
    hkv: int
    d: int
    S: int
    kv: str
    qdt: str
    lens: list
    new: list
    pad_rows: int = 0
    extra_pages: int = 0
    mp: int = 0
    seed: int = 0
    poison: float = float("nan")

    def __post_init__(self):
        g = torch.Generator().manual_seed(self.seed + 17)
        B, S = len(self.lens), self.S
        pages = [-(-L // S) for L in self.lens]
        self.mp = max(self.mp, max(pages + [1]))
        self.n_phys = sum(pages) + self.extra_pages + 1
        perm = torch.randperm(self.n_phys, generator=g)
        self.page_table = torch.full((B, self.mp), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.page_table[b, : pages[b]] = perm[at : at + pages[b]].int()
            at += pages[b]
        self.free = perm[at:].int()
        starts = [0]
        for n in self.new:
            starts.append(starts[-1] + n)
        self.starts = starts
        self.T = starts[-1] + self.pad_rows
        self.q_start = torch.tensor(starts, dtype=torch.int32)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32)
        qt = DT[self.qdt]
        self.q = torch.randn((self.T, self.hq, self.d), generator=g).to(qt)
        self.k = torch.randn((self.T, self.hkv, self.d), generator=g).to(qt)
        self.v = torch.randn((self.T, self.hkv, self.d), generator=g).to(qt)
        shape = (self.n_phys, self.hkv, S, self.d)
        self.k_scale = self.v_scale = None
        if self.kv == "i8":
            self.k_pool = torch.randint(-127, 128, shape, generator=g).to(torch.int8)
            self.v_pool = torch.randint(-127, 128, shape, generator=g).to(torch.int8)
            self.k_scale = (0.005 + 0.02 * torch.rand(shape[:3], generator=g)).half()
            self.v_scale = (0.005 + 0.02 * torch.rand(shape[:3], generator=g)).half()
        else:
            self.k_pool = torch.randn(shape, generator=g).to(qt)
            self.v_pool = torch.randn(shape, generator=g).to(qt)
        # slots that hold no token: whatever the pool holds must not matter
        live = torch.zeros((self.n_phys, S), dtype=torch.bool)
        for b, L in enumerate(self.lens):
            for t0 in range(0, L, S):
                live[int(self.page_table[b, t0 // S]), : min(S, L - t0)] = True
        dead = ~live[:, None].expand(self.n_phys, self.hkv, S)
        if self.kv == "i8":
            for codes, scale in ((self.k_pool, self.k_scale), (self.v_pool, self.v_scale)):
                codes[dead] = 127
                scale[dead] = self.poison
        else:
            self.k_pool[dead] = self.poison
            self.v_pool[dead] = self.poison

    @property
    def group(self):
        return self.hq // self.hkv

    def params(self, spg, **kw):
        a = dict(batch=len(self.lens), num_q_heads=self.hq, num_kv_heads=self.hkv, head_dim=self.d, page_size=self.S,
                 num_phys_pages=self.n_phys, max_pages_per_seq=self.mp, kv_dtype=self.kv, q_dtype=self.qdt,
                 selector="all")
        a.update(kw)
        return spg.make_params(**a)

    def tokens(self, pool, scale, b, h):
        """The cached rows of (b, h) in order, [L][d] float64."""
        L = self.lens[b]
        pg = self.page_table[b, : -(-L // self.S)].long()
        x = pool[pg, h].to(F64)
        if scale is not None:
            x = x * scale[pg, h].to(F64)[..., None]
        return x.reshape(-1, self.d)[:L]

    def logits(self, b, h, j):
        """[n][L] scaled logits of query head h * G + j, -inf above the diagonal, and sum |q k| scale of each."""
        lo, hi, L, n = self.starts[b], self.starts[b + 1], self.lens[b], self.new[b]
        q = self.q[lo:hi, h * self.group + j].to(F64)
        k = self.tokens(self.k_pool, self.k_scale, b, h)
        z = q @ k.T / math.sqrt(self.d)
        size = q.abs() @ k.abs().T / math.sqrt(self.d)
        hidden = torch.arange(L)[None] > torch.arange(L - n, L)[:, None]
        return z.masked_fill(hidden, -math.inf), size


def attention(c: Chunk, drop=()):
    """out, lse and how far a 16-bit result may be from them: see TOLERANCES.

    drop: (b, page) pairs whose tokens take no part.

    TOLERANCES.  With e = eps / 2 of the output's type, p the normalised
    probabilities and A = sum p |v|: rounding p costs e * A, rounding the
    output e * |out|.  A logit is a sum of d products in 32 bits, off by at
    most d * 2^-24 * sum |q k| scale, and the exponent's argument adds a few
    2^-24 * |z|; a relative error dz of every p moves out by at most 2 dz A.
    fp16 holds unnormalised p below 2^-14 with an absolute step of 2^-24:
    half of it times sum |v| over exp(lse - max) >= 1 (int8: of the codes,
    whose factor carries 2^4 more)."""
    out = torch.zeros((c.T, c.hq, c.d), dtype=F64)
    tol = torch.zeros_like(out)
    lse = torch.full((c.T, c.hq), -math.inf, dtype=F64)
    lse_tol = torch.zeros_like(lse)
    e = torch.finfo(DT[c.qdt]).eps / 2
    for b in range(len(c.lens)):
        lo, hi = c.starts[b], c.starts[b + 1]
        if lo == hi:
            continue
        gone = torch.zeros(c.lens[b], dtype=torch.bool)
        for bb, pg in drop:
            if bb == b:
                gone[pg * c.S : (pg + 1) * c.S] = True
        for h in range(c.hkv):
            v = c.tokens(c.v_pool, c.v_scale, b, h)
            v = v.masked_fill(gone[:, None], 0.0)
            code = v if c.kv != "i8" else c.tokens(c.v_pool, None, b, h)
            for j in range(c.group):
                z, size = c.logits(b, h, j)
                z = z.masked_fill(gone[None], -math.inf)
                i = h * c.group + j
                ls = torch.logsumexp(z, dim=1)
                p = torch.exp(z - torch.where(torch.isfinite(ls), ls, 0.0)[:, None])
                p = torch.where(torch.isfinite(z), p, torch.zeros_like(p))
                o = p @ v
                A = p @ v.abs()
                zmax = z.masked_fill(~torch.isfinite(z), 0.0).abs().amax(dim=1)
                dz = c.d * 2.0 ** -24 * size.amax(dim=1) + 8 * 2.0 ** -24 * (zmax + 1)
                t = e * (A + o.abs()) + 2 * dz[:, None] * A
                if c.qdt == "f16":
                    step = 2.0 ** -25 / (16 if c.kv == "i8" else 1)
                    t = t + step * code.abs().sum(dim=0)[None] + 2.0 ** -25
                out[lo:hi, i], tol[lo:hi, i], lse[lo:hi, i] = o, 1.01 * t, ls
                lse_tol[lo:hi, i] = dz + 8 * 2.0 ** -24 * (1 + torch.where(torch.isfinite(ls), ls.abs(), 0.0))
    return out, tol, lse, lse_tol


def mass_of(c: Chunk, lse, mass_in, decay):
    """Accumulated mass [B][Hkv][MP * S] (NaN past each length), and its tolerance: every term's exponent is off
    by dz as in attention() plus the rounding of lse, and terms are added in 32 bits."""
    out = torch.full((len(c.lens), c.hkv, c.mp * c.S), math.nan, dtype=F64)
    tol = torch.zeros_like(out)
    for b, L in enumerate(c.lens):
        n, lo = c.new[b], c.starts[b]
        for h in range(c.hkv):
            w, t = torch.zeros(L, dtype=F64), torch.zeros(L, dtype=F64)
            for j in range(c.group):
                if n == 0:
                    continue
                z, size = c.logits(b, h, j)
                ls = lse[lo : lo + n, h * c.group + j].to(F64)
                e = torch.where(torch.isfinite(ls)[:, None], torch.exp(z - ls[:, None]), torch.zeros_like(z))
                dz = c.d * 2.0 ** -24 * size + 8 * 2.0 ** -24 * (z.masked_fill(~torch.isfinite(z), 0.0).abs() + ls.masked_fill(~torch.isfinite(ls), 0.0).abs()[:, None] + 1)
                w, t = w + e.sum(dim=0), t + (2 * dz * e).sum(dim=0)
            old = torch.zeros(L, dtype=F64)
            if mass_in is not None and decay > 0:
                old[: L - n] = mass_in[b, h, : L - n].to(F64) * decay
            out[b, h, :L] = old + w
            tol[b, h, :L] = t + (n * c.group + 4) * 2.0 ** -24 * (old.abs() + w)
    return out, tol


def rope_freqs(rot, base, scaling, factor, orig):
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "ntk":
        b2 = base * factor ** (rot / (rot - 2))
        return [b2 ** (-2.0 * i / rot) for i in range(rot // 2)], 1.0
    if scaling == "yarn":
        idx = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(idx(32.0)), 0), min(math.ceil(idx(1.0)), rot - 1)
        r = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(rot // 2)]
        return [x / factor * w + x * (1 - w) for x, w in zip(f, r)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rotate(x, pos, rot, layout, inv, m):
    """x [n][H][d] (any float type) at integer positions [n], float64."""
    y = x.to(F64).clone()
    ang = pos.to(F64)[:, None] * torch.tensor(inv, dtype=F64)[None]
    c, s = (torch.cos(ang) * m)[:, None], (torch.sin(ang) * m)[:, None]
    one = slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)
    two = slice(rot // 2, rot) if layout == "half" else slice(1, rot, 2)
    a, b = y[..., one].clone(), y[..., two].clone()
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    return y


def rotate_tol(x, rot, layout, m):
    """Rounding angle (pi 2^-25 in 32 bits, 2 pi 2^-33 of the fixed-point turn, 2^-22 of sincos) times both channels of the pair,
    and two 32-bit products and a sum."""
    y = x.to(F64).abs().clone()
    one = slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)
    two = slice(rot // 2, rot) if layout == "half" else slice(1, rot, 2)
    s = y[..., one] + y[..., two]
    t = torch.zeros_like(y)
    t[..., one] = t[..., two] = s * m * (math.pi * 2.0 ** -25 + 2 * math.pi * 2.0 ** -33 + 2.0 ** -22 + 4 * 2.0 ** -24)
    return t


def kept_positions(mass, L, keep, n_sink, n_recent):
    """Positions kept of one (batch, kv-head), by a full sort."""
    if L <= keep:
        return list(range(L))
    forced = set(range(min(n_sink, L))) | set(range(max(0, L - n_recent), L))
    rest = [t for t in range(L) if t not in forced]
    key = lambda t: (math.inf if math.isnan(mass[t]) else -mass[t], math.isnan(mass[t]), t)  # noqa: E731
    return sorted(forced | set(sorted(rest, key=key)[: keep - len(forced)]))
