"""Attention over a paged cache of latent vectors, as it is measured.

One vector per token (latent_dim channels, from which every head's keys and
values come by that head's own matrices) and one rotary key shared by all heads
are all the cache holds.  Four entry points that a serving loop calls per layer:

* ``paged_latent_append``: the latent vectors of a ragged chunk of new tokens,
  normalised, and their rotated keys into the pages; the rotated part of the
  queries beside the absorbed one;
* ``latent_absorb``: each head's key matrix taken over to its queries, which
  then meet the latent vectors themselves;
* ``paged_latent_attention``: causal attention of those queries over the
  cache, its result one latent vector per head;
* ``latent_project``: each head's value matrix applied to that result.

``run`` computes them with elementary torch operations, or, when ``own`` is
set, through the library.  Ragged batches: sequence b owns rows
q_start[b]..q_start[b+1] of the chunk, and its seq_lens[b] cached tokens count
the chunk's own.
"""

import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}
_NEG = float("-inf")
_EPS = 1e-6


def _case(op, name=None, **kw):
    c = dict(op=op, batch=1, heads=32, latent=512, rope=64, nope=128, vdim=128, page=64, dtype="bf16", n_lo=1, n_hi=1,
             len_lo=1024, len_hi=1024)
    if op == "append":
        c.update(norm=True, layout="interleaved", base=10000.0, scaling="none", factor=1.0, orig=4096)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step's new token of 16 sequences: latency
        _case("append", "append-decode-b16", batch=16, heads=16, len_lo=100, len_hi=2000),
        # a prompt written into an empty fp16 cache of small pages, positions scaled past the trained length
        _case("append", "append-prompt-8k", page=16, dtype="f16", n_lo=8192, n_hi=8192, len_lo=8192, len_hi=8192,
              layout="half", scaling="yarn", factor=4.0, orig=2048),
        # the queries of one decode step of 16 sequences, 128 heads: bound by the matrices' bytes
        _case("absorb", "absorb-decode-b16-h128", batch=16, heads=128),
        # the queries of a prompt piece
        _case("absorb", "absorb-piece-2k", dtype="f16", n_lo=2048, n_hi=2048, len_lo=2048, len_hi=2048),
        # the values of one decode step of 16 sequences, 128 heads
        _case("project", "project-decode-b16-h128", batch=16, heads=128),
        # the values of ragged drafts, heads of 64 channels, a small latent vector
        _case("project", "project-drafts-b13", batch=13, heads=20, latent=256, vdim=64, dtype="f16", n_lo=1, n_hi=9),
        # the smallest attention: one token of 4 heads over 1K, a latent vector of 256
        _case("attend", "attend-tiny-1k", heads=4, latent=256, page=16, dtype="f16"),
        # one sequence decoding at 32K: split over the cache's length
        _case("attend", "attend-decode-b1-32k", len_lo=32768, len_hi=32768),
        # one decode step of 8 sequences of 4K to 64K: bound by the cache's bytes
        _case("attend", "attend-decode-b8-4k-64k", batch=8, page=16, len_lo=4096, len_hi=65536),
        # one decode step of 16 sequences at 10K with 128 heads: as many products as bytes
        _case("attend", "attend-decode-b16-h128-10k", batch=16, heads=128, len_lo=9000, len_hi=10240),
        # a few drafted tokens of 8 sequences checked at once over 4K to 32K, 16 heads
        _case("attend", "attend-draft-b8-4k-32k", batch=8, heads=16, page=32, dtype="f16", n_lo=1, n_hi=8, len_lo=4096,
              len_hi=32768),
        # the last piece of a prompt over what the cache holds of it: bound by the tensor cores
        _case("attend", "attend-piece-500-16k", heads=16, n_lo=500, n_hi=500, len_lo=16384, len_hi=16384),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "absorb", "project", "attend"])
    kw = dict(heads=rng.choice([1, 3, 4, 8, 16, 20, 32, 48, 64, 128]), latent=rng.choice([256, 512]),
              nope=rng.choice([64, 128]), vdim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
              dtype=rng.choice(["f16", "bf16"]))
    if op == "append":
        hi = _logint(rng, 1, 4096)
        ln = hi + _logint(rng, 1, 2048) - 1
        return _case(op, batch=_logint(rng, 1, 16), n_lo=max(1, hi // rng.choice([1, 2, 5])), n_hi=hi, len_lo=ln,
                     len_hi=ln + 37, norm=rng.choice([True, True, False]), layout=rng.choice(["half", "interleaved"]),
                     base=rng.choice([10000.0, 500000.0]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                     factor=rng.choice([2.0, 4.0, 8.0]), orig=rng.choice([2048, 4096]), **kw)
    if op in ("absorb", "project"):
        n = _logint(rng, 1, 2048)
        if kw["heads"] > 32:
            n = min(n, 500)
        return _case(op, n_lo=n, n_hi=n, len_lo=n, len_hi=n, **kw)
    # attention: rows x tokens bounded by the largest listed case's
    batch, ln = _logint(rng, 1, 16), _logint(rng, 1, 65536)
    hi = min(ln, rng.choice([1, 1, _logint(rng, 1, 500)]))
    while batch * kw["heads"] * hi * ln > 16 * 500 * 16384:
        if hi > 1:
            hi //= 2
        else:
            batch = max(1, batch // 2)
    while batch * ln > 8 * 65536:
        batch //= 2
    return _case(op, batch=batch, n_lo=max(1, hi // rng.choice([1, 3, 10])), n_hi=hi,
                 len_lo=max(hi, ln // rng.choice([1, 2, 4])), len_hi=ln, **kw)


# ---- inputs ---------------------------------------------------------------------


def _ints(lo, hi, n, g):
    return [int(x) for x in torch.randint(lo, hi + 1, (n,), generator=g)]


def _sizes(case):
    """Lengths and new tokens of the case's sequences."""
    g = torch.Generator().manual_seed(case["batch"] + 7 * case["n_hi"] + 1009 * case["len_hi"])
    lens = _ints(case["len_lo"], case["len_hi"], case["batch"], g)
    return lens, [min(n, L) for n, L in zip(_ints(case["n_lo"], case["n_hi"], case["batch"], g), lens)]


def prepare(case, seed):
    hg = torch.Generator().manual_seed(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B, S, H, r, dr = case["op"], case["batch"], case["page"], case["heads"], case["latent"], case["rope"]
    dt = _DT[case["dtype"]]
    lens, new = _sizes(case)
    order = torch.randperm(B, generator=hg).tolist()  # the batch's sizes are the case's; their order is the seed's
    lens, new = [lens[b] for b in order], [new[b] for b in order]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    T = starts[-1]
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case=dict(case), T=T)
    n_phys = mp = 1
    if op in ("append", "attend"):
        pages = [-(-L // S) for L in lens]
        mp, n_phys = -(-case["len_hi"] // S), sum(pages)
        perm = torch.randperm(n_phys, generator=hg).to(torch.int32)
        pt = torch.full((B, mp), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            pt[b, : pages[b]] = perm[at : at + pages[b]]
            at += pages[b]
        dev = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
        s.update(mp=mp, seq_lens=dev(lens), q_start=dev(starts), page_table=pt.cuda())
    if op == "append":
        # the down-projection's output: a latent vector and a rotary key per token
        kv = rand(T, r + dr).to(dt)
        s["c"], s["k_pe"] = kv[:, :r], kv[:, r:]
        s["norm"] = (1.0 + 0.1 * rand(r)).to(dt) if case["norm"] else None
        s["pool"] = torch.zeros((n_phys, S, r + dr), dtype=dt, device="cuda")
    if op in ("append", "absorb"):
        s["q"] = rand(T, H, case["nope"] + dr).to(dt)
        s["q_lat"] = torch.zeros((T, H, r + dr), dtype=dt, device="cuda")
    if op in ("absorb", "project"):
        s["w_kv"] = (rand(H, case["nope"] + case["vdim"], r) / math.sqrt(r)).to(dt)
    if op == "attend":
        s["q_lat"] = rand(T, H, r + dr).to(dt)
        s["pool"] = rand(n_phys, S, r + dr).to(dt)
        s["lse"] = torch.zeros((T, H), dtype=torch.float32, device="cuda")
    if op == "project":
        s["o_lat"] = (0.1 * rand(T, H, r)).to(dt)
        s["out"] = torch.zeros((T, H, case["vdim"]), dtype=dt, device="cuda")
    if op == "attend":
        s["o_lat"] = torch.zeros((T, H, r), dtype=dt, device="cuda")
    if own:
        import query_aware_sparse_page_gb300 as spg

        s["p"] = spg.make_latent_params(batch=B, num_heads=H, latent_dim=r, rope_dim=dr, nope_dim=case["nope"],
                                        v_dim=case["vdim"], page_size=S, num_phys_pages=n_phys, max_pages_per_seq=mp,
                                        dtype=case["dtype"])
        if op in ("append", "attend"):
            s["ws"] = torch.zeros(spg.spg_latent_workspace_size(s["p"], T), dtype=torch.uint8, device="cuda")
        if op == "append":
            s["rope"] = spg.make_rope(rot_dim=dr, layout=case["layout"], base=case["base"], scaling=case["scaling"],
                                      factor=case["factor"], orig_len=case["orig"])
    return s


# ---- plain forms ------------------------------------------------------------------


def _rows(s):
    """Row index of every (sequence, new token), and (sequence, new token) of every row."""
    start = s["q_start"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(s["case"]["n_hi"], device="cuda")
    rows = (start[:-1, None] + i[None]).clamp(max=max(s["T"] - 1, 0))
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    return rows, n, b, t - start[b]


def _inv_freq(c):
    """Angle per position of every channel pair, and the factor on cos and sin."""
    r, base, f = c["rope"], c["base"], c["factor"]
    i = torch.arange(0, r, 2, dtype=torch.float64, device="cuda")
    if c["scaling"] == "ntk":
        base = base * f ** (r / (r - 2))
    inv = base ** (-i / r)
    if c["scaling"] == "linear":
        return inv / f, 1.0
    if c["scaling"] == "yarn":
        # by parts: pairs that turn more than 32 times over the trained length stay, less than once are divided
        at = lambda turns: r * math.log(c["orig"] / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r - 1)
        ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1.0
    return inv, 1.0


def _rotated(x, ang, m, layout):
    """x [..., rope] turned by ang [..., rope / 2], in 32 bits."""
    cos, sin = (torch.cos(ang) * m).float(), (torch.sin(ang) * m).float()
    x = x.to(torch.float32)
    if layout == "half":
        a, b = x.chunk(2, dim=-1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)


def _plain_append(s):
    c = s["case"]
    r, dt = c["latent"], _DT[c["dtype"]]
    _, n, b, i = _rows(s)
    pos = (s["seq_lens"].long() - n)[b] + i
    inv, m = _inv_freq(c)
    ang = pos.to(torch.float64)[:, None] * inv[None]
    x = s["c"].to(torch.float32)
    if s["norm"] is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + _EPS) * s["norm"].to(torch.float32)
    row = torch.cat([x, _rotated(s["k_pe"], ang, m, c["layout"])], dim=-1).to(dt)
    s["pool"][s["page_table"][b, pos // c["page"]].long(), pos % c["page"]] = row
    s["q_lat"][..., r:] = _rotated(s["q"][..., c["nope"]:], ang[:, None], m, c["layout"]).to(dt)


def _plain_attend(s):
    c = s["case"]
    B, H, n_hi, r = c["batch"], c["heads"], c["n_hi"], c["latent"]
    rows, n, b, i = _rows(s)
    kv = s["pool"][s["page_table"].clamp(min=0).long()].to(torch.float32).view(B, s["mp"] * c["page"], -1)
    q = s["q_lat"][rows].to(torch.float32).view(B, n_hi * H, -1)
    z = torch.matmul(q, kv.transpose(1, 2))
    z *= 1.0 / math.sqrt(c["nope"] + c["rope"])
    pos = (s["seq_lens"].long() - n)[:, None] + torch.arange(n_hi, device="cuda")[None]
    pos = torch.where(torch.arange(n_hi, device="cuda")[None] < n[:, None], pos, -1).repeat_interleave(H, dim=1)
    z = z.masked_fill_(torch.arange(z.shape[-1], device="cuda")[None, None] > pos[:, :, None], _NEG)
    m = z.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    z = torch.exp(z.sub_(m))
    l = z.sum(dim=-1, keepdim=True)
    o = torch.matmul(z, kv[..., :r]) / l
    o, lse = o.view(B, n_hi, H, r)[b, i], (m + torch.log(l)).view(B, n_hi, H)[b, i]
    return {"o_lat": o.to(_DT[c["dtype"]]), "lse": lse}


def run(s):
    c = s["case"]
    if own:
        return _own(s)
    dt, dn, r = _DT[c["dtype"]], c["nope"], c["latent"]
    if c["op"] == "attend":
        return _plain_attend(s)
    if c["op"] == "append":
        _plain_append(s)
        return {"q_lat": s["q_lat"], "pool": s["pool"]}
    w = s["w_kv"].to(torch.float32)
    if c["op"] == "absorb":
        x = s["q"][..., :dn].to(torch.float32).transpose(0, 1)
        s["q_lat"][..., :r] = torch.matmul(x, w[:, :dn]).transpose(0, 1).to(dt)
        return {"q_lat": s["q_lat"]}
    x = s["o_lat"].to(torch.float32).transpose(0, 1)
    return {"out": torch.matmul(x, w[:, dn:].transpose(1, 2)).transpose(0, 1).to(dt)}


def _own(s):
    import query_aware_sparse_page_gb300 as spg

    c = s["case"]
    if c["op"] == "attend":
        spg.paged_latent_attention(s["p"], s["q_lat"], s["q_start"], s["pool"], s["page_table"], s["seq_lens"],
                                   s["o_lat"], s["lse"], s["ws"])
        return {"o_lat": s["o_lat"], "lse": s["lse"]}
    if c["op"] == "append":
        spg.paged_latent_append(s["p"], s["rope"], s["c"], s["k_pe"], s["norm"], _EPS, s["q"], s["q_start"],
                                s["page_table"], s["seq_lens"], s["pool"], s["q_lat"], ws=s["ws"])
        return {"q_lat": s["q_lat"], "pool": s["pool"]}
    if c["op"] == "absorb":
        spg.latent_absorb(s["p"], s["q"], s["w_kv"], s["q_lat"])
        return {"q_lat": s["q_lat"]}
    spg.latent_project(s["p"], s["o_lat"], s["w_kv"], s["out"])
    return {"out": s["out"]}


# ---- work, and the definition in 64 bits ---------------------------------------------


def work(case):
    H, r, dr, dn, dv = (case[k] for k in ("heads", "latent", "rope", "nope", "vdim"))
    lens, new = _sizes(case)
    T = sum(new)
    if case["op"] == "append":
        return {"bytes": 2 * (2 * T * (r + dr) + 2 * T * H * dr + (r if case["norm"] else 0)),
                "flops": T * (4 * r + 3 * (H + 1) * dr)}
    if case["op"] == "absorb":
        return {"bytes": 2 * H * (T * dn + dn * r + T * r), "flops": 2 * T * H * dn * r}
    if case["op"] == "project":
        return {"bytes": 2 * H * (T * r + dv * r + T * dv), "flops": 2 * T * H * dv * r}
    pairs = sum(n * (L - 0.5 * (n - 1)) for L, n in zip(lens, new))  # (new token, cached token) pairs seen
    return {"bytes": 2 * sum(lens) * (r + dr) + T * H * (2 * (2 * r + dr) + 4), "flops": 2 * H * pairs * (2 * r + dr)}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    S, H, r, dr, dn = (case[k] for k in ("page", "heads", "latent", "rope", "nope"))
    if case["op"] == "absorb":
        out = s["q_lat"].to(f64)
        out[..., :r] = torch.einsum("thd,hdc->thc", s["q"][..., :dn].to(f64), s["w_kv"][:, :dn].to(f64))
        return {"q_lat": out}
    if case["op"] == "project":
        return {"out": torch.einsum("thc,hvc->thv", s["o_lat"].to(f64), s["w_kv"][:, dn:].to(f64))}
    lens, starts = s["seq_lens"].tolist(), s["q_start"].tolist()
    if case["op"] == "attend":
        out = torch.zeros((s["T"], H, r), dtype=f64, device="cuda")
        lse = torch.zeros((s["T"], H), dtype=f64, device="cuda")
        for b, L in enumerate(lens):
            lo, hi = starts[b], starts[b + 1]
            kv = s["pool"][s["page_table"][b, : -(-L // S)].long()].reshape(-1, r + dr)[:L].to(f64)
            for t in range(lo, hi):
                seen = L - (hi - 1 - t)
                z = s["q_lat"][t].to(f64) @ kv[:seen].T / math.sqrt(dn + dr)
                lse[t] = torch.logsumexp(z, dim=1)
                out[t] = torch.exp(z - lse[t][:, None]) @ kv[:seen, :r]
        return {"o_lat": out, "lse": lse}
    inv, m = _inv_freq(case)
    q, pool = s["q_lat"].to(f64), s["pool"].to(f64)
    half = case["layout"] == "half"
    one = torch.arange(dr // 2, device="cuda") if half else torch.arange(0, dr, 2, device="cuda")
    two = one + (dr // 2 if half else 1)
    for b, L in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        pos = torch.arange(L - (hi - lo), L, device="cuda")
        turn = torch.polar(torch.full((), m, dtype=f64, device="cuda"), pos[:, None].to(f64) * inv)

        def rot(x, t):
            y = x.to(f64).clone()
            z = torch.complex(y[..., one], y[..., two]) * t
            y[..., one], y[..., two] = z.real, z.imag
            return y

        x = s["c"][lo:hi].to(f64)
        if s["norm"] is not None:
            x = x / torch.sqrt(x.square().mean(dim=1, keepdim=True) + _EPS) * s["norm"].to(f64)
        pages = s["page_table"][b, pos // S].long()
        pool[pages, pos % S] = torch.cat([x, rot(s["k_pe"][lo:hi], turn)], dim=1)
        q[lo:hi, :, r:] = rot(s["q"][lo:hi, :, dn:], turn[:, None])
    return {"q_lat": q, "pool": pool}
