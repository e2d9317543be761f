"""The operators around a paged KV cache, as they are measured.

Four entry points that a serving loop calls before and between decode steps:

* ``paged_rope_append``: rotary positions of a ragged chunk of new tokens, and
  their keys and values written into the pages of the cache;
* ``paged_chunk_attention``: causal attention of those tokens over the cache;
* ``paged_attention_mass``: the attention weight every cached token received,
  accumulated per kv-head;
* ``paged_cache_evict``: a cache compacted to its sinks, its recent tokens and
  the heaviest of the others.

``run`` computes them with elementary torch operations, or, when ``own`` is
set, through the library.  Ragged batches: sequence b owns rows
q_start[b]..q_start[b+1] of the chunk, and its seq_lens[b] cached tokens count
the chunk's own.
"""

import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}
_NEG = float("-inf")


def _case(op, name=None, **kw):
    c = dict(op=op, batch=1, hq=32, hkv=8, d=128, page=16, kv="bf16", q="bf16", n_lo=1, n_hi=1, len_lo=1024,
             len_hi=1024)
    if op == "rope":
        c.update(layout="half", rot=128, base=10000.0, scaling="none", factor=1.0, orig=4096)
    if op == "mass":
        c.update(decay=1.0)
    if op == "evict":
        c.update(keep=256, sink=4, recent=64)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step's new token of 16 sequences, GQA 32/8: latency
        _case("rope", "rope-decode-b16", batch=16, n_lo=1, n_hi=1, len_lo=100, len_hi=2000),
        # a prompt of an MHA-32 model written into an empty fp16 cache, positions scaled past the trained length
        _case("rope", "rope-prompt-mha-8k", hkv=32, kv="f16", q="f16", n_lo=8192, n_hi=8192, len_lo=8192, len_hi=8192,
              scaling="yarn", factor=4.0, orig=2048),
        # ragged prompts into int8 pages of 64 tokens, half of the head rotated, neighbouring channels paired
        _case("rope", "rope-int8-ragged-b4", batch=4, page=64, kv="i8", q="f16", n_lo=300, n_hi=2000, len_lo=2000,
              len_hi=2100, layout="interleaved", rot=64, scaling="linear", factor=8.0),
        # the smallest chunk: 64 tokens of a GQA-4 model at d 64 over 1K
        _case("chunk", "chunk-tiny-1k", hq=4, hkv=1, d=64, kv="f16", q="f16", n_lo=64, n_hi=64, len_lo=1024,
              len_hi=1024),
        # a few drafted tokens of 8 sequences checked at once over 4K to 32K: bound by the cache's bytes
        _case("chunk", "chunk-draft-b8-4k-32k", batch=8, n_lo=1, n_hi=8, len_lo=4096, len_hi=32768),
        # one piece of a long prompt, MHA-32 at 32K: bound by the tensor cores
        _case("chunk", "chunk-prompt-mha-32k", hkv=32, kv="f16", q="f16", n_lo=2048, n_hi=2048, len_lo=32768,
              len_hi=32768),
        # a mixed batch of prompts and continuations, ragged, GQA 32/8
        _case("chunk", "chunk-ragged-b4-16k", batch=4, n_lo=7, n_hi=1000, len_lo=1000, len_hi=16384),
        # int8 cache of 64-token pages at 10K, ragged pieces
        _case("chunk", "chunk-int8-b8-10k", batch=8, page=64, kv="i8", q="f16", n_lo=1, n_hi=512, len_lo=5000,
              len_hi=10240),
        # one decode step's weights of 16 sequences over an int8 cache: bound by the keys' bytes
        _case("mass", "mass-decode-int8-b16-10k", batch=16, page=64, kv="i8", q="f16", len_lo=9000, len_hi=10240),
        # the weights of a prompt piece over 32K
        _case("mass", "mass-prompt-32k", n_lo=2048, n_hi=2048, len_lo=32768, len_hi=32768, decay=0.5),
        # a short int8 cache to a quarter
        _case("evict", "evict-int8-b2-4k", batch=2, page=64, kv="i8", q="f16", len_lo=3500, len_hi=4096, keep=1024),
        # four long caches to a quarter
        _case("evict", "evict-b4-128k", batch=4, len_lo=131072, len_hi=131072, keep=32768, recent=1024),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "chunk", "mass", "evict"])
    kv = rng.choice(["f16", "bf16", "i8"])
    q = kv if kv != "i8" else rng.choice(["f16", "bf16"])
    d = rng.choice([64, 128])
    g = rng.choice([1, 2, 4, 8])
    hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64])
    kw = dict(hq=g * hkv, hkv=hkv, d=d, page=page, kv=kv, q=q)
    batch = _logint(rng, 1, 16)
    if op == "rope":
        hi = _logint(rng, 1, 4096)
        ln = hi + _logint(rng, 1, 2048) - 1
        return _case(op, batch=batch, n_lo=max(1, hi // rng.choice([1, 2, 5])), n_hi=hi, len_lo=ln, len_hi=ln + 37,
                     layout=rng.choice(["half", "interleaved"]), rot=rng.choice([d, d // 2]),
                     base=rng.choice([10000.0, 500000.0]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                     factor=rng.choice([2.0, 4.0, 8.0]), orig=rng.choice([2048, 4096]), **kw)
    if op == "evict":
        ln = _logint(rng, 64, 32768)
        keep = max(16, int(ln * rng.uniform(0.05, 0.9)))
        return _case(op, batch=batch, len_lo=max(1, ln - ln // 3), len_hi=ln, keep=keep,
                     sink=min(rng.choice([0, 1, 4]), keep // 4), recent=rng.randrange(0, keep // 2 + 1), **kw)
    # chunk and mass: rows x tokens of the padded logits bounded by the largest listed case's
    ln = _logint(rng, 64, 32768)
    hi = _logint(rng, 1, min(ln, 2048))
    while batch * g * hkv * hi * ln > 32 * 2048 * 32768:
        batch, hi = max(1, batch // 2), max(1, hi // 2)
    kw.update(batch=batch, n_lo=max(1, hi // rng.choice([1, 3, 10])), n_hi=hi, len_lo=max(hi, ln // rng.choice([1, 2, 4])),
              len_hi=ln)
    if op == "mass":
        kw["decay"] = rng.choice([0.0, 0.5, 1.0])
    return _case(op, **kw)


# ---- inputs ---------------------------------------------------------------------


def _ints(lo, hi, n, g):
    return [int(x) for x in torch.randint(lo, hi + 1, (n,), generator=g)]


def _sizes(case):
    """Lengths and new tokens of the case's sequences."""
    g = torch.Generator().manual_seed(case["batch"] + 7 * case["n_hi"] + 1009 * case["len_hi"])
    lens = _ints(case["len_lo"], case["len_hi"], case["batch"], g)
    return lens, [min(n, L) for n, L in zip(_ints(case["n_lo"], case["n_hi"], case["batch"], g), lens)]


def _quantised(x):
    """Codes and fp16 scales per token and head of x [..., d] (scale absmax / 127)."""
    s = (x.abs().amax(dim=-1) / 127.0).to(torch.float16)
    s = torch.where(s > 0, s, torch.ones_like(s))
    return torch.clamp(torch.round(x / s.to(torch.float32).unsqueeze(-1)), -127, 127).to(torch.int8), s


def _pool(case, pages, g):
    x = torch.randn((pages, case["hkv"], case["page"], case["d"]), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((case["hkv"], 1, case["d"]), generator=g, device="cuda"))
    if case["kv"] == "i8":
        return _quantised(x)
    return x.to(_DT[case["kv"]]), None


def prepare(case, seed):
    hg = torch.Generator().manual_seed(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, S, d, hq, hkv = case["batch"], case["page"], case["d"], case["hq"], case["hkv"]
    lens, new = _sizes(case)
    order = torch.randperm(B, generator=hg).tolist()  # the batch's sizes are the case's; their order is the seed's
    lens, new = [lens[b] for b in order], [new[b] for b in order]
    pages = [-(-L // S) for L in lens]
    mp = -(-case["len_hi"] // S)
    dst_pages = [-(-min(L, case["keep"]) // S) for L in lens] if case["op"] == "evict" else [0] * B
    n_phys = sum(pages) + sum(dst_pages)
    perm = torch.randperm(n_phys, generator=hg).to(torch.int32)
    pt = torch.full((B, mp), -1, dtype=torch.int32)
    dst = torch.full((B, mp), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        pt[b, : pages[b]] = perm[at : at + pages[b]]
        at += pages[b]
        dst[b, : dst_pages[b]] = perm[at : at + dst_pages[b]]
        at += dst_pages[b]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    T = starts[-1]
    dev = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    s = dict(case=dict(case), T=T, mp=mp, n_phys=n_phys, seq_lens=dev(lens), q_start=dev(starts), page_table=pt.cuda())
    qt = _DT[case["q"]]
    if case["op"] == "rope":
        # the projection's output: one row of q, k and v per token
        qkv = torch.randn((T, hq + 2 * hkv, d), generator=g, device="cuda").to(qt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq : hq + hkv], qkv[:, hq + hkv :]
        s["q_out"] = torch.zeros((T, hq, d), dtype=qt, device="cuda")
        kt = _DT[case["kv"]]
        s["k_pool"] = torch.zeros((n_phys, hkv, S, d), dtype=kt, device="cuda")
        s["v_pool"] = torch.zeros((n_phys, hkv, S, d), dtype=kt, device="cuda")
        i8 = case["kv"] == "i8"
        s["k_scale"] = torch.ones((n_phys, hkv, S), dtype=torch.float16, device="cuda") if i8 else None
        s["v_scale"] = torch.ones((n_phys, hkv, S), dtype=torch.float16, device="cuda") if i8 else None
    else:
        s["k_pool"], s["k_scale"] = _pool(case, n_phys, g)
        if case["op"] != "mass":
            s["v_pool"], s["v_scale"] = _pool(case, n_phys, g)
    if case["op"] in ("chunk", "mass"):
        s["q"] = torch.randn((T, hq, d), generator=g, device="cuda").to(qt)
        s["lse"] = torch.zeros((T, hq), dtype=torch.float32, device="cuda")
    if case["op"] == "chunk":
        s["out"] = torch.zeros((T, hq, d), dtype=qt, device="cuda")
    if case["op"] in ("mass", "evict"):
        # weights as they accumulate: few tokens hold most of them
        s["mass"] = torch.exp(2.0 * torch.randn((B, hkv, mp * S), generator=g, device="cuda"))
        s["mass_out"] = torch.zeros_like(s["mass"])
    if case["op"] == "mass":
        s["lse"] = _logsumexp(s)
    if case["op"] == "evict":
        s["dst"] = dst.cuda()
        s["kept"] = torch.full((B, hkv, case["keep"]), -1, dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if own:
        import query_aware_sparse_page_gb300 as spg

        s["p"] = spg.make_params(batch=B, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=S,
                                 num_phys_pages=n_phys, max_pages_per_seq=mp, kv_dtype=case["kv"], q_dtype=case["q"],
                                 selector="all")
        s["ws"] = torch.zeros(spg.spg_chunk_workspace_size(s["p"], T), dtype=torch.uint8, device="cuda")
        if case["op"] == "rope":
            s["rope"] = spg.make_rope(rot_dim=case["rot"], layout=case["layout"], base=case["base"],
                                      scaling=case["scaling"], factor=case["factor"], orig_len=case["orig"])
    return s


# ---- plain forms ------------------------------------------------------------------


def _values(pool, scale):
    """What a pool's entries stand for, in 32 bits."""
    x = pool.to(torch.float32)
    return x if scale is None else x * scale.to(torch.float32).unsqueeze(-1)


def _cache(s, pool, scale):
    """The pages of every sequence in order: [B][Hkv][MP * S][d], fp32."""
    c = s["case"]
    x = _values(pool, scale)[s["page_table"].clamp(min=0).long()]
    return x.transpose(1, 2).reshape(c["batch"], c["hkv"], s["mp"] * c["page"], c["d"])


def _rows(s):
    """Row index of every (sequence, new token), and (sequence, new token) of every row."""
    start = s["q_start"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(s["case"]["n_hi"], device="cuda")
    rows = (start[:-1, None] + i[None]).clamp(max=max(s["T"] - 1, 0))
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    return rows, n, b, t - start[b]


def _logits(s):
    """Masked logits [B][Hkv][n_hi * G][MP * S] of the padded batch, in 32 bits."""
    c = s["case"]
    B, hkv, g = c["batch"], c["hkv"], c["hq"] // c["hkv"]
    rows, n, _, _ = _rows(s)
    q = s["q"].to(torch.float32)[rows].view(B, c["n_hi"], hkv, g, c["d"])
    q = q.permute(0, 2, 1, 3, 4).reshape(B, hkv, c["n_hi"] * g, c["d"])
    z = torch.matmul(q, _cache(s, s["k_pool"], s["k_scale"]).transpose(2, 3))
    z *= 1.0 / math.sqrt(c["d"])
    i = torch.arange(c["n_hi"], device="cuda")
    pos = (s["seq_lens"].long() - n)[:, None] + i[None]
    pos = torch.where(i[None] < n[:, None], pos, -1).repeat_interleave(g, dim=1)
    seen = torch.arange(z.shape[-1], device="cuda")[None, None] <= pos[:, :, None]
    return z.masked_fill_(~seen[:, None], _NEG)


def _per_row(s, x):
    """[B][Hkv][n_hi * G][...] back to [T][Hq][...]."""
    c = s["case"]
    g = c["hq"] // c["hkv"]
    _, _, b, i = _rows(s)
    x = x.reshape(c["batch"], c["hkv"], c["n_hi"], g, -1)[b, :, i]
    return x.reshape(s["T"], c["hq"], -1)


def _logsumexp(s):
    z = _logits(s)
    m = z.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    lse = m + torch.log(torch.exp(z - m).sum(dim=-1, keepdim=True))
    return _per_row(s, lse)[..., 0].contiguous()


def _plain_chunk(s):
    z = _logits(s)
    m = z.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    z = torch.exp(z.sub_(m))
    l = z.sum(dim=-1, keepdim=True)
    o = torch.matmul(z, _cache(s, s["v_pool"], s["v_scale"])) / l
    return {"out": _per_row(s, o).to(_DT[s["case"]["q"]]), "lse": _per_row(s, m + torch.log(l))[..., 0]}


def _plain_mass(s):
    c = s["case"]
    B, hkv, g = c["batch"], c["hkv"], c["hq"] // c["hkv"]
    rows, n, _, _ = _rows(s)
    lse = s["lse"][rows].view(B, c["n_hi"], hkv, g).permute(0, 2, 1, 3).reshape(B, hkv, c["n_hi"] * g, 1)
    w = torch.exp(_logits(s).sub_(lse)).sum(dim=2)
    t = torch.arange(w.shape[-1], device="cuda")[None, None]
    L = s["seq_lens"].long()
    old = torch.where(t < (L - n)[:, None, None], s["mass"] * c["decay"], torch.zeros_like(w))
    return {"mass": torch.where(t < L[:, None, None], old + w, s["mass_out"])}


def _inv_freq(c, dtype=torch.float64):
    """Angle per position of every channel pair, and the factor on cos and sin."""
    r, base, f = c["rot"], c["base"], c["factor"]
    i = torch.arange(0, r, 2, dtype=dtype, device="cuda")
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


def _rotated(x, ang, m, c):
    """x [T][H][d] turned by ang [T][rot / 2], in 32 bits."""
    r = c["rot"]
    cos, sin = (torch.cos(ang) * m).float()[:, None], (torch.sin(ang) * m).float()[:, None]
    x = x.to(torch.float32)
    y, rest = x[..., :r], x[..., r:]
    if c["layout"] == "half":
        a, b = y[..., : r // 2], y[..., r // 2 :]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([y, rest], dim=-1)


def _plain_rope(s):
    c = s["case"]
    _, n, b, i = _rows(s)
    pos = (s["seq_lens"].long() - n)[b] + i
    inv, m = _inv_freq(c)
    ang = pos.to(torch.float64)[:, None] * inv[None]
    phys = s["page_table"][b, pos // c["page"]].long()
    slot = pos % c["page"]
    k, v = _rotated(s["k"], ang, m, c), s["v"].to(torch.float32)
    if c["kv"] == "i8":
        (k, ks), (v, vs) = _quantised(k), _quantised(v)
        s["k_scale"][phys, :, slot] = ks
        s["v_scale"][phys, :, slot] = vs
    s["k_pool"][phys, :, slot] = k.to(_DT[c["kv"]])
    s["v_pool"][phys, :, slot] = v.to(_DT[c["kv"]])
    s["q_out"] = _rotated(s["q"], ang, m, c).to(_DT[c["q"]])


def _plain_evict(s):
    c = s["case"]
    B, hkv, S, keep = c["batch"], c["hkv"], c["page"], c["keep"]
    N = s["mp"] * S
    t = torch.arange(N, device="cuda")[None, None]
    L = s["seq_lens"].long()[:, None, None]
    w = torch.where((t < c["sink"]) | (t >= L - c["recent"]), math.inf, s["mass"])
    w = torch.where(t < L, w, torch.full_like(w, -1.0))
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    j = torch.arange(keep, device="cuda")[None, None]
    order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]))
    new = L.clamp(max=keep)
    kept = torch.where(j < new, order, N + j).sort(dim=-1).values
    live = (j < new).expand(B, hkv, keep)
    kept = torch.where(live, kept, 0)
    bi, hi = torch.arange(B, device="cuda")[:, None, None], torch.arange(hkv, device="cuda")[None, :, None]
    src = s["page_table"][bi, kept // S].long().clamp(min=0), hi, kept % S
    # entries past a sequence's end rewrite their own slot of the last destination page
    dj = torch.minimum(j, new - 1)
    dst = s["dst"][bi, dj // S].long().clamp(min=0), hi, dj % S
    last = torch.gather(kept, 2, (new - 1).expand(B, hkv, 1))
    src_last = s["page_table"][bi, last // S].long().clamp(min=0), hi, last % S
    for name in ("k_pool", "v_pool", "k_scale", "v_scale"):
        x = s[name]
        if x is not None:
            lv = live if x.dim() == 3 else live[..., None]
            x[dst] = torch.where(lv, x[src], x[src_last])
    s["kept"] = torch.where(live, kept, -1).to(torch.int32)
    s["new_lens"] = new[:, 0, 0].to(torch.int32)
    m = torch.gather(s["mass"], 2, kept)
    out = s["mass_out"]
    w = min(keep, N)
    out[..., :w] = torch.where(live, m, torch.nn.functional.pad(out, (0, max(0, keep - N)))[..., :keep])[..., :w]


def _pools(s):
    """The cache as it stands; int8 entries as the 16-bit values they stand for."""
    if s["case"]["kv"] != "i8":
        return {"k": s["k_pool"], "v": s["v_pool"]}
    return {"k": s["k_pool"].to(torch.float16) * s["k_scale"][..., None],
            "v": s["v_pool"].to(torch.float16) * s["v_scale"][..., None]}


def run(s):
    c = s["case"]
    if own:
        return _own(s)
    if c["op"] == "chunk":
        return _plain_chunk(s)
    if c["op"] == "mass":
        return _plain_mass(s)
    if c["op"] == "rope":
        _plain_rope(s)
        return {"q": s["q_out"], **_pools(s)}
    _plain_evict(s)
    return {"kept": s["kept"], "new_lens": s["new_lens"], "mass": s["mass_out"], **_pools(s)}


def _own(s):
    import query_aware_sparse_page_gb300 as spg

    c = s["case"]
    if c["op"] == "chunk":
        spg.paged_chunk_attention(s["p"], s["q"], s["q_start"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                                  s["page_table"], s["seq_lens"], s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "mass":
        spg.paged_attention_mass(s["p"], s["q"], s["q_start"], s["k_pool"], s["k_scale"], s["page_table"],
                                 s["seq_lens"], s["lse"], s["mass"], s["mass_out"], c["decay"], s["ws"])
        return {"mass": s["mass_out"]}
    if c["op"] == "rope":
        spg.paged_rope_append(s["p"], s["rope"], s["q"], s["k"], s["v"], s["q_start"], s["page_table"], s["seq_lens"],
                              s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["q_out"], ws=s["ws"])
        return {"q": s["q_out"], **_pools(s)}
    spg.paged_cache_evict(s["p"], s["mass"], c["keep"], c["sink"], c["recent"], s["k_pool"], s["v_pool"], s["k_scale"],
                          s["v_scale"], s["page_table"], s["dst"], s["seq_lens"], s["kept"], s["new_lens"],
                          s["mass_out"], s["ws"])
    return {"kept": s["kept"], "new_lens": s["new_lens"], "mass": s["mass_out"], **_pools(s)}


# ---- work, and the definition in 64 bits ---------------------------------------------


def work(case):
    B, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    lens, new = _sizes(case)
    T, tokens = sum(new), sum(lens)
    elem, extra = (1, 2) if case["kv"] == "i8" else (2, 0)
    row = d * elem + extra  # one token of one kv-head, K or V
    if case["op"] == "rope":
        return {"bytes": T * (2 * hq * d * 2 + 2 * hkv * d * 2 + 2 * hkv * row), "flops": T * 3 * (hq + hkv) * case["rot"]}
    if case["op"] == "evict":
        kept = sum(min(L, case["keep"]) for L in lens)
        return {"bytes": hkv * (4 * tokens + kept * (4 * row + 8)) + 4 * B, "flops": 0}
    pairs = sum(n * (L - 0.5 * (n - 1)) for L, n in zip(lens, new))  # (new token, cached token) pairs seen
    if case["op"] == "mass":
        return {"bytes": T * hq * (2 * d + 4) + hkv * tokens * (row + 4 * (2 if case["decay"] else 1)), "flops": 2 * d * hq * pairs}
    return {"bytes": T * hq * (4 * d + 4) + 2 * hkv * tokens * row, "flops": 4 * d * hq * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    B, S, hkv, d = case["batch"], case["page"], case["hkv"], case["d"]
    g = case["hq"] // hkv
    lens, starts = s["seq_lens"].tolist(), s["q_start"].tolist()
    f64 = torch.float64

    def tokens(pool, scale, b, h):
        pages = s["page_table"][b, : -(-lens[b] // S)].long()
        x = pool[pages, h].to(f64)
        if scale is not None:
            x = x * scale[pages, h].to(f64)[..., None]
        return x.reshape(-1, d)[: lens[b]]

    if case["op"] in ("chunk", "mass"):
        out = torch.zeros((s["T"], case["hq"], d), dtype=f64, device="cuda")
        lse = torch.zeros((s["T"], case["hq"]), dtype=f64, device="cuda")
        mass = s["mass_out"].to(f64) if case["op"] == "mass" else None
        for b in range(B):
            L, lo, hi = lens[b], starts[b], starts[b + 1]
            n = hi - lo
            later = torch.arange(L, device="cuda")[None] > torch.arange(L - n, L, device="cuda")[:, None]
            for h in range(hkv):
                k = tokens(s["k_pool"], s["k_scale"], b, h)
                v = tokens(s["v_pool"], s["v_scale"], b, h) if mass is None else None
                if mass is not None:
                    keep = torch.arange(L, device="cuda") < L - n
                    old = s["mass"][b, h, :L].to(f64) * case["decay"]
                    mass[b, h, :L] = torch.where(keep, old, torch.zeros_like(old))
                for j in range(g):
                    z = (s["q"][lo:hi, h * g + j].to(f64) @ k.T) / math.sqrt(d)
                    z = z.masked_fill(later, _NEG)
                    if mass is not None:
                        mass[b, h, :L] += torch.exp(z - s["lse"][lo:hi, h * g + j].to(f64)[:, None]).sum(dim=0)
                        continue
                    e = torch.logsumexp(z, dim=1)
                    lse[lo:hi, h * g + j] = e
                    out[lo:hi, h * g + j] = torch.exp(z - e[:, None]) @ v
        return {"mass": mass} if mass is not None else {"out": out, "lse": lse}
    if case["op"] == "rope":
        inv, m = _inv_freq(case)
        q = torch.zeros((s["T"], case["hq"], d), dtype=f64, device="cuda")
        kp, vp = s["k_pool"].to(f64), s["v_pool"].to(f64)
        r, half = case["rot"], case["layout"] == "half"
        one = torch.arange(r // 2, device="cuda") if half else torch.arange(0, r, 2, device="cuda")
        two = one + (r // 2 if half else 1)
        for b in range(B):
            lo, hi = starts[b], starts[b + 1]
            pos = torch.arange(lens[b] - (hi - lo), lens[b], device="cuda")
            turn = torch.polar(torch.full((), m, dtype=f64, device="cuda"), pos[:, None].to(f64) * inv)[:, None]

            def rot(x):
                y = x.to(f64).clone()
                z = torch.complex(y[..., one], y[..., two]) * turn
                y[..., one], y[..., two] = z.real, z.imag
                return y

            q[lo:hi] = rot(s["q"][lo:hi])
            ph = s["page_table"][b, pos // S].long()
            kp[ph, :, pos % S] = rot(s["k"][lo:hi])
            vp[ph, :, pos % S] = s["v"][lo:hi].to(f64)
        if case["kv"] == "i8":  # a code next to a border has no value of its own
            kp = vp = None
        return {"q": q, "k": kp, "v": vp}
    # evict: every value is moved, none computed
    return None
