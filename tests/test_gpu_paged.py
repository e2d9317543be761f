"""The paged-chunk operators on the GPU against their 64-bit forms (tests/paged_ref.py, where the tolerances are
derived): ragged chunks, empty sequences, padded batches, values past the lengths, bad pages, streams and graphs,
and the operators one after the other as a serving loop runs them."""

import math

import pytest
import torch

import paged_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spg():
    import query_aware_sparse_page_gb300 as m

    return m


def dev(t):
    return None if t is None else t.cuda()


def host(t):
    return t.detach().cpu()


class Run:
    """A chunk's tensors on the GPU, with its parameters and workspace."""

    def __init__(self, spg, c, **kw):
        self.spg, self.c = spg, c
        self.p = c.params(spg, **kw)
        assert spg.spg_validate(self.p) == 0
        self.ws = torch.zeros(spg.spg_chunk_workspace_size(self.p, c.T), dtype=torch.uint8, device="cuda")
        for n in ("q", "k", "v", "k_pool", "v_pool", "k_scale", "v_scale", "page_table", "seq_lens", "q_start"):
            setattr(self, n, dev(getattr(c, n)))
        self.out = torch.full((c.T, c.hq, c.d), 7.0, dtype=R.DT[c.qdt], device="cuda")
        self.lse = torch.full((c.T, c.hq), 7.0, device="cuda")

    def chunk(self, **kw):
        self.spg.paged_chunk_attention(self.p, self.q, self.q_start, self.k_pool, self.v_pool, self.k_scale,
                                       self.v_scale, self.page_table, self.seq_lens, self.out, self.lse, self.ws, **kw)

    def mass(self, lse, mass_in, mass_out, decay):
        self.spg.paged_attention_mass(self.p, self.q, self.q_start, self.k_pool, self.k_scale, self.page_table,
                                      self.seq_lens, lse, mass_in, mass_out, decay, self.ws)

    def append(self, rope, q_out, positions=None):
        self.spg.paged_rope_append(self.p, rope, self.q, self.k, self.v, self.q_start, self.page_table, self.seq_lens,
                                   self.k_pool, self.v_pool, self.k_scale, self.v_scale, q_out, positions, self.ws)

    def err(self):
        return self.spg.spg_read_device_error(self.ws)


def close(got, want, tol, what):
    d = (host(got).to(R.F64) - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {d[bad].max():.3e} (allowed {tol[bad].min():.3e})"


def check_chunk(r, drop=()):
    c = r.c
    out, tol, lse, lse_tol = R.attention(c, drop)
    n = c.starts[-1]
    fin = torch.isfinite(lse[:n])
    assert torch.equal(torch.isfinite(host(r.lse[:n])), fin)
    close(r.out[:n], out[:n], tol[:n] + 1e-30, "out")
    if n:
        close(r.lse[:n][dev(fin)], lse[:n][fin], lse_tol[:n][fin], "lse")
        assert bool((host(r.lse[:n])[~fin] == -math.inf).all())
    # rows behind the last sequence are left as they were
    assert bool((r.out[n:] == 7.0).all()) and bool((r.lse[n:] == 7.0).all())


SHAPES = [  # hq, hkv, d, S, kv, q
    (4, 1, 64, 16, "f16", "f16"), (4, 4, 128, 16, "f16", "f16"), (8, 2, 128, 16, "bf16", "bf16"),
    (8, 1, 64, 32, "bf16", "bf16"), (4, 2, 128, 64, "f16", "f16"), (2, 1, 64, 128, "bf16", "bf16"),
    (8, 2, 128, 64, "i8", "f16"), (4, 4, 64, 32, "i8", "f16"), (8, 1, 128, 16, "i8", "bf16"),
    (2, 1, 64, 128, "i8", "bf16"), (8, 8, 64, 16, "i8", "f16"), (4, 2, 128, 128, "i8", "f16"),
]
RAGGED = [  # lens, new, rows behind
    ([1], [1], 0),
    ([300], [300], 0),
    ([0, 17, 64, 1], [0, 17, 3, 1], 5),
    ([129, 0, 700, 33], [1, 0, 130, 0], 0),
    ([1000, 255, 256, 257], [2, 255, 1, 128], 3),
    ([300, 0, 77, 16, 1000], [2, 0, 1, 0, 1], 0),  # few rows everywhere
    ([600, 601, 9, 40], [0, 30, 0, 1], 1),         # few on average, in one sequence
]


@pytest.mark.parametrize("lens, new, pad", RAGGED)
@pytest.mark.parametrize("hq, hkv, d, S, kv, q", SHAPES)
def test_chunk_attention(spg, hq, hkv, d, S, kv, q, lens, new, pad):
    r = Run(spg, R.Chunk(hq, hkv, d, S, kv, q, lens, new, pad_rows=pad))
    r.chunk()
    assert r.err() == 0
    check_chunk(r)


@pytest.mark.parametrize("kv, q, S", [("bf16", "bf16", 16), ("f16", "f16", 64), ("i8", "f16", 64)])
def test_chunk_attention_long_cache_few_rows(spg, kv, q, S):
    """Few rows over long ragged caches: the work of one tile is split over its tokens and joined."""
    r = Run(spg, R.Chunk(8, 2, 128, S, kv, q, [9000, 40, 5001], [3, 40, 1]))
    for _ in range(2):  # the second call finds the workspace as the first left it
        r.out.fill_(7.0)
        r.chunk()
        assert r.err() == 0
        check_chunk(r)
    a, b = r.out.clone(), r.lse.clone()
    r.chunk()
    assert torch.equal(a, r.out) and torch.equal(b, r.lse)


@pytest.mark.parametrize("kv, q", [("f16", "f16"), ("bf16", "bf16"), ("i8", "f16")])
def test_chunk_attention_growing_logits(spg, kv, q):
    """Logits that grow along the cache, and one far above the others: the running maximum moves many times."""
    c = R.Chunk(4, 2, 128, 16, kv, q, [777], [200])
    ramp = torch.linspace(0.1, 4.0, c.n_phys * 16).view(c.n_phys, 1, 16, 1)
    order = torch.argsort(c.page_table[0, : -(-777 // 16)].long())
    ramp_pages = torch.zeros_like(ramp)
    ramp_pages[c.page_table[0, : -(-777 // 16)].long()] = ramp[: -(-777 // 16)]
    del order
    if kv == "i8":
        c.k_scale = torch.where(torch.isfinite(c.k_scale), (ramp_pages[..., 0] * 0.02).half().expand_as(c.k_scale), c.k_scale)
    else:
        c.k_pool = (c.k_pool.float() * ramp_pages).to(c.k_pool.dtype)
    r = Run(spg, c)
    r.chunk()
    assert r.err() == 0
    check_chunk(r)


def test_chunk_equals_dense_decode_for_one_token(spg):
    c = R.Chunk(8, 2, 128, 16, "bf16", "bf16", [700, 1, 0, 33], [1, 1, 0, 1])
    r = Run(spg, c)
    r.chunk()
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16, device="cuda")
    q[[0, 1, 3]] = r.q
    out = torch.empty((4, 8, 128), device="cuda")
    lse = torch.empty((4, 8), device="cuda")
    spg.dense_decode_attention(r.p, q, r.k_pool, r.v_pool, None, None, r.page_table, r.seq_lens, out, lse, r.ws)
    assert r.err() == 0
    _, tol, _, lse_tol = R.attention(c)
    rows = [0, 1, 3]
    close(r.out, host(out)[rows].to(R.F64), tol * 2, "out")
    close(r.lse, host(lse)[rows].to(R.F64), lse_tol * 2, "lse")


@pytest.mark.parametrize("kv, q", [("f16", "f16"), ("i8", "f16")])
def test_bad_pages_are_skipped(spg, kv, q):
    c = R.Chunk(4, 2, 128, 16, kv, q, [100, 40, 16], [30, 40, 16], poison=0.0)
    r = Run(spg, c)
    r.page_table[0, 2] = c.n_phys      # one page of several
    r.page_table[1, 0] = -7            # rows that see that page alone are left with nothing
    r.page_table[2, 0] = 2 ** 30       # every token of the sequence
    r.chunk()
    assert r.err() == spg.DEVERR_PAGE_ID
    check_chunk(r, drop=[(0, 2), (1, 0), (2, 0)])
    spg.spg_clear_device_error(r.ws)
    m = torch.full((3, 2, c.mp * 16), 5.0, device="cuda")
    r.mass(r.lse, None, m, 1.0)
    assert r.err() == spg.DEVERR_PAGE_ID
    assert bool((m[0, :, 32:48] == 0).all()) and bool((m[1, :, :16] == 0).all()) and bool((m[2, :, :16] == 0).all())
    total = m[0, :, :100].sum(dim=1)
    assert torch.allclose(total, torch.full_like(total, 30.0 * 2), rtol=1e-4)  # each row of each head weighs 1


@pytest.mark.parametrize("starts, bits", [([0, 30, 20, 50], 16), ([-1, 30, 40, 50], 16), ([0, 30, 40, 60], 16)])
def test_bad_q_start_is_reported(spg, starts, bits):
    c = R.Chunk(4, 2, 64, 16, "f16", "f16", [100, 40, 16], [30, 10, 10])
    r = Run(spg, c)
    r.q_start.copy_(torch.tensor(starts, dtype=torch.int32))
    r.chunk()
    assert r.err() & bits
    spg.spg_clear_device_error(r.ws)
    r.mass(r.lse, None, torch.zeros((3, 2, c.mp * 16), device="cuda"), 1.0)
    assert r.err() & bits
    spg.spg_clear_device_error(r.ws)
    r.seq_lens[0] = c.mp * 16 + 1
    r.chunk()
    assert r.err() & spg.DEVERR_SEQ_LEN
    torch.cuda.synchronize()


def test_chunk_offsets_past_32_bits(spg):
    """Pages beyond 2^32 bytes and 2^31 elements of the pools."""
    n_phys = 2 ** 31 // (2 * 16 * 128) + 300
    c = R.Chunk(4, 2, 128, 16, "bf16", "bf16", [200, 70], [70, 70])
    r = Run(spg, c)
    for n in ("k_pool", "v_pool"):
        big = torch.empty((n_phys, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
        big[n_phys - c.n_phys :] = getattr(r, n)
        setattr(r, n, big)
    r.p.num_phys_pages = n_phys
    r.page_table = torch.where(r.page_table >= 0, r.page_table + (n_phys - c.n_phys), r.page_table)
    r.chunk()
    assert r.err() == 0
    check_chunk(r)
    m = torch.zeros((2, 2, c.mp * 16), device="cuda")
    r.mass(r.lse, None, m, 1.0)
    want, tol = R.mass_of(c, host(r.lse), None, 1.0)
    for b, L in enumerate(c.lens):
        close(m[b, :, :L], want[b, :, :L], tol[b, :, :L], "mass")
    # written there too: the chunk's keys and values
    c2 = R.Chunk(4, 2, 128, 16, "bf16", "bf16", [200, 70], [70, 70])
    r.append(None, torch.empty_like(r.q))
    assert r.err() == 0
    at = n_phys - c.n_phys + int(c2.page_table[0, 190 // 16])
    assert torch.equal(host(r.k_pool[at, :, 190 % 16]), c.k[190 - 130])
    kept = torch.empty((2, 2, 64), dtype=torch.int32, device="cuda")
    nl = torch.empty(2, dtype=torch.int32, device="cuda")
    src = host(r.k_pool[at, :, 190 % 16]).clone()
    spg.paged_cache_evict(r.p, m, 64, 0, 16, r.k_pool, r.v_pool, None, None, r.page_table, None, r.seq_lens, kept, nl, m,
                          r.ws)
    assert r.err() == 0
    j = host(kept)[0, 0].tolist().index(190)
    assert torch.equal(host(r.k_pool[n_phys - c.n_phys + int(c2.page_table[0, j // 16]), 0, j % 16]), src[0])


@pytest.mark.parametrize("scale", [0.01, 0.3, 2.0])
def test_chunk_attention_softmax_scale(spg, scale):
    """A caller's own scale: the reference's logits are those of q times scale sqrt(d)."""
    c = R.Chunk(4, 2, 64, 16, "bf16", "bf16", [300, 90], [40, 90])
    r = Run(spg, c, softmax_scale=scale)
    r.chunk()
    assert r.err() == 0
    exact = c.q
    c.q = c.q.double() * (scale * 8.0)
    out, tol, lse, lse_tol = R.attention(c)
    c.q = exact
    close(r.out, out, tol, "out")
    close(r.lse, lse, lse_tol, "lse")


def test_chunk_attention_many_sequences_and_odd_heads(spg):
    """More sequences than a warp has lanes, three kv-heads, prompts, continuations and empty ones."""
    g = torch.Generator().manual_seed(11)
    lens = torch.randint(0, 400, (70,), generator=g).tolist()
    new = [min(L, n) for L, n in zip(lens, torch.randint(0, 90, (70,), generator=g).tolist())]
    new[3:40:4] = [0] * len(new[3:40:4])
    for kv, q in (("f16", "f16"), ("i8", "bf16")):
        c = R.Chunk(6, 3, 64, 32, kv, q, lens, new, pad_rows=7)
        r = Run(spg, c)
        r.chunk()
        assert r.err() == 0
        check_chunk(r)
        want, tol = R.mass_of(c, host(r.lse), None, 1.0)
        m = torch.zeros((70, 3, c.mp * 32), device="cuda")
        r.mass(r.lse, None, m, 1.0)
        assert r.err() == 0
        for b, L in enumerate(lens):
            close(m[b, :, :L], want[b, :, :L], tol[b, :, :L], "mass")


def test_one_workspace_for_chunks_of_all_sizes(spg):
    """Chunks of other sizes, batches and lengths one after the other on the workspace of the largest."""
    big = R.Chunk(8, 2, 128, 16, "bf16", "bf16", [4000, 700, 1], [600, 10, 1])
    small = R.Chunk(8, 2, 128, 16, "bf16", "bf16", [4000, 33, 5], [1, 1, 1], mp=big.mp)
    rb, rs = Run(spg, big), Run(spg, small)
    rs.ws = rb.ws
    for r in (rb, rs, rb, rs):
        r.out.fill_(7.0)
        r.lse.fill_(7.0)
        r.chunk()
        assert r.err() == 0
        check_chunk(r)


def test_two_streams_with_their_own_workspaces(spg):
    """Two chunks, their weights and an eviction in flight at once give what they give alone."""
    rs = [Run(spg, R.Chunk(8, 2, 128, 16, "bf16", "bf16", [3000, 900], [300, 900], seed=s)) for s in (1, 2)]
    masses = [torch.zeros((2, 2, r.c.mp * 16), device="cuda") for r in rs]
    alone = []
    for r, m in zip(rs, masses):
        r.chunk()
        r.mass(r.lse, None, m, 1.0)
        alone.append([t.clone() for t in (r.out, r.lse, m)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in rs]
    for _ in range(5):
        for r, m in zip(rs, masses):
            r.out.zero_(), r.lse.zero_(), m.zero_()
        torch.cuda.synchronize()
        for st, r, m in zip(streams, rs, masses):
            with torch.cuda.stream(st):
                r.chunk()
                r.mass(r.lse, None, m, 1.0)
        torch.cuda.synchronize()
        for r, m, want in zip(rs, masses, alone):
            assert r.err() == 0
            for a, b in zip((r.out, r.lse, m), want):
                assert torch.equal(a, b)


# ---- mass -------------------------------------------------------------------------------------


@pytest.mark.parametrize("lens, new, pad", RAGGED)
@pytest.mark.parametrize("hq, hkv, d, S, kv, q", SHAPES)
def test_attention_mass(spg, hq, hkv, d, S, kv, q, lens, new, pad):
    c = R.Chunk(hq, hkv, d, S, kv, q, lens, new, pad_rows=pad)
    r = Run(spg, c)
    lse = R.attention(c)[2].float()
    g = torch.Generator().manual_seed(1)
    for decay, given in ((1.0, True), (0.0, True), (0.5, True), (1.0, False)):
        old = torch.rand((len(lens), hkv, c.mp * S), generator=g)
        if decay == 0.0:
            old[:] = math.nan  # not read
        for b, L in enumerate(lens):
            old[b, :, L - new[b] :] = math.nan  # slots that held nothing before the chunk
        want, tol = R.mass_of(c, lse, old if given else None, decay)
        out = torch.full(old.shape, 3.0, device="cuda")
        r.mass(dev(lse), dev(old) if given else None, out, decay)
        assert r.err() == 0
        for b, L in enumerate(lens):
            close(out[b, :, :L], want[b, :, :L], tol[b, :, :L], "mass")
            assert bool((out[b, :, L:] == 3.0).all())
        if given and decay == 0.5:  # in place gives the same bits, and so does a second call
            acc = dev(old)
            r.mass(dev(lse), acc, acc, decay)
            for b, L in enumerate(lens):
                assert torch.equal(acc[b, :, :L], out[b, :, :L])


def test_mass_without_rows(spg):
    """An empty chunk decays what is there; a row without a log-sum-exp adds nothing."""
    c = R.Chunk(4, 2, 64, 16, "f16", "f16", [40, 9], [0, 0])
    r = Run(spg, c)
    old = torch.rand((2, 2, c.mp * 16), device="cuda")
    out = torch.full_like(old, 3.0)
    r.mass(r.lse, old, out, 0.25)
    assert r.err() == 0
    assert torch.equal(out[0, :, :40], old[0, :, :40] * 0.25) and bool((out[0, :, 40:] == 3.0).all())
    assert torch.equal(out[1, :, :9], old[1, :, :9] * 0.25) and bool((out[1, :, 9:] == 3.0).all())
    c = R.Chunk(4, 2, 64, 16, "f16", "f16", [40], [5])
    r = Run(spg, c)
    lse = torch.full((5, 4), -math.inf, device="cuda")
    out = torch.full((1, 2, c.mp * 16), 3.0, device="cuda")
    r.mass(lse, None, out, 1.0)
    assert bool((out[0, :, :40] == 0).all())


# ---- rotary append ------------------------------------------------------------------------------


@pytest.mark.parametrize("layout, rot, scaling", [("half", 0, "none"), ("interleaved", 0, "yarn"), ("half", 32, "linear"),
                                                  ("interleaved", 16, "ntk"), ("half", 48, "yarn")])
@pytest.mark.parametrize("hq, hkv, d, S, kv, q", SHAPES)
def test_rope_append(spg, hq, hkv, d, S, kv, q, layout, rot, scaling):
    for lens, new, pad in RAGGED[1:]:
        check_append(spg, R.Chunk(hq, hkv, d, S, kv, q, lens, new, pad_rows=pad), layout, rot, scaling)


def check_append(spg, c, layout, rot, scaling, positions=None, fused=False):
    r = Run(spg, c)
    if fused:  # q, k and v as slices of one projection's rows
        qkv = torch.cat([r.q, r.k, r.v], dim=1)
        r.q, r.k, r.v = qkv[:, : c.hq], qkv[:, c.hq : c.hq + c.hkv], qkv[:, c.hq + c.hkv :]
    before = [host(t).clone() if t is not None else None for t in (r.k_pool, r.v_pool, r.k_scale, r.v_scale)]
    rope = spg.make_rope(rot_dim=rot, layout=layout, scaling=scaling, factor=4.0, orig_len=512)
    q_out = torch.full((c.T, c.hq, c.d), 7.0, dtype=R.DT[c.qdt], device="cuda")
    r.append(rope, q_out, None if positions is None else positions.cuda())
    assert r.err() == 0
    rd = rot or c.d
    inv, m = R.rope_freqs(rd, 10000.0, scaling, 4.0, 512)
    n = c.starts[-1]
    cache_pos = torch.cat([torch.arange(L - k, L) for L, k in zip(c.lens, c.new)] + [torch.zeros(0)]).long()
    owner = torch.cat([torch.full((k,), b) for b, k in enumerate(c.new)] + [torch.zeros(0)]).long()
    pos = cache_pos if positions is None else positions[:n].long()
    e = torch.finfo(R.DT[c.qdt]).eps / 2
    sub = 2.0 ** -25 if c.qdt == "f16" else 0.0
    want = R.rotate(c.q[:n], pos, rd, layout, inv, m)
    close(q_out[:n], want, e * want.abs() + (1 + e) * R.rotate_tol(c.q[:n], rd, layout, m) + sub, "q")
    assert bool((q_out[n:] == 7.0).all())
    k = R.rotate(c.k[:n], pos, rd, layout, inv, m)
    kt = R.rotate_tol(c.k[:n], rd, layout, m)
    v = c.v[:n].to(R.F64)
    phys = c.page_table[owner, cache_pos // c.S].long()
    slot = cache_pos % c.S
    written = torch.zeros((c.n_phys, c.S), dtype=torch.bool)
    written[phys, slot] = True
    for x, tol, pool, scale, old, olds in ((k, kt, r.k_pool, r.k_scale, before[0], before[2]),
                                           (v, torch.zeros_like(kt), r.v_pool, r.v_scale, before[1], before[3])):
        got = host(pool)[phys, :, slot].to(R.F64)
        if c.kv == "i8":
            s = host(scale)[phys, :, slot].to(R.F64)
            amax = x.abs().amax(dim=-1)
            assert bool(((s - amax / 127).abs() <= amax / 127 * (2.0 ** -11 + 1e-6) + 2.0 ** -25 + (amax == 0) * 1.0).all())
            d = (got * s[..., None] - x).abs()
            # half a step, and for the largest what the rounded scale falls short of it: 127 * 2^-11 of a step
            assert bool((d <= s[..., None] * (0.5 + 127 * 2.0 ** -11 + 1e-4) + tol).all())
            assert int(got.abs().max()) <= 127 if n else True
        elif pool is r.v_pool:
            assert torch.equal(got, x)
        else:
            assert bool(((got - x).abs() <= e * x.abs() + (1 + e) * tol + sub).all())
        # nothing else of the pool changes
        keep = ~written[:, None].expand(c.n_phys, c.hkv, c.S)
        as_bits = lambda t: t.view(torch.int16) if t.dtype != torch.int8 else t  # noqa: E731
        assert torch.equal(as_bits(host(pool))[keep], as_bits(old)[keep])
        if olds is not None:
            assert torch.equal(as_bits(host(scale))[keep], as_bits(olds)[keep])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kv, q", [("bf16", "bf16"), ("f16", "f16"), ("i8", "f16")])
def test_rope_append_far_positions_and_slices(spg, kv, q, layout):
    c = R.Chunk(4, 2, 128, 16, kv, q, [50, 3], [20, 3], pad_rows=2)
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, 2 ** 31 - 1, (c.T,), generator=g, dtype=torch.int64)
    pos[:3] = torch.tensor([2 ** 31 - 1, 0, 2 ** 24 + 1])
    # at 2^31 the 64-bit reference itself holds t * f to 2^31 * 2^-52 = 5e-7; kept under it by 2^26
    check_append(spg, c, layout, 0, "none", torch.minimum(pos, torch.tensor(2 ** 26 + 3)).int(), fused=True)


def test_rope_append_in_place_zero_rows_and_no_rotation(spg):
    c = R.Chunk(4, 2, 128, 16, "i8", "f16", [5], [5])
    c.k[2] = 0.0
    c.v[3, 1] = 0.0
    r = Run(spg, c)
    q0 = r.q.clone()
    r.append(None, r.q)
    assert r.err() == 0 and torch.equal(r.q, q0)
    pg = int(c.page_table[0, 0])
    assert bool((r.k_pool[pg, :, 2] == 0).all()) and bool((r.k_scale[pg, :, 2] == 1).all())
    assert bool((r.v_pool[pg, 1, 3] == 0).all()) and float(r.v_scale[pg, 1, 3]) == 1.0
    rope = spg.make_rope()
    other = torch.empty_like(r.q)
    r.append(rope, other)
    r.append(rope, r.q)  # in place: the same bits
    assert torch.equal(r.q, other)
    # keys and values alone
    spg.paged_rope_append(r.p, rope, None, r.k, r.v, r.q_start, r.page_table, r.seq_lens, r.k_pool, r.v_pool, r.k_scale,
                          r.v_scale, None, ws=r.ws)
    assert r.err() == 0


# ---- eviction -----------------------------------------------------------------------------------


def cached(c, r, b, h, t):
    pg, s = host(r.page_table)[b, t // c.S], t % c.S
    return pg, s


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kv, q, d, S", [("f16", "f16", 128, 16), ("bf16", "bf16", 64, 32), ("i8", "f16", 128, 64),
                                         ("i8", "bf16", 64, 16)])
@pytest.mark.parametrize("lens, keep, sink, recent", [([1], 1, 0, 0), ([70, 0, 33, 200], 33, 1, 5),
                                                      ([500, 64, 65], 64, 0, 0), ([3000, 2999], 1500, 4, 700),
                                                      ([300], 10, 5, 5), ([9000, 100], 5000, 2, 64)])
def test_evict(spg, lens, keep, sink, recent, kv, q, d, S, in_place):
    check_evict(spg, lens, keep, sink, recent, kv, q, d, S, in_place, "lognormal")


@pytest.mark.parametrize("masses", ["equal", "zeros", "three", "nan", "inf", "denormal", "near"])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict_ties_and_odd_masses(spg, masses, in_place):
    check_evict(spg, [700, 100, 5000], 300, 3, 20, "f16", "f16", 64, 16, in_place, masses)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("masses", ["lognormal", "three"])
def test_evict_tables_past_shared_memory(spg, masses, in_place):
    """A page table of more tokens than a cluster's shared memory holds masses of."""
    check_evict(spg, [3000, 40], 500, 2, 33, "bf16", "bf16", 64, 16, in_place, masses, mp=25000)
    check_evict(spg, [30000], 20000, 2, 33, "i8", "f16", 64, 16, in_place, masses)
    check_evict(spg, [20000], 500, 2, 33, "f16", "f16", 64, 16, in_place, masses, mp=24576)  # the most that it holds


def check_evict(spg, lens, keep, sink, recent, kv, q, d, S, in_place, masses, mp=0):
    B, hkv = len(lens), 2
    dst_pages = [-(-min(L, keep) // S) for L in lens]
    c = R.Chunk(4, hkv, d, S, kv, q, lens, [0] * B, extra_pages=0 if in_place else sum(dst_pages), mp=mp)
    r = Run(spg, c)
    g = torch.Generator().manual_seed(9)
    N = c.mp * S
    m = torch.exp(2 * torch.randn((B, hkv, N), generator=g))
    if masses == "equal":
        m[:] = 0.25
    elif masses == "zeros":
        m[:] = 0.0
        m[:, :, 50:60] = 1.0
    elif masses == "three":
        m = torch.randint(0, 3, m.shape, generator=g).float()
    elif masses == "nan":
        m[:, :, 7::11] = math.nan
        m[:, :, 5::13] = -math.inf
    elif masses == "inf":
        m[:, :, 3::7] = math.inf
        m[:, :, 4::7] = -1.0
    elif masses == "denormal":
        m *= 1e-41
    elif masses == "near":
        m = 1.0 + torch.randint(0, 5, m.shape, generator=g).float() * 2.0 ** -23
    for b, L in enumerate(lens):
        m[b, :, L:] = 99.0  # never read
    dst = None
    if not in_place:
        dst = torch.full((B, c.mp), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            dst[b, : dst_pages[b]] = c.free[at : at + dst_pages[b]]
            at += dst_pages[b]
    mass = m.cuda()
    mass_out = mass if in_place else torch.full_like(mass, 5.0)
    kept = torch.full((B, hkv, keep), 77, dtype=torch.int32, device="cuda")
    new_lens = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    spg.paged_cache_evict(r.p, mass, keep, sink, recent, r.k_pool, r.v_pool, r.k_scale, r.v_scale, r.page_table, dev(dst),
                          r.seq_lens, kept, new_lens, mass_out, r.ws)
    assert r.err() == 0
    assert host(new_lens).tolist() == [min(L, keep) for L in lens]
    bits = lambda t: t.view(torch.int16) if t.dtype != torch.int8 else t  # noqa: E731
    expect = [bits(t.clone()) if t is not None else None for t in (c.k_pool, c.v_pool, c.k_scale, c.v_scale)]
    table = c.page_table if in_place else dst
    want_mass = m.clone() if in_place else torch.full_like(m, 5.0)
    for b, L in enumerate(lens):
        for h in range(hkv):
            ids = R.kept_positions(m[b, h].tolist(), L, keep, sink, recent)
            assert host(kept)[b, h].tolist() == ids + [-1] * (keep - len(ids)), (b, h)
            t, j = torch.tensor(ids, dtype=torch.long), torch.arange(len(ids))
            for x, src in zip(expect, (c.k_pool, c.v_pool, c.k_scale, c.v_scale)):
                if x is not None:
                    x[table[b, j // S].long(), h, j % S] = bits(src)[c.page_table[b, t // S].long(), h, t % S]
            want_mass[b, h, : len(ids)] = m[b, h, t]
    for x, got in zip(expect, (r.k_pool, r.v_pool, r.k_scale, r.v_scale)):
        if x is not None:
            assert torch.equal(bits(host(got)), x)
    assert torch.equal(host(mass_out).view(torch.int32), want_mass.view(torch.int32))


def test_evict_bad_pages_and_lengths(spg):
    c = R.Chunk(4, 2, 64, 16, "f16", "f16", [100, 60], [0, 0])
    r = Run(spg, c)
    r.page_table[0, 3] = -5
    mass = torch.rand((2, 2, c.mp * 16), device="cuda")
    kept = torch.empty((2, 2, 50), dtype=torch.int32, device="cuda")
    nl = torch.empty(2, dtype=torch.int32, device="cuda")
    args = lambda: spg.paged_cache_evict(r.p, mass, 50, 0, 50, r.k_pool, r.v_pool, None, None, r.page_table, None,  # noqa: E731
                                         r.seq_lens, kept, nl, mass, r.ws)
    args()
    assert r.err() == spg.DEVERR_PAGE_ID
    assert host(kept)[1, 0].tolist() == list(range(10, 60))
    spg.spg_clear_device_error(r.ws)
    r.seq_lens[0] = -1
    args()
    assert r.err() & spg.DEVERR_SEQ_LEN
    assert host(nl).tolist()[0] == 0 and bool((kept[0] == -1).all())


# ---- together, streams and graphs -----------------------------------------------------------------


def serve(spg, r, rope, q_out, mass, kept, new_lens, buf, decode_q, sel):
    """A prompt into the cache, its attention and weights, the light half evicted, one decode step over the rest."""
    r.append(rope, q_out)
    spg.paged_chunk_attention(r.p, q_out, r.q_start, r.k_pool, r.v_pool, r.k_scale, r.v_scale, r.page_table, r.seq_lens,
                              r.out, r.lse, r.ws)
    spg.paged_attention_mass(r.p, q_out, r.q_start, r.k_pool, r.k_scale, r.page_table, r.seq_lens, r.lse, None, mass, 1.0,
                             r.ws)
    spg.paged_cache_evict(r.p, mass, kept.shape[2], 4, 16, r.k_pool, r.v_pool, r.k_scale, r.v_scale, r.page_table, None,
                          r.seq_lens, kept, new_lens, mass, r.ws)
    spg.sparse_page_meta_update(sel, r.k_pool, r.k_scale, r.page_table, new_lens, 1, buf.minmax, None, None, None, r.ws)
    spg.sparse_decode_select_attend(sel, decode_q, r.k_pool, r.v_pool, r.k_scale, r.v_scale, r.page_table, new_lens,
                                    buf.minmax, None, None, None, buf.sel, buf.sel_cnt, buf.out, buf.lse, r.ws)


@pytest.mark.parametrize("kv, q", [("bf16", "bf16"), ("f16", "f16"), ("i8", "f16")])
def test_operators_together(spg, kv, q):
    """Each operator's result is the next one's input; checked at every step against the 64-bit forms of that input,
    eagerly on a stream of its own and replayed from a graph."""
    c = R.Chunk(8, 2, 128, 16, kv, q, [300, 129, 40], [300, 60, 1])
    r = Run(spg, c, selector="quest", token_budget=16 * 16, n_sink_pages=1, n_recent_pages=1)
    sel = r.p
    buf = spg.alloc_buffers(sel)
    keep = 128
    rope = spg.make_rope(base=10000.0, scaling="yarn", factor=2.0, orig_len=128)
    q_out = torch.empty_like(r.q)
    mass = torch.zeros((3, 2, c.mp * 16), device="cuda")
    kept = torch.empty((3, 2, keep), dtype=torch.int32, device="cuda")
    new_lens = torch.empty(3, dtype=torch.int32, device="cuda")
    dq = torch.randn((3, 8, 128), device="cuda").to(R.DT[q])
    pools = [t.clone() if t is not None else None for t in (r.k_pool, r.v_pool, r.k_scale, r.v_scale)]
    args = (spg, r, rope, q_out, mass, kept, new_lens, buf, dq, sel)

    def restore():
        for t, o in zip((r.k_pool, r.v_pool, r.k_scale, r.v_scale), pools):
            if o is not None:
                t.copy_(o)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        serve(*args)
    side.synchronize()
    assert r.err() == 0
    res = [t.clone() for t in (q_out, r.out, r.lse, mass, kept, new_lens, buf.out, buf.lse, buf.sel)]

    # step by step: the attention over the cache as appended
    restore()
    r.append(rope, q_out)
    c.q, c.k_pool, c.v_pool = host(q_out), host(r.k_pool), host(r.v_pool)
    c.k_scale, c.v_scale = (None, None) if kv != "i8" else (host(r.k_scale), host(r.v_scale))
    r.out.copy_(res[1])
    r.lse.copy_(res[2])
    check_chunk(r)
    w, tol = R.mass_of(c, host(res[2]), None, 1.0)
    spg.paged_attention_mass(r.p, q_out, r.q_start, r.k_pool, r.k_scale, r.page_table, r.seq_lens, res[2], None, mass, 1.0,
                             r.ws)
    for b, L in enumerate(c.lens):
        close(mass[b, :, :L], w[b, :, :L], tol[b, :, :L], "mass")
    for b, L in enumerate(c.lens):
        for h in range(2):
            ids = R.kept_positions(host(mass)[b, h].tolist(), L, keep, 4, 16)
            assert host(res[4])[b, h].tolist()[: len(ids)] == ids
            k = c.tokens(c.k_pool, c.k_scale, b, h)[ids]
            v = c.tokens(c.v_pool, c.v_scale, b, h)[ids]
            z = host(dq)[b, h * 4 : h * 4 + 4].to(R.F64) @ k.T / math.sqrt(128)
            # a budget of 16 pages covers every one of the 8 kept
            o = torch.softmax(z, dim=1) @ v
            assert float((host(res[6])[b, h * 4 : h * 4 + 4].to(R.F64) - o).abs().max()) <= 5e-3

    restore()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        serve(*args)
    for _ in range(2):
        restore()
        for t in (q_out, r.out, r.lse, mass):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert r.err() == 0
        for got, want in zip((q_out, r.out, r.lse, kept, new_lens, buf.out, buf.lse, buf.sel),
                             res[:3] + res[4:]):
            assert torch.equal(got, want)
