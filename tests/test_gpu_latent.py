"""The latent-cache operators on the GPU against their 64-bit forms (tests/latent_ref.py, where the tolerances are
derived): ragged chunks, empty sequences, padded batches, values past the lengths, bad pages, streams and graphs, and
the operators one after the other as a serving loop runs them."""

import math

import pytest
import torch

import latent_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spg():
    import query_aware_sparse_page_gb300 as m

    return m


def host(t):
    return t.detach().cpu()


class Run:
    """A chunk's tensors on the GPU, with its parameters and workspace."""

    def __init__(self, spg, c, **kw):
        self.spg, self.c = spg, c
        self.p = c.params(spg, **kw)
        assert spg.spg_latent_validate(self.p) == 0
        self.ws = torch.zeros(spg.spg_latent_workspace_size(self.p, c.T), dtype=torch.uint8, device="cuda")
        for n in ("q", "q_lat", "kv", "pool", "w_kv", "norm", "page_table", "seq_lens", "q_start"):
            setattr(self, n, getattr(c, n).cuda())
        dt = R.DT[c.dt]
        self.o_lat = torch.full((c.T, c.H, c.r), 7.0, dtype=dt, device="cuda")
        self.lse = torch.full((c.T, c.H), 7.0, device="cuda")
        self.out = torch.full((c.T, c.H, c.dv), 7.0, dtype=dt, device="cuda")

    def attend(self, **kw):
        self.spg.paged_latent_attention(self.p, self.q_lat, self.q_start, self.pool, self.page_table, self.seq_lens,
                                        self.o_lat, self.lse, self.ws, **kw)

    def append(self, rope, norm=True, eps=1e-6, **kw):
        c = self.c
        self.spg.paged_latent_append(self.p, rope, self.kv[:, : c.r], self.kv[:, c.r :], self.norm if norm else None, eps,
                                     self.q, self.q_start, self.page_table, self.seq_lens, self.pool, self.q_lat,
                                     ws=self.ws, **kw)

    def err(self):
        return self.spg.spg_read_device_error(self.ws)


def close(got, want, tol, what):
    d = (host(got).to(R.F64) - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {d[bad].max():.3e} (allowed {tol[bad].min():.3e})"


def check_attend(r, drop=(), parts=2):
    c = r.c
    out, tol, lse, lse_tol = R.attention(c, drop, parts)
    n = c.starts[-1]
    fin = torch.isfinite(lse[:n])
    assert torch.equal(torch.isfinite(host(r.lse[:n])), fin)
    close(r.o_lat[:n], out[:n], tol[:n] + 1e-30, "o_lat")
    if n:
        close(r.lse[:n][fin.cuda()], lse[:n][fin], lse_tol[:n][fin], "lse")
        assert bool((host(r.lse[:n])[~fin] == -math.inf).all())
    # rows behind the last sequence are left as they were
    assert bool((r.o_lat[n:] == 7.0).all()) and bool((r.lse[n:] == 7.0).all())


SHAPES = [  # H, r, S, dtype
    (4, 256, 16, "f16"), (16, 512, 64, "bf16"), (1, 512, 16, "f16"), (20, 256, 32, "bf16"), (64, 512, 128, "f16"),
    (128, 512, 64, "bf16"), (96, 256, 16, "f16"), (7, 512, 32, "bf16"), (130, 256, 128, "bf16"),
]
RAGGED = [  # lens, new, rows behind
    ([1], [1], 0),
    ([64], [1], 0),
    ([0, 17, 64, 1], [0, 17, 3, 1], 5),
    ([129, 0, 700, 33], [1, 0, 13, 0], 0),
    ([1000, 65, 256, 257], [2, 65, 1, 28], 3),
    ([300, 0, 77, 16, 1000], [2, 0, 1, 0, 1], 0),  # few rows everywhere
    ([600, 601, 9, 40], [0, 30, 0, 1], 1),         # few on average, many in one sequence
]


@pytest.mark.parametrize("lens, new, pad", RAGGED)
@pytest.mark.parametrize("H, r, S, dt", SHAPES)
def test_attention(spg, H, r, S, dt, lens, new, pad):
    x = Run(spg, R.Latent(H, r, S, dt, lens, new, pad_rows=pad))
    x.attend()
    assert x.err() == 0
    check_attend(x)


@pytest.mark.parametrize("dt, H, S, r", [("bf16", 16, 16, 512), ("f16", 64, 64, 512), ("bf16", 128, 32, 512), ("f16", 24, 128, 256)])
def test_attention_long_cache_few_rows(spg, dt, H, S, r):
    """Few rows over long ragged caches: an item's steps are split over many CTAs and joined."""
    x = Run(spg, R.Latent(H, r, S, dt, [9000, 40, 5001], [3, 40, 1]))
    for _ in range(2):  # the second call finds the workspace as the first left it
        x.o_lat.fill_(7.0)
        x.attend()
        assert x.err() == 0
        check_attend(x)
    a, b = x.o_lat.clone(), x.lse.clone()
    x.attend()
    assert torch.equal(a, x.o_lat) and torch.equal(b, x.lse)


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention_parts(spg, dt, parts):
    x = Run(spg, R.Latent(16, 512, 64, dt, [500, 300], [3, 1]))
    try:
        spg.spg_set_chunk_parts(parts)
        x.attend()
    finally:
        spg.spg_set_chunk_parts(2)
    assert x.err() == 0
    check_attend(x, parts=parts)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("up", [True, False])
def test_attention_moving_logits(spg, dt, up):
    """Logits that grow (or fall) along the cache: the running maximum moves many times, or once."""
    c = R.Latent(16, 512, 16, dt, [777, 1300], [5, 1])
    for b, L in enumerate(c.lens):
        n = -(-L // 16)
        ramp = torch.linspace(0.1, 6.0, n) if up else torch.linspace(6.0, 0.1, n)
        pg = c.page_table[b, :n].long()
        c.pool[pg] = (c.pool[pg].float() * ramp[:, None, None]).to(c.pool.dtype)
    x = Run(spg, c)
    x.attend()
    assert x.err() == 0
    check_attend(x)


def test_attention_softmax_scale(spg):
    c = R.Latent(8, 256, 32, "f16", [200], [3])
    c.scale = 0.25
    x = Run(spg, c, softmax_scale=0.25)
    x.attend()
    check_attend(x)


@pytest.mark.parametrize("H, dt", [(4, "f16"), (128, "bf16")])
def test_bad_pages_are_skipped(spg, H, dt):
    c = R.Latent(H, 512, 16, dt, [100, 40, 16], [30, 40, 16], poison=math.nan)
    x = Run(spg, c)
    x.page_table[0, 2] = c.n_phys      # one page of several
    x.page_table[1, 0] = -7            # rows that see that page alone are left with nothing
    x.page_table[2, 0] = 2 ** 30       # every token of the sequence
    x.attend()
    assert x.err() == spg.DEVERR_PAGE_ID
    check_attend(x, drop=[(0, 2), (1, 0), (2, 0)])


@pytest.mark.parametrize("starts", [[0, 30, 20, 50], [-1, 30, 40, 50], [0, 30, 40, 60]])
def test_bad_rows_are_reported(spg, starts):
    c = R.Latent(4, 256, 16, "f16", [100, 40, 16], [30, 10, 10])
    x = Run(spg, c)
    x.q_start.copy_(torch.tensor(starts, dtype=torch.int32))
    x.attend()
    assert x.err() & spg.DEVERR_Q_START
    spg.spg_clear_device_error(x.ws)
    x.append(None)
    assert x.err() & spg.DEVERR_Q_START
    x = Run(spg, c)  # the append above wrote what was sound of its chunk
    x.seq_lens[0] = c.mp * 16 + 1
    x.attend()
    assert x.err() & spg.DEVERR_SEQ_LEN
    # the sequences that are sound have their results
    c.new[0] = 0
    want, tol, _, _ = R.attention(c)
    close(x.o_lat[30:], want[30:], tol[30:], "o_lat")


def test_offsets_past_32_bits(spg):
    """Pages beyond 2^32 bytes and 2^31 elements of the pool."""
    c = R.Latent(16, 512, 64, "bf16", [200, 70], [2, 70])
    n_phys = 2 ** 32 // (64 * 576) + 300
    x = Run(spg, c)
    big = torch.empty((n_phys, 64, 576), dtype=torch.bfloat16, device="cuda")
    big[n_phys - c.n_phys :] = x.pool
    x.pool, x.p.num_phys_pages = big, n_phys
    x.page_table = torch.where(x.page_table >= 0, x.page_table + (n_phys - c.n_phys), x.page_table)
    x.attend()
    assert x.err() == 0
    check_attend(x)
    x.append(None, norm=False)
    assert x.err() == 0
    assert torch.equal(x.pool[x.page_table[0, 3].long(), 199 - 192], x.kv[1])


def test_many_sequences(spg):
    g = torch.Generator().manual_seed(5)
    lens = [int(v) for v in torch.randint(0, 200, (170,), generator=g)]
    new = [min(L, int(v)) for L, v in zip(lens, torch.randint(0, 4, (170,), generator=g))]
    x = Run(spg, R.Latent(16, 256, 16, "bf16", lens, new, pad_rows=2))
    x.attend()
    assert x.err() == 0
    check_attend(x)


# ---- the products around it --------------------------------------------------------------


@pytest.mark.parametrize("T", [1, 5, 127, 128, 129, 300])
@pytest.mark.parametrize("H, r, dn, dv, dt", [(3, 512, 128, 128, "bf16"), (16, 256, 64, 128, "f16"), (130, 512, 128, 64, "bf16"),
                                              (1, 256, 128, 64, "f16"), (2, 512, 64, 64, "bf16")])
def test_head_products(spg, H, r, dn, dv, dt, T):
    if H > 100 and T > 130:
        T = 140
    c = R.Latent(H, r, 16, dt, [T], [T], dn=dn, dv=dv)
    x = Run(spg, c)
    x.q_lat.fill_(5.0)
    spg.latent_absorb(x.p, x.q, x.w_kv, x.q_lat)
    y, tol = R.absorb(c)
    close(x.q_lat[..., :r], y, tol, "absorb")
    assert bool((x.q_lat[..., r:] == 5.0).all())
    o = (0.1 * torch.randn(T, H, r, generator=torch.Generator().manual_seed(T))).to(R.DT[dt])
    spg.latent_project(x.p, o.cuda(), x.w_kv, x.out)
    y, tol = R.project(c, o)
    close(x.out, y, tol, "project")


def test_absorb_strided_queries(spg):
    """Queries that are a slice of a wider projection's rows."""
    c = R.Latent(4, 512, 16, "bf16", [50], [50])
    x = Run(spg, c)
    wide = torch.full((50, 6, 192), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, :4] = x.q
    spg.latent_absorb(x.p, wide[:, :4], x.w_kv, x.q_lat)
    y, tol = R.absorb(c)
    close(x.q_lat[..., :512], y, tol, "absorb")


def test_products_behind_the_rows_are_left(spg):
    """Buffers longer than the rows of the call."""
    c = R.Latent(2, 256, 16, "f16", [40], [40])
    x = Run(spg, c)
    x.q_lat.fill_(5.0)
    spg.latent_absorb(x.p, x.q[:33], x.w_kv, x.q_lat[:33])
    assert bool((x.q_lat[33:] == 5.0).all())
    spg.latent_project(x.p, x.o_lat[:33], x.w_kv, x.out[:33])
    assert bool((x.out[33:] == 7.0).all())


# ---- into the cache ------------------------------------------------------------------------


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot, scaling, norm", [(64, "none", True), (32, "yarn", True), (48, "ntk", False), (64, "linear", False)])
@pytest.mark.parametrize("H, r, S, dt", [(1, 256, 16, "f16"), (16, 512, 64, "bf16"), (50, 512, 32, "f16"), (128, 256, 128, "bf16")])
def test_append(spg, H, r, S, dt, rot, scaling, norm, layout):
    c = R.Latent(H, r, S, dt, [0, 17, 64, 1, 200], [0, 17, 3, 1, 30], pad_rows=4, extra_pages=2)
    x = Run(spg, c)
    x.q_lat.fill_(5.0)
    before = x.pool.clone()
    rope = spg.make_rope(rot_dim=rot, layout=layout, base=1e4, scaling=scaling, factor=4.0, orig_len=2048)
    inv, m = R.rope_freqs(rot, 1e4, scaling, 4.0, 2048)
    x.append(rope, norm=norm, eps=1e-5)
    assert x.err() == 0
    row, row_tol, q, q_tol = R.append(c, rot, layout, inv, m, 1e-5, norm)
    n = c.starts[-1]
    close(x.q_lat[:n, :, r:], q[:n], q_tol[:n], "q_lat")
    assert bool((x.q_lat[:, :, :r] == 5.0).all()) and bool((x.q_lat[n:] == 5.0).all())
    pool, untouched = host(x.pool), torch.ones(c.n_phys, S, dtype=torch.bool)
    for b, L in enumerate(c.lens):
        for i in range(c.new[b]):
            t = L - c.new[b] + i
            pg, sl = int(c.page_table[b, t // S]), t % S
            k = c.starts[b] + i
            close(pool[pg, sl], row[k], row_tol[k], f"row {k}")
            untouched[pg, sl] = False
    a, w = pool[untouched].view(torch.int16), host(before)[untouched].view(torch.int16)
    assert torch.equal(a, w)


def test_append_positions_and_plain(spg):
    """Positions of their own, far ones among them; without rope, norm and queries rows are copied as they are."""
    c = R.Latent(3, 512, 16, "bf16", [40], [5])
    x = Run(spg, c)
    pos = torch.tensor([0, 7, 100000, 2 ** 31 - 1, 12345], dtype=torch.int32)
    x.append(spg.make_rope(rot_dim=64, layout="interleaved"), positions=pos.cuda())
    inv, m = R.rope_freqs(64, 1e4, "none", 1.0, 1)
    row, row_tol, q, q_tol = R.append(c, 64, "interleaved", inv, m, 1e-6, True, pos)
    # the reference's own angle is a product in 64 bits: t * 2^-53 of it in all
    far = 2.0 ** 31 * 2.0 ** -52
    size = c.q[..., c.dn :].abs().amax().item() * 2
    close(x.q_lat[:, :, 512:], q, q_tol + far * size, "q_lat")
    x.q_lat.fill_(5.0)
    spg.paged_latent_append(x.p, None, x.kv[:, :512], x.kv[:, 512:], None, 0.0, None, x.q_start, x.page_table, x.seq_lens,
                            x.pool, ws=x.ws)
    pg = x.page_table[0].long()
    assert torch.equal(x.pool[pg].view(-1, 576)[35:40], x.kv) and bool((x.q_lat == 5.0).all())
    assert x.err() == 0


def test_append_bad_page_writes_nothing_there(spg):
    c = R.Latent(2, 256, 16, "f16", [40, 20], [20, 3], poison=0.0)
    x = Run(spg, c)
    x.page_table[0, 2] = -1
    before = x.pool.clone()
    x.append(None, norm=False)
    assert x.err() == spg.DEVERR_PAGE_ID
    assert torch.equal(x.q_lat[:, :, 256:], x.q[:, :, c.dn :])
    changed = (x.pool != before).any(dim=2)
    assert int(changed.sum()) == 20 - 8 + 3


# ---- together ------------------------------------------------------------------------------


def layer(x, rope):
    """What a layer runs of them per call, on x's tensors."""
    spg = x.spg
    x.append(rope)
    spg.latent_absorb(x.p, x.q, x.w_kv, x.q_lat)
    x.attend()
    spg.latent_project(x.p, x.o_lat, x.w_kv, x.out)


@pytest.mark.parametrize("H, r, dt", [(8, 512, "bf16"), (128, 512, "f16")])
def test_a_layer_equals_expanded_attention(spg, H, r, dt):
    """A prompt and then single tokens, against attention over the expanded keys and values in 64 bits."""
    rope = spg.make_rope(rot_dim=64, layout="interleaved")
    inv, m = R.rope_freqs(64, 1e4, "none", 1.0, 1)
    x = None
    for lens, new in (([70, 130], [70, 130]), ([71, 131], [1, 1]), ([73, 132], [2, 1])):
        c = R.Latent(H, r, 16, dt, lens, new, mp=10, extra_pages=20, seed=len(lens) + lens[0])
        if x is not None:  # the cache goes on
            c.n_phys, c.page_table, pool, w = x.c.n_phys, x.page_table.cpu(), x.pool, x.w_kv
            c.w_kv = w.cpu()
            c.pool = host(pool)
            if c.norm is not None:
                c.norm = x.c.norm
        else:
            free = iter(sorted(set(range(c.n_phys)) - set(c.page_table.flatten().tolist())))
            for b in range(2):
                for j in range(c.mp):
                    if c.page_table[b, j] < 0 and j < 9:
                        c.page_table[b, j] = next(free)
        x = Run(spg, c)
        layer(x, rope)
        assert x.err() == 0
        got, pool = host(x.out).to(R.F64), host(x.pool).to(R.F64)
        _, _, q_rot, _ = R.append(c, 64, "interleaved", inv, m, 1e-6)
        w = c.w_kv.to(R.F64)
        for b, L in enumerate(lens):
            kv = pool[c.page_table[b, : -(-L // 16)].long()].reshape(-1, r + 64)[:L]
            k = torch.cat([torch.einsum("tc,hdc->htd", kv[:, :r], w[:, : c.dn]), kv[:, r:].expand(H, L, 64)], dim=2)
            v = torch.einsum("tc,hvc->htv", kv[:, :r], w[:, c.dn :])
            lo, n = c.starts[b], new[b]
            q = torch.cat([c.q[lo : lo + n, :, : c.dn].to(R.F64), q_rot[lo : lo + n]], dim=2)
            z = torch.einsum("nhd,htd->hnt", q, k) * c.scale
            z = z.masked_fill(torch.arange(L)[None] > torch.arange(L - n, L)[:, None], -math.inf)
            p = torch.softmax(z, dim=2)
            want = torch.einsum("hnt,htv->nhv", p, v)
            # q_lat and o_lat are rounded on the way: e of each logit's terms, and e of o_lat under W_uv
            e = torch.finfo(R.DT[dt]).eps / 2
            qa = torch.einsum("nhd,hdc->nhc", q[..., : c.dn], w[:, : c.dn])
            size = (torch.einsum("nhc,tc->hnt", qa.abs(), kv[:, :r].abs()) + torch.einsum("nhd,td->hnt", q[..., c.dn :].abs(), kv[:, r:].abs())) * c.scale
            dz = 1.1 * e * size.masked_fill(z == -math.inf, 0.0).amax(dim=2)
            va = torch.einsum("hnt,tc->nhc", p, kv[:, :r].abs())
            A = torch.einsum("hnt,htv->nhv", p, v.abs())
            o = torch.einsum("hnt,tc->nhc", p, kv[:, :r]).abs()
            tol = 2 * dz.permute(1, 0)[..., None] * A + 1.1 * e * torch.einsum("nhc,hvc->nhv", o, w[:, c.dn :].abs()) + 1.1 * e * want.abs()
            tol = tol + 2.0 ** -14 * torch.einsum("nhc,hvc->nhv", va, w[:, c.dn :].abs())
            close(got[lo : lo + n], want, tol, f"out of sequence {b}")


def test_graph_replay(spg):
    c = R.Latent(16, 512, 64, "bf16", [300, 1000], [1, 4])
    x = Run(spg, c)
    rope = spg.make_rope(rot_dim=64)
    layer(x, rope)
    want, q, pool = x.out.clone(), x.q_lat.clone(), x.pool.clone()
    x.q_lat.zero_()
    x.out.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        layer(x, rope)
    for _ in range(3):
        x.o_lat.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x.out, want) and torch.equal(x.q_lat, q)
        assert torch.equal(x.pool.view(torch.int16), pool.view(torch.int16))
    assert x.err() == 0


def test_two_streams_at_once(spg):
    """Two chunks with a workspace each on two streams."""
    runs = [Run(spg, R.Latent(16, 512, 64, "bf16", [4000, 900], [1, 4], seed=1)),
            Run(spg, R.Latent(128, 256, 16, "f16", [3000], [2], seed=2))]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, s in zip(runs, streams):
            x.attend(stream=s.cuda_stream)
    torch.cuda.synchronize()
    for x in runs:
        assert x.err() == 0
        check_attend(x)


def test_one_workspace_for_different_calls(spg):
    """A workspace that is large enough serves any parameters."""
    a = Run(spg, R.Latent(64, 512, 64, "bf16", [3000, 900], [1, 4], seed=1))
    b = Run(spg, R.Latent(128, 256, 16, "f16", [2000], [2], seed=2))
    assert a.ws.numel() >= b.ws.numel()
    b.ws = a.ws
    for _ in range(2):
        for x in (a, b):
            x.o_lat.fill_(7.0)
            x.attend()
            check_attend(x)
    assert a.err() == 0


# ---- where these are easily wrong ---------------------------------------------------------------


def test_rows_with_nan_queries_stay_to_themselves(spg):
    c = R.Latent(20, 512, 16, "bf16", [900, 70], [2, 1], poison=0.0)
    c.q_lat[0, 3, 5] = math.nan
    c.q_lat[2, 19, 570] = math.nan
    x = Run(spg, c)
    x.attend()
    assert x.err() == 0
    bad = torch.zeros(3, 20, dtype=torch.bool)
    bad[0, 3] = bad[2, 19] = True
    assert torch.equal(torch.isnan(host(x.lse)), bad)
    assert bool(torch.isnan(x.o_lat[bad.cuda()]).all())
    c.q_lat = torch.nan_to_num(c.q_lat)
    out, tol, lse, lse_tol = R.attention(c)
    close(x.o_lat[(~bad).cuda()], out[~bad], tol[~bad], "o_lat")
    close(x.lse[(~bad).cuda()], lse[~bad], lse_tol[~bad], "lse")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_one_token_far_above_and_far_below_the_others(spg, dt):
    """One logit thousands above the rest (all weight on one token), and rows whose logits are all thousands below 0."""
    c = R.Latent(16, 512, 64, dt, [500, 3000], [1, 1])
    c.q_lat[:, :8] = 4.0
    for b, L in enumerate(c.lens):
        pg = c.page_table[b].long()
        c.pool[pg[300 // 64], 300 % 64] = 4.0     # 4 * 4 * 576 / 13.9: about 660 above
    c.q_lat[:, 8:] = -8.0
    for b, L in enumerate(c.lens):
        for t0 in range(0, L, 64):
            n = min(64, L - t0)
            row = c.pool[int(c.page_table[b, t0 // 64]), :n]
            row.copy_((row.float().abs() + 1.0).to(row.dtype))
    x = Run(spg, c)
    x.attend()
    assert x.err() == 0
    check_attend(x)


def test_a_logit_of_the_range_s_size(spg):
    """bf16 reaches logits of -1e36: a row's only token has all of its weight whatever its logit is."""
    c = R.Latent(4, 256, 16, "bf16", [1], [1])
    c.q_lat[:] = 1e18
    c.pool[c.page_table[0, 0].long(), 0] = -1e16
    x = Run(spg, c)
    x.attend()
    assert bool(torch.isfinite(x.lse).all()) and bool((x.lse < -1e35).all())
    assert torch.equal(x.o_lat, x.pool[x.page_table[0, 0].long(), 0, :256].expand(1, 4, 256))


def test_shared_pages(spg):
    """Sequences with a common prefix in the same physical pages."""
    c = R.Latent(32, 512, 16, "bf16", [200, 170], [2, 1])
    c.page_table[1, :8] = c.page_table[0, :8]
    x = Run(spg, c)
    x.attend()
    assert x.err() == 0
    check_attend(x)


@pytest.mark.parametrize("H, lens, new", [(1024, [90, 33], [1, 1]), (1023, [70], [2]), (65, [200, 0, 64], [3, 0, 1]), (63, [130], [5])])
def test_head_counts(spg, H, lens, new):
    x = Run(spg, R.Latent(H, 256, 32, "bf16", lens, new, pad_rows=1))
    x.attend()
    assert x.err() == 0
    check_attend(x)


@pytest.mark.parametrize("L", [63, 64, 65, 127, 128, 129, 191, 192])
@pytest.mark.parametrize("S", [16, 128])
def test_lengths_around_a_step(spg, L, S):
    x = Run(spg, R.Latent(17, 512, S, "f16", [L, L + 1, L], [1, min(L, 5), L]))
    x.attend()
    assert x.err() == 0
    check_attend(x)


def test_more_sequences_than_ctas_of_one_step(spg):
    """Items of one step each, several to a CTA, with 64 and with 128 rows an item."""
    for H in (64, 128):
        x = Run(spg, R.Latent(H, 256, 16, "f16", [1 + i % 60 for i in range(330)], [1] * 330))
        x.attend()
        assert x.err() == 0
        check_attend(x)


def test_calls_in_a_row_on_one_stream(spg):
    """A layer's four calls back to back many times over, each launch free to start while the one before ends."""
    c = R.Latent(16, 512, 64, "bf16", [700, 130], [1, 3])
    x, rope = Run(spg, c), spg.make_rope(rot_dim=64)
    layer(x, rope)
    want = [t.clone() for t in (x.out, x.o_lat, x.lse, x.q_lat)]
    for _ in range(50):
        layer(x, rope)
    for a, b in zip((x.out, x.o_lat, x.lse, x.q_lat), want):
        assert torch.equal(a, b)
    assert x.err() == 0


def test_calls_from_a_side_stream(spg):
    """The binding takes the current stream: work queued on it comes first."""
    c = R.Latent(16, 512, 64, "bf16", [700, 130], [1, 3])
    x = Run(spg, c)
    s = torch.cuda.Stream()
    q = x.q_lat.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x.q_lat.zero_()
        torch.cuda._sleep(2_000_000)
        x.q_lat.copy_(q)
        x.attend()
    s.synchronize()
    check_attend(x)


def test_two_graphs_share_a_workspace(spg):
    """Two captured calls of different sizes on one workspace, replayed in turn."""
    a = Run(spg, R.Latent(64, 512, 64, "bf16", [3000, 900], [1, 4], seed=1))
    b = Run(spg, R.Latent(128, 256, 16, "f16", [2000], [2], seed=2))
    b.ws = a.ws
    for x in (a, b):
        x.attend()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            x.attend()
        graphs.append(g)
    for _ in range(3):
        for x, g in zip((a, b), graphs):
            x.o_lat.fill_(7.0)
            g.replay()
    torch.cuda.synchronize()
    for x in (a, b):
        check_attend(x)
    assert a.err() == 0


def test_append_of_many_rows_in_ragged_sequences(spg):
    """Rows of 40 sequences, empty ones among them, found by every CTA for itself."""
    g = torch.Generator().manual_seed(3)
    lens = [int(v) for v in torch.randint(0, 90, (40,), generator=g)]
    new = [min(L, int(v)) for L, v in zip(lens, torch.randint(0, 30, (40,), generator=g))]
    c = R.Latent(5, 256, 16, "bf16", lens, new, pad_rows=3)
    x = Run(spg, c)
    x.append(None, norm=False)
    assert x.err() == 0
    pool = host(x.pool)
    for b, L in enumerate(lens):
        for i in range(new[b]):
            t = L - new[b] + i
            assert torch.equal(pool[int(c.page_table[b, t // 16]), t % 16], c.kv[c.starts[b] + i])
