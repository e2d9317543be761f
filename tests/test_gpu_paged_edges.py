"""The paged-chunk operators where they are easily wrong.  References in 64 bits, as in tests/paged_ref.py."""
import decimal
import math

import pytest
import torch

import paged_ref as R
from test_gpu_paged import RAGGED, SHAPES, Run, check_chunk, close, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spg():
    import query_aware_sparse_page_gb300 as m

    return m


# ---- chunk attention: weights over a wide range ------------------------------------------------


def sink_chunk(kv, q, gap, scales, new=3, L=32768, S=64, hq=2, hkv=1, d=128, seed=0):
    """Token 0 of each sequence `gap` nats above the others, whose logits lie within 0.1 of one another and whose values
    have one sign, so that weight lost from them shows."""
    c = R.Chunk(hq, hkv, d, S, kv, q, [L], [new], seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    a = 8.0
    c.q = (0.05 * torch.randn(c.q.shape, generator=g)).to(c.q.dtype)
    c.q[..., 0] = a
    first = int(c.page_table[0, 0])
    key = gap * math.sqrt(d) / a
    live = torch.zeros((c.n_phys, S), dtype=torch.bool)
    for t0 in range(0, L, S):
        live[int(c.page_table[0, t0 // S]), : min(S, L - t0)] = True
    live = live[:, None].expand(c.n_phys, hkv, S)
    if kv == "i8":
        c.k_pool[..., 0][live] = 0
        c.k_pool[first, :, 0] = 0
        c.k_pool[first, :, 0, 0] = 127
        c.k_scale[live] = 0.005
        c.k_scale[first, :, 0] = key / 127
        c.v_pool[live] = c.v_pool[live].abs().clamp(min=1)
        c.v_scale[live] = scales(live.sum(), g).half()
    else:
        c.k_pool[..., 0][live] = 0
        c.k_pool[first, :, 0] = 0
        c.k_pool[first, :, 0, 0] = key
        c.v_pool[live] = c.v_pool[live].abs()
    return c, first


def wide_tolerance(c):
    """out and its tolerance, relative to what the row holds (terms as in paged_ref.attention): the weights that enter
    the products are rounded to 16 bits, half a step each; in fp16 they are scaled so that the largest of a row is at
    least 2^7 in units whose subnormal half step is 2^-25, that is 2^-32 of the largest weight times value scale."""
    out, tol = torch.zeros((c.T, c.hq, c.d), dtype=R.F64), torch.zeros((c.T, c.hq, c.d), dtype=R.F64)
    e = torch.finfo(R.DT[c.qdt]).eps / 2
    for h in range(c.hkv):
        v = c.tokens(c.v_pool, c.v_scale, 0, h)
        code = v if c.kv != "i8" else c.tokens(c.v_pool, None, 0, h)
        page = c.page_table[0, : -(-c.lens[0] // c.S)].long()
        vs = torch.ones(c.lens[0], dtype=R.F64) if c.kv != "i8" else c.v_scale[page, h].to(R.F64).reshape(-1)[: c.lens[0]]
        for j in range(c.group):
            z, size = c.logits(0, h, j)
            i = h * c.group + j
            p = torch.softmax(z, dim=1)
            o, A = p @ v, p @ v.abs()
            zmax = z.masked_fill(~torch.isfinite(z), 0.0).abs().amax(dim=1)
            dz = c.d * 2.0 ** -24 * size.amax(dim=1) + 8 * 2.0 ** -24 * (zmax + 1)
            t = e * (A + o.abs()) + 2 * dz[:, None] * A
            if c.qdt == "f16":
                t = t + 2.0 ** -32 * (p * vs).amax(dim=1)[:, None] * code.abs().sum(dim=0)[None] + 2.0 ** -25
            out[:, i], tol[:, i] = o, 1.01 * t
    return out, tol


SCALES = {
    "1e-7": lambda n, g: torch.full((n,), 1e-7),
    "1e-5": lambda n, g: 1e-5 * (0.5 + torch.rand(n, generator=g)),
    "1e-4": lambda n, g: 1e-4 * (0.5 + torch.rand(n, generator=g)),
    "1e-2": lambda n, g: 1e-2 * (0.5 + torch.rand(n, generator=g)),
    "400": lambda n, g: 400.0 * (0.5 + torch.rand(n, generator=g)),
    "all": lambda n, g: torch.exp2(-20 + 24 * torch.rand(n, generator=g)),
}


@pytest.mark.parametrize("q", ["f16", "bf16"])
@pytest.mark.parametrize("gap", [0.0, 8.0, 12.0])
@pytest.mark.parametrize("scales", list(SCALES))
def test_chunk_int8_value_scales(spg, scales, gap, q):
    c, _ = sink_chunk("i8", q, gap, SCALES[scales])
    r = Run(spg, c)
    r.chunk()
    assert r.err() == 0
    out, tol = wide_tolerance(c)
    close(r.out, out, tol, "out")


@pytest.mark.parametrize("new, hq", [(3, 2), (200, 2), (1, 8)])
def test_chunk_int8_scales_that_differ(spg, new, hq):
    """A first token with the smallest scale there is, or none, before values of an ordinary size; and the other way
    round.  In a short prompt too, whose rows see few tokens."""
    for first_scale, rest in ((2.0 ** -24, 0.02), (0.0, 0.02), (0.02, 2.0 ** -20), (60000.0, 1e-4)):
        for L in (5000, max(new, 40)):
            c, first = sink_chunk("i8", "f16", 12.0, lambda n, g: torch.full((n,), rest), new=new, L=L, hq=hq, d=64)
            c.v_pool.clamp_(max=16)  # 60000 * 16 is past fp16, and what the first token leaves of it is not
            c.v_scale[first, :, 0] = first_scale
            if first_scale > 1:
                c.v_pool[first, :, 0] = 1
            r = Run(spg, c)
            r.chunk()
            assert r.err() == 0
            out, tol = wide_tolerance(c)
            close(r.out, out, tol, "out")


@pytest.mark.parametrize("scale", [100.0, 300.0, 500.0])
@pytest.mark.parametrize("odd", [0, 1])
def test_chunk_int8_large_scales_rising_logits(spg, scale, odd):
    """Logits that rise by less than the running maximum's slack, over values close to fp16's range."""
    c, _ = sink_chunk("i8", "f16", 0.0, lambda n, g: torch.full((n,), scale), new=50, L=6000, hq=4)
    pages = c.page_table[0].long()
    for t in range(6000):
        if t // 128 % 2 == odd:  # 2.4 nats above its neighbours
            pg = pages[t // 64]
            c.k_pool[pg, :, t % 64, 0] = 127
            c.k_scale[pg, :, t % 64] = 2.4 * math.sqrt(128) / 8.0 / 127
            c.k_pool[pg, :, t % 64, 1:] = (c.k_pool[pg, :, t % 64, 1:].float() * 0.18).to(torch.int8)
    r = Run(spg, c)
    r.chunk()
    assert r.err() == 0
    out, tol = wide_tolerance(c)
    close(r.out, out, tol, "out")


@pytest.mark.parametrize("gap", [8.0, 12.0, 14.0])
@pytest.mark.parametrize("kv", ["f16", "bf16"])
def test_chunk_one_token_above_a_long_cache(spg, kv, gap):
    c, _ = sink_chunk(kv, kv, gap, None, L=40000, S=16)
    r = Run(spg, c)
    r.chunk()
    assert r.err() == 0
    out, tol = wide_tolerance(c)
    close(r.out, out, tol, "out")


# ---- chunk attention: the parts of a weight -------------------------------------------------------


@pytest.fixture
def one_part(spg):
    spg.spg_set_chunk_parts(1)
    yield
    spg.spg_set_chunk_parts(2)


def equal_tail(kv, q, gap, new, hq, d):
    """One token `gap` above 499 of exactly equal logits: every weight of the tail is rounded in the same direction."""
    c, first = sink_chunk(kv, q, gap, lambda n, g: torch.full((n,), 0.01), new=new, L=500, S=16, hq=hq, d=d)
    c.q[..., 1:] = 0
    return c


@pytest.mark.parametrize("new, hq, d", [(1, 2, 128), (3, 8, 64), (140, 2, 128)])
@pytest.mark.parametrize("kv, q", [("f16", "f16"), ("bf16", "bf16"), ("i8", "f16"), ("i8", "bf16")])
def test_chunk_weights_are_not_rounded_to_16_bits(spg, kv, q, new, hq, d):
    """Off by the output's rounding e |o|, that of a weight's second part e e A, and sums of L terms in 32 bits."""
    e = torch.finfo(R.DT[q]).eps / 2
    for gap in (1.7, 1.9, 2.0, 2.1, 2.2, 2.35):
        c = equal_tail(kv, q, gap, new, hq, d)
        r = Run(spg, c)
        r.chunk()
        assert r.err() == 0
        out = wide_tolerance(c)[0]
        _, size = c.logits(0, 0, 0)
        dz = float(d * 2.0 ** -24 * size.max() + 8 * 2.0 ** -24 * 4)
        v = c.tokens(c.v_pool, c.v_scale, 0, 0)
        assert bool((v >= 0).all())  # A = o
        tol = (e + e * e + 2 * dz + 2 * 500 * 2.0 ** -24) * out.abs() + (2.0 ** -25 if q == "f16" else 0.0)
        close(r.out, out, tol, f"out at {gap}")


@pytest.mark.parametrize("lens, new, pad", RAGGED)
@pytest.mark.parametrize("hq, hkv, d, S, kv, q", SHAPES)
def test_chunk_attention_with_one_part(spg, one_part, hq, hkv, d, S, kv, q, lens, new, pad):
    r = Run(spg, R.Chunk(hq, hkv, d, S, kv, q, lens, new, pad_rows=pad))
    r.chunk()
    assert r.err() == 0
    check_chunk(r)


@pytest.mark.parametrize("q", ["f16", "bf16"])
@pytest.mark.parametrize("gap", [0.0, 12.0])
@pytest.mark.parametrize("scales", list(SCALES))
def test_chunk_int8_value_scales_with_one_part(spg, one_part, scales, gap, q):
    test_chunk_int8_value_scales(spg, scales, gap, q)


def test_chunk_nan_rows_with_one_part(spg, one_part):
    test_chunk_nan_rows(spg, "f16")


# ---- rows that hold a NaN ------------------------------------------------------------------------


@pytest.mark.parametrize("kv", ["f16", "bf16", "i8"])
def test_chunk_nan_rows(spg, kv):
    """A NaN in a row's query makes that row NaN, whether one CTA has its whole work or many share it, and no other."""
    c = R.Chunk(4, 2, 64, 16, kv, "bf16" if kv == "bf16" else "f16", [40, 5000, 700], [40, 3, 300])
    r = Run(spg, c)
    rows = [(5, 1), (41, 2), (43, 0), (342, 3)]
    clean = r.q.clone()
    for t, h in rows:
        r.q[t, h, 7] = math.nan
    r.chunk()
    assert r.err() == 0
    for t, h in rows:
        assert bool(torch.isnan(r.out[t, h]).all()) and bool(torch.isnan(r.lse[t, h])), (t, h)
    out, lse = r.out.clone(), r.lse.clone()
    r.q = clean
    r.chunk()
    for t, h in rows:
        out[t, h], lse[t, h] = r.out[t, h], r.lse[t, h]
    assert torch.equal(out, r.out) and torch.equal(lse, r.lse)
    check_chunk(r)


@pytest.mark.parametrize("hq, hkv, d, kv, q, lens, new", [
    (4, 2, 64, "f16", "f16", [300, 40], [5, 40]), (8, 2, 128, "bf16", "bf16", [2000], [300]),
    (4, 2, 128, "i8", "f16", [300, 40], [9, 1]),
    (4, 2, 64, "f16", "f16", [300, 40], [2, 1]), (4, 2, 128, "i8", "f16", [300, 40], [1, 2]),
])
def test_mass_rows_without_lse_add_nothing(spg, hq, hkv, d, kv, q, lens, new):
    """Rows taken out by lse = -inf add nothing whatever their queries hold."""
    c = R.Chunk(hq, hkv, d, 16, kv, q, lens, new)
    lse = R.attention(c)[2].float()
    gone = [0, c.T - 1]
    lse[gone] = -math.inf
    want, tol = R.mass_of(c, lse, None, 1.0)
    r = Run(spg, c)
    r.q[gone[0]] = math.nan
    r.q[gone[1], :, ::2] = math.inf
    m = torch.full((len(lens), hkv, c.mp * 16), 3.0, device="cuda")
    r.mass(dev(lse), None, m, 1.0)
    assert r.err() == 0
    for b, L in enumerate(lens):
        close(m[b, :, :L], want[b, :, :L], tol[b, :, :L], "mass")


# ---- one workspace ------------------------------------------------------------------------------


def test_one_workspace_under_several_selectors(spg):
    """Chunks, masses and decode steps take turns on one workspace with parameters that differ in the selector alone."""
    c = R.Chunk(8, 2, 128, 16, "bf16", "bf16", [3000, 2001], [300, 200])
    r = Run(spg, c)
    ps = [r.p] + [c.params(spg, selector="quest", token_budget=16 * n, n_sink_pages=1, n_recent_pages=1) for n in (8, 64, 180)]
    r.ws = torch.zeros(max(spg.spg_chunk_workspace_size(p, c.T) for p in ps), dtype=torch.uint8, device="cuda")
    mass = torch.zeros((2, 2, c.mp * 16), device="cuda")

    def chunk(p):
        r.p = p
        r.out.fill_(7.0), r.lse.fill_(7.0), mass.fill_(7.0)
        r.chunk()
        r.mass(r.lse, None, mass, 1.0)
        assert r.err() == 0
        return [t.clone() for t in (r.out, r.lse, mass)]

    want = chunk(ps[0])
    check_chunk(r)
    dq = torch.randn((2, 8, 128), device="cuda").bfloat16()
    steps = {}
    spg.spg_set_step_kernel(spg.STEP_KERNEL_SCHED)
    try:
        for i in (1, 0, 2, 3, 1, 0, 3):
            if i:
                buf = spg.alloc_buffers(ps[i])
                spg.sparse_page_meta_update(ps[i], r.k_pool, None, r.page_table, r.seq_lens, 1, buf.minmax, None, None, None,
                                            r.ws)
                spg.sparse_decode_select_attend(ps[i], dq, r.k_pool, r.v_pool, None, None, r.page_table, r.seq_lens,
                                                buf.minmax, None, None, None, buf.sel, buf.sel_cnt, buf.out, buf.lse, r.ws)
                assert r.err() == 0
                first = steps.setdefault(i, (buf.out.clone(), buf.sel.clone()))
                assert torch.equal(first[0], buf.out) and torch.equal(first[1], buf.sel)
            for p in (ps[0], ps[i]):
                for a, b in zip(chunk(p), want):
                    assert torch.equal(a, b)
    finally:
        spg.spg_set_step_kernel(spg.STEP_KERNEL_AUTO)


# ---- rotary append ------------------------------------------------------------------------------


@pytest.mark.parametrize("q", ["f16", "bf16"])
@pytest.mark.parametrize("d, S", [(64, 16), (128, 64)])
def test_append_int8_codes_are_those_of_the_quotient(spg, d, S, q):
    """code = rint(x / s) of the quotient in 32 bits, ties to the even code: rows whose values lie exactly between two
    codes, and random ones."""
    c = R.Chunk(8, 8, d, S, "i8", q, [700, 300], [700, 300])
    bits = 11 if q == "f16" else 8
    t = 0
    for m in (1, 3, 5, 7, 9, 11, 13, 15):  # s = m 2^-9, exactly
        odd = [k for k in range(1, 254, 2) if k * m < 1 << bits]
        if 127 * m >= 1 << bits:
            continue
        for i in range(0, len(odd), d - 1):
            for sign in (1, -1):
                row = torch.zeros(d, dtype=R.F64)
                row[0] = 127 * m * 2.0 ** -9
                part = odd[i : i + d - 1]
                row[1 : 1 + len(part)] = sign * torch.tensor(part, dtype=R.F64) * m * 2.0 ** -10
                for x in (c.k, c.v):
                    x[t, t % 8] = row.to(x.dtype)
                assert torch.equal(c.k[t, t % 8].to(R.F64), row)
                t += 1
    r = Run(spg, c)
    r.append(None, torch.empty_like(r.q))
    assert r.err() == 0
    pos = torch.cat([torch.arange(700), torch.arange(300)])
    owner = torch.cat([torch.zeros(700), torch.ones(300)]).long()
    phys, slot = c.page_table[owner, pos // S].long(), pos % S
    for x, pool, scale in ((c.k, r.k_pool, r.k_scale), (c.v, r.v_pool, r.v_scale)):
        s = (x.float().abs().amax(dim=-1) / 127.0).half()
        s = torch.where(s > 0, s, torch.ones_like(s))
        code = torch.round(x.float() / s.float()[..., None]).clamp(-127, 127).to(torch.int8)
        assert torch.equal(host(scale)[phys, :, slot], s)
        assert torch.equal(host(pool)[phys, :, slot], code)


def exact_turns(rot, base, positions):
    """Angles [n][rot / 2] in radians within one turn, from 60 digits."""
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        two_pi = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
        f = [(decimal.Decimal(base).ln() * -2 * i / rot).exp() / two_pi for i in range(rot // 2)]
        return torch.tensor([[float((p * x) % 1 * two_pi) for x in f] for p in positions], dtype=R.F64)


@pytest.mark.parametrize("base", [10000, 500000])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_append_positions_to_the_end_of_32_bits(spg, layout, base):
    """The rotation at any position: the angle is off by at most 2^-26 of a turn (its 32-bit form) and t 2^-54 (the
    frequency's 64-bit form), with rotate_tol's other terms."""
    c = R.Chunk(2, 1, 128, 16, "f16", "f16", [64], [64])
    pos = [0, 1, 2, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, 2 ** 31 - 2] + [
        int(x) for x in torch.randint(0, 2 ** 31 - 1, (57,), generator=torch.Generator().manual_seed(3))]
    c.q[:] = torch.where(c.q.abs() < 2 ** -3, torch.full_like(c.q, 0.5), c.q)
    r = Run(spg, c)
    out = torch.empty_like(r.q)
    r.append(spg.make_rope(layout=layout, base=float(base)), out, torch.tensor(pos, dtype=torch.int32, device="cuda"))
    assert r.err() == 0
    ang = exact_turns(128, base, pos)[:, None]
    x = c.q.to(R.F64)
    one = slice(0, 64) if layout == "half" else slice(0, 128, 2)
    two = slice(64, 128) if layout == "half" else slice(1, 128, 2)
    want = torch.empty_like(x)
    want[..., one] = x[..., one] * torch.cos(ang) - x[..., two] * torch.sin(ang)
    want[..., two] = x[..., two] * torch.cos(ang) + x[..., one] * torch.sin(ang)
    far = torch.tensor(pos, dtype=R.F64)[:, None, None] * 2.0 ** -54 * 2 * math.pi
    pair = (x[..., one].abs() + x[..., two].abs()) * far
    tol = R.rotate_tol(c.q, 128, layout, 1.0)
    tol[..., one] += pair
    tol[..., two] += pair
    e = 2.0 ** -11
    close(out, want, e * want.abs() + (1 + e) * tol + 2.0 ** -25, "q")


# ---- eviction: sizes --------------------------------------------------------------------------------


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_more_units_than_a_grid_dimension(spg, in_place):
    """batch * kv-heads past 65535."""
    B, H, S, L, keep = 8200, 8, 16, 13, 5
    p = spg.make_params(batch=B, num_q_heads=H, num_kv_heads=H, head_dim=64, page_size=S, num_phys_pages=2 * B,
                        max_pages_per_seq=1, kv_dtype="i8", q_dtype="f16", selector="all")
    ws = torch.zeros(spg.spg_workspace_size(p), dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    pool = lambda: torch.randint(-127, 128, (2 * B, H, S, 64), generator=g, device="cuda").to(torch.int8)  # noqa: E731
    scale = lambda: torch.rand((2 * B, H, S), generator=g, device="cuda").half()  # noqa: E731
    k, v, ks, vs = pool(), pool(), scale(), scale()
    perm = torch.randperm(2 * B, generator=g, device="cuda").int()
    pt, dst = perm[:B].view(B, 1).contiguous(), perm[B:].view(B, 1).contiguous()
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    mass = torch.rand((B, H, S), generator=g, device="cuda")
    kept = torch.empty((B, H, keep), dtype=torch.int32, device="cuda")
    nl = torch.empty(B, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(mass)
    order = mass[..., :L].clone()
    order[..., L - 1] = math.inf  # the last token stays
    ids = order.topk(keep, dim=-1).indices.sort(dim=-1).values
    table = pt if in_place else dst
    want = [x[pt[:, 0].long()].gather(2, ids[..., None].expand(-1, -1, -1, 64) if x.dim() == 4 else ids) for x in (k, v, ks, vs)]
    spg.paged_cache_evict(p, mass, keep, 0, 1, k, v, ks, vs, pt, None if in_place else dst, lens, kept, nl, out, ws)
    assert spg.spg_read_device_error(ws) == 0
    assert torch.equal(kept.long(), ids) and bool((nl == keep).all())
    assert torch.equal(out[..., :keep], mass.gather(2, ids)) and bool((out[..., keep:] == 0).all())
    for x, w in zip((k, v, ks, vs), want):
        assert torch.equal(x[table[:, 0].long()][:, :, :keep], w)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("masses", ["lognormal", "three"])
def test_evict_lengths_past_shared_memory(spg, masses, in_place):
    """A sequence of more tokens than a cluster's shared memory holds masses of, beside a short one."""
    N, S = 400000, 64
    g = torch.Generator().manual_seed(4)
    m = torch.exp(2 * torch.randn((2, 1, N), generator=g)) if masses == "lognormal" else torch.randint(0, 3, (2, 1, N), generator=g).float()
    lens = [N - 7, 500]
    p = spg.make_params(batch=2, num_q_heads=1, num_kv_heads=1, head_dim=64, page_size=S, num_phys_pages=2 * (N // S),
                        max_pages_per_seq=N // S, kv_dtype="i8", q_dtype="f16", selector="all")
    ws = torch.zeros(spg.spg_workspace_size(p), dtype=torch.uint8, device="cuda")
    for keep in (390000, 20000):
        pages = torch.randperm(2 * (N // S), generator=g).int()
        pt = pages.view(2, -1).cuda()
        k = torch.randint(-127, 128, (2 * (N // S), 1, S, 64), generator=g).to(torch.int8).cuda()
        ks = torch.rand((2 * (N // S), 1, S), generator=g).half().cuda()
        k0, ks0 = k.clone(), ks.clone()
        mass = m.cuda()
        out = mass if in_place else torch.full_like(mass, 5.0)
        kept = torch.empty((2, 1, keep), dtype=torch.int32, device="cuda")
        nl = torch.empty(2, dtype=torch.int32, device="cuda")
        spg.paged_cache_evict(p, mass, keep, 4, 100, k, k.clone(), ks, ks.clone(), pt, None,
                              torch.tensor(lens, dtype=torch.int32, device="cuda"), kept, nl, out, ws)
        assert spg.spg_read_device_error(ws) == 0
        assert host(nl).tolist() == [min(L, keep) for L in lens]
        for b, L in enumerate(lens):
            w = m[b, 0, :L].double()
            w[:4] = math.inf
            w[L - 100 :] = math.inf
            n = min(L, keep)
            ids = torch.sort(w, descending=True, stable=True).indices[:n].sort().values
            assert torch.equal(host(kept)[b, 0, :n].long(), ids) and bool((kept[b, 0, n:] == -1).all())
            assert torch.equal(host(out)[b, 0, :n], m[b, 0, ids])
            assert torch.equal(host(out)[b, 0, n:], m[b, 0, n:] if in_place else torch.full((N - n,), 5.0))
            j, t = torch.arange(n, device="cuda"), ids.cuda()
            row = pt[b].long()
            assert torch.equal(k[row[j // S], 0, j % S], k0[row[t // S], 0, t % S])
            assert torch.equal(ks[row[j // S], 0, j % S], ks0[row[t // S], 0, t % S])


# ---- uneven batches -------------------------------------------------------------------------------


@pytest.mark.parametrize("hq, hkv, d, S, kv, q", [(8, 2, 128, 16, "bf16", "bf16"), (8, 1, 64, 32, "f16", "f16"),
                                                  (4, 2, 128, 64, "i8", "f16"), (4, 2, 128, 64, "bf16", "bf16")])
@pytest.mark.parametrize("at", [0, 17, 39])
@pytest.mark.parametrize("rows", [40, 64])
def test_mass_of_a_batch_with_one_piece(spg, hq, hkv, d, S, kv, q, rows, at):
    """One sequence with nearly all the rows of a batch, whose others have one row or none."""
    B = 40
    g = torch.Generator().manual_seed(at)
    lens = torch.randint(1, 500, (B,), generator=g).tolist()
    lens[at] = 900
    new = [b % 3 == 0 for b in range(B)]
    new = [int(x) for x in new]
    new[at] = rows - sum(new)
    c = R.Chunk(hq, hkv, d, S, kv, q, lens, new)
    r = Run(spg, c)
    lse = R.attention(c)[2].float()
    old = torch.rand((B, hkv, c.mp * S), generator=g)
    want, tol = R.mass_of(c, lse, old, 0.5)
    for _ in range(2):
        m = torch.full(old.shape, 3.0, device="cuda")
        r.mass(dev(lse), dev(old), m, 0.5)
        assert r.err() == 0
        for b, L in enumerate(lens):
            close(m[b, :, :L], want[b, :, :L], tol[b, :, :L], "mass")
            assert bool((m[b, :, L:] == 3.0).all())
