"""The paged-chunk entry points on the host: frequencies, workspace sizes, and every refusal, without a GPU."""

import ctypes
import math

import pytest
import torch

import paged_ref as R


@pytest.fixture(scope="module")
def spg():
    import __graft_entry__

    __graft_entry__.build()
    import query_aware_sparse_page_gb300 as m

    return m


def _p(spg, **kw):
    a = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_phys_pages=100,
             max_pages_per_seq=64, kv_dtype="f16", selector="all")
    a.update(kw)
    return spg.make_params(**a)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot, base, factor, orig", [(128, 1e4, 4.0, 2048), (64, 5e5, 8.0, 4096), (16, 1e4, 1.0, 1),
                                                      (32, 1e6, 2.5, 8192)])
def test_rope_freqs(spg, scaling, rot, base, factor, orig):
    r = spg.make_rope(rot_dim=rot, base=base, scaling=scaling, factor=factor, orig_len=orig)
    got, m = spg.spg_rope_freqs(r, 128)
    want, wm = R.rope_freqs(rot, base, scaling, factor, orig)
    assert m == pytest.approx(wm, rel=1e-14)
    assert got == pytest.approx(want, rel=1e-13)
    assert len(got) == rot // 2


def test_rope_yarn_between_plain_and_linear(spg):
    f = lambda s: spg.spg_rope_freqs(spg.make_rope(base=1e4, scaling=s, factor=8.0, orig_len=4096), 128)[0]  # noqa: E731
    plain, lin, yarn = f("none"), f("linear"), f("yarn")
    assert yarn[0] == plain[0] and yarn[-1] == pytest.approx(lin[-1], rel=1e-15)
    assert all(a <= y * (1 + 1e-15) and y <= b * (1 + 1e-15) for a, y, b in zip(lin, yarn, plain))
    assert spg.spg_rope_freqs(spg.make_rope(), 64)[0][0] == 1.0  # rot_dim 0: the whole head


@pytest.mark.parametrize("kw", [dict(rot_dim=130), dict(rot_dim=7), dict(rot_dim=-2), dict(layout=2), dict(scaling=4),
                                dict(base=1.0), dict(base=math.inf), dict(base=math.nan),
                                dict(scaling="linear", factor=0.5), dict(scaling="yarn", factor=math.nan),
                                dict(scaling="yarn", factor=2.0, orig_len=0), dict(scaling="ntk", rot_dim=2)])
def test_rope_freqs_refuses(spg, kw):
    with pytest.raises(spg.SpgError):
        spg.spg_rope_freqs(spg.make_rope(**kw), 128)


def test_chunk_workspace(spg):
    p = _p(spg)
    base = spg.spg_workspace_size(p)
    sizes = [spg.spg_chunk_workspace_size(p, t) for t in (0, 1, 100, 10000)]
    assert base <= sizes[0] and sizes == sorted(sizes)
    with pytest.raises(spg.SpgError):
        spg.spg_chunk_workspace_size(p, -1)
    with pytest.raises(spg.SpgError):
        spg.spg_chunk_workspace_size(_p(spg, head_dim=48), 1)


A = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: every call below is refused before a launch
ODD = ctypes.c_void_p((1 << 20) + 8)
WS = ctypes.c_size_t(1 << 40)


def _chunk(spg, p, total=4, q=A, st=A, k=A, v=A, ks=None, vs=None, pt=A, sl=A, out=A, lse=None, ws=A, wn=WS):
    return spg.LIB.paged_chunk_attention(ctypes.byref(p), total, q, st, k, v, ks, vs, pt, sl, out, lse, ws, wn, None)


@pytest.mark.parametrize("kw, status", [
    (dict(total=-1), 1), (dict(q=None), 1), (dict(q=ODD), 1), (dict(st=None), 1), (dict(k=None), 1), (dict(v=ODD), 1),
    (dict(pt=None), 1), (dict(sl=None), 1), (dict(out=None), 1), (dict(lse=ODD), 1), (dict(ws=None), 1),
    (dict(wn=ctypes.c_size_t(16)), 4), (dict(total=0, q=None, out=None), 0),
])
def test_chunk_refusals(spg, kw, status):
    assert _chunk(spg, _p(spg), **kw) == status


def test_chunk_refuses_params(spg):
    assert _chunk(spg, _p(spg, head_dim=96)) == 2
    assert _chunk(spg, _p(spg, num_q_heads=6)) == 2
    assert _chunk(spg, _p(spg, kv_dtype="i8")) == 1  # no scales
    assert _chunk(spg, _p(spg, kv_dtype="i8"), ks=A) == 1


def _rope(spg, p, rope="default", total=4, q=A, qs=1024, k=A, ks=256, v=A, vs=256, st=A, pos=None, pt=A, sl=A, kp=A,
          vp=A, ksc=None, vsc=None, out=A, ws=A, wn=WS):
    r = spg.make_rope() if rope == "default" else rope
    return spg.LIB.paged_rope_append(ctypes.byref(p), None if r is None else ctypes.byref(r), total, q, qs, k, ks, v, vs,
                                     st, pos, pt, sl, kp, vp, ksc, vsc, out, ws, wn, None)


@pytest.mark.parametrize("kw, status", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(q=ODD), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(qs=1020), 1),
    (dict(qs=512), 1), (dict(ks=128), 1), (dict(vs=260), 1), (dict(qs=2048, k=A), 1), (dict(pos=ODD), 1),
    (dict(st=None), 1), (dict(kp=None), 1), (dict(vp=ODD), 1), (dict(total=-3), 1), (dict(ws=ODD), 1),
    (dict(wn=ctypes.c_size_t(8)), 4), (dict(total=0, k=None), 0),
])
def test_rope_refusals(spg, kw, status):
    # qs=2048 with q_out == q: rows of q that are not where q_out's are
    assert _rope(spg, _p(spg), **kw) == status


def test_rope_refuses_rope(spg):
    p = _p(spg)
    assert _rope(spg, p, spg.make_rope(rot_dim=24)) == 2  # valid, not built
    assert _rope(spg, p, spg.make_rope(rot_dim=256)) == 1
    assert _rope(spg, p, spg.make_rope(base=0.5)) == 1
    assert _rope(spg, _p(spg, kv_dtype="i8"), ksc=A) == 1


def _mass(spg, p, total=4, q=A, st=A, k=A, ks=None, pt=A, sl=A, lse=A, mi=A, mo=A, decay=1.0, ws=A, wn=WS):
    return spg.LIB.paged_attention_mass(ctypes.byref(p), total, q, st, k, ks, pt, sl, lse, mi, mo, decay, ws, wn, None)


@pytest.mark.parametrize("kw, status", [
    (dict(q=None), 1), (dict(lse=None), 1), (dict(mo=None), 1), (dict(mi=ODD), 1), (dict(decay=-0.1), 1),
    (dict(decay=1.5), 1), (dict(decay=math.nan), 1), (dict(k=None), 1), (dict(pt=ODD), 1), (dict(total=-1), 1),
    (dict(ws=None), 1), (dict(wn=ctypes.c_size_t(8)), 4),
])
def test_mass_refusals(spg, kw, status):
    assert _mass(spg, _p(spg), **kw) == status
    assert _mass(spg, _p(spg, kv_dtype="i8")) == 1


B2 = ctypes.c_void_p(1 << 21)


def _evict(spg, p, mass=A, keep=64, sink=4, recent=16, k=A, v=A, ks=None, vs=None, pt=A, dst=None, sl=A, kept=A, nl=B2,
           mo=A, ws=A, wn=WS):
    return spg.LIB.paged_cache_evict(ctypes.byref(p), mass, keep, sink, recent, k, v, ks, vs, pt, dst, sl, kept, nl, mo,
                                     ws, wn, None)


@pytest.mark.parametrize("kw, status", [
    (dict(mass=None), 1), (dict(keep=0), 1), (dict(sink=-1), 1), (dict(recent=-1), 1), (dict(sink=40, recent=40), 1),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), 1), (dict(k=None), 1), (dict(v=ODD), 1), (dict(dst=ODD), 1),
    (dict(nl=A), 1), (dict(nl=None), 1), (dict(kept=None), 1), (dict(mo=None), 1), (dict(ws=None), 1),
    (dict(wn=ctypes.c_size_t(8)), 4),
])
def test_evict_refusals(spg, kw, status):
    # nl=A: new_lens may not be seq_lens
    assert _evict(spg, _p(spg), **kw) == status
    assert _evict(spg, _p(spg, kv_dtype="i8"), ks=A) == 1


def test_binding_refuses_shapes_types_and_host_tensors(spg):
    p = _p(spg)
    z = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt)  # noqa: E731
    pool, st, pt, sl = z(100, 2, 16, 128), z(3, dt=torch.int32), z(2, 64, dt=torch.int32), z(2, dt=torch.int32)
    ws = z(1, dt=torch.uint8)
    with pytest.raises(ValueError, match="shape"):
        spg.paged_chunk_attention(p, z(4, 8, 64), st, pool, pool, None, None, pt, sl, z(4, 8, 64), ws=ws)
    with pytest.raises(ValueError):  # host tensors
        spg.paged_chunk_attention(p, z(4, 8, 128), st, pool, pool, None, None, pt, sl, z(4, 8, 128), ws=ws)
    with pytest.raises(ValueError, match="expected torch.float16"):
        spg.paged_rope_append(p, None, None, z(4, 2, 128, dt=torch.float32), z(4, 2, 128), st, pt, sl, pool, pool, ws=ws)
    with pytest.raises(ValueError, match="shape"):
        spg.paged_attention_mass(p, z(4, 2, 128), st, pool, None, pt, sl, z(4, 8, dt=torch.float32), None, z(2, 2, 64),
                                 1.0, ws)


def test_reference_forms_agree_with_a_library_routine():
    """The tests' own 64-bit forms: attention and mass against torch's attention, rotation against complex products."""
    c = R.Chunk(4, 2, 64, 16, "f16", "f16", [37, 5], [9, 5], seed=3, poison=0.0)
    out, _, lse, _ = R.attention(c)
    mass, _ = R.mass_of(c, lse, None, 1.0)
    for b, L in enumerate(c.lens):
        lo, hi = c.starts[b], c.starts[b + 1]
        q = c.q[lo:hi].to(R.F64).transpose(0, 1)
        k = torch.stack([c.tokens(c.k_pool, None, b, h // 2) for h in range(4)])
        v = torch.stack([c.tokens(c.v_pool, None, b, h // 2) for h in range(4)])
        see = torch.arange(L)[None] <= torch.arange(L - (hi - lo), L)[:, None]
        ref = torch.nn.functional.scaled_dot_product_attention(q, k, v, attn_mask=see)
        assert torch.allclose(out[lo:hi].transpose(0, 1), ref, atol=1e-12)
        w = torch.nn.functional.scaled_dot_product_attention(q, k, torch.eye(L, dtype=R.F64).expand(4, L, L), attn_mask=see)
        assert torch.allclose(mass[b, :, :L], w.sum(dim=1).view(2, 2, L).sum(dim=1), atol=1e-12)
    x, pos = torch.randn(5, 3, 64, dtype=R.F64), torch.tensor([0, 1, 7, 1000, 99999])
    inv, m = R.rope_freqs(64, 1e4, "none", 1.0, 1)
    turn = torch.polar(torch.tensor(m, dtype=R.F64), pos[:, None].double() * torch.tensor(inv, dtype=R.F64))[:, None]
    z = torch.complex(x[..., 0::2], x[..., 1::2]) * turn
    assert torch.allclose(R.rotate(x, pos, 64, "interleaved", inv, m), torch.view_as_real(z).flatten(-2), atol=1e-12)
    z = torch.complex(x[..., :32], x[..., 32:]) * turn
    assert torch.allclose(R.rotate(x, pos, 64, "half", inv, m), torch.cat([z.real, z.imag], -1), atol=1e-12)
