"""The latent-cache entry points on the host: workspace sizes and every refusal, without a GPU, and the tests' own
64-bit forms against a library routine."""

import ctypes
import math

import pytest
import torch

import latent_ref as R


@pytest.fixture(scope="module")
def spg():
    import __graft_entry__

    __graft_entry__.build()
    import query_aware_sparse_page_gb300 as m

    return m


def _p(spg, **kw):
    a = dict(batch=2, num_heads=16, latent_dim=512, page_size=64, num_phys_pages=100, max_pages_per_seq=32, dtype="bf16")
    a.update(kw)
    return spg.make_latent_params(**a)


@pytest.mark.parametrize("kw, status", [
    (dict(), 0), (dict(latent_dim=256, nope_dim=64, v_dim=64, page_size=16, dtype="f16"), 0), (dict(num_heads=1024), 0),
    (dict(batch=0), 1), (dict(num_heads=0), 1), (dict(latent_dim=0), 1), (dict(latent_dim=500), 1), (dict(rope_dim=0), 1),
    (dict(rope_dim=8), 1), (dict(nope_dim=0), 1), (dict(v_dim=20), 1), (dict(page_size=24), 1), (dict(page_size=256), 1),
    (dict(num_phys_pages=0), 1), (dict(max_pages_per_seq=0), 1), (dict(max_pages_per_seq=2 ** 26), 1), (dict(dtype=3), 1),
    (dict(dtype=-1), 1), (dict(softmax_scale=-1.0), 1), (dict(softmax_scale=math.inf), 1), (dict(softmax_scale=math.nan), 1),
    # valid, not built
    (dict(num_heads=1025), 2), (dict(latent_dim=384), 2), (dict(rope_dim=32), 2), (dict(nope_dim=96), 2), (dict(v_dim=256), 2),
    (dict(page_size=8), 2), (dict(dtype="i8"), 2), (dict(num_phys_pages=2 ** 29), 2),
])
def test_validate(spg, kw, status):
    assert spg.spg_latent_validate(_p(spg, **kw)) == status
    assert spg.LIB.spg_latent_validate(None) == 1


def test_workspace(spg):
    sizes = [spg.spg_latent_workspace_size(_p(spg), t) for t in (0, 1, 4, 10000)]
    assert sizes == sorted(sizes) and sizes[0] > 256 and sizes[2] == sizes[3]
    assert spg.spg_latent_workspace_size(_p(spg, latent_dim=256), 4) < sizes[2]
    for kw, t in ((dict(), -1), (dict(latent_dim=500), 1), (dict(num_heads=1024), 2 ** 22)):
        with pytest.raises(spg.SpgError):
            spg.spg_latent_workspace_size(_p(spg, **kw), t)


A = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: every call below is refused before a launch
B = ctypes.c_void_p(1 << 21)
ODD = ctypes.c_void_p((1 << 20) + 8)
WS = ctypes.c_size_t(1 << 40)


def _attend(spg, p, total=4, q=A, st=A, pool=A, pt=A, sl=A, out=B, lse=None, ws=A, wn=WS):
    return spg.LIB.paged_latent_attention(ctypes.byref(p), total, q, st, pool, pt, sl, out, lse, ws, wn, None)


@pytest.mark.parametrize("kw, status", [
    (dict(total=-1), 1), (dict(q=None), 1), (dict(q=ODD), 1), (dict(st=None), 1), (dict(pool=None), 1), (dict(pool=ODD), 1),
    (dict(pt=None), 1), (dict(sl=None), 1), (dict(out=None), 1), (dict(out=A), 1), (dict(lse=ODD), 1), (dict(ws=None), 1),
    (dict(ws=ODD), 1),
    (dict(wn=ctypes.c_size_t(16)), 4), (dict(total=0, q=None, out=None), 0), (dict(total=2 ** 30), 2),
])
def test_attention_refusals(spg, kw, status):
    assert _attend(spg, _p(spg), **kw) == status


def _append(spg, p, rope="default", total=4, c=A, cs=576, k=A, ks=576, w=None, eps=1e-6, q=A, qs=16 * 192, st=A, pos=None,
            pt=A, sl=A, pool=A, out=B, ws=A, wn=WS):
    r = spg.make_rope(rot_dim=64) if rope == "default" else rope
    return spg.LIB.paged_latent_append(ctypes.byref(p), None if r is None else ctypes.byref(r), total, c, cs, k, ks, w, eps, q,
                                       qs, st, pos, pt, sl, pool, out, ws, wn, None)


@pytest.mark.parametrize("kw, status", [
    (dict(c=None), 1), (dict(c=ODD), 1), (dict(k=None), 1), (dict(cs=504), 1), (dict(cs=580), 1), (dict(ks=56), 1), (dict(ks=60), 1),
    (dict(w=ODD), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(q=None), 1), (dict(out=None), 1),
    (dict(out=A), 1), (dict(qs=16 * 192 - 8), 1), (dict(qs=16 * 192 + 4), 1), (dict(st=None), 1), (dict(pos=ODD), 1),
    (dict(pool=None), 1), (dict(sl=None), 1), (dict(pt=ODD), 1), (dict(total=-3), 1), (dict(ws=None), 1),
    (dict(wn=ctypes.c_size_t(8)), 4), (dict(total=0, c=None), 0),
])
def test_append_refusals(spg, kw, status):
    assert _append(spg, _p(spg), **kw) == status


def test_append_refuses_rope(spg):
    assert _append(spg, _p(spg), spg.make_rope(rot_dim=24)) == 2  # valid, not built
    assert _append(spg, _p(spg), spg.make_rope(rot_dim=128)) == 1
    assert _append(spg, _p(spg), spg.make_rope(base=0.5)) == 1
    assert _append(spg, _p(spg, dtype="i8")) == 2


@pytest.mark.parametrize("kw, status", [
    (dict(total=-1), 1), (dict(q=None), 1), (dict(q=ODD), 1), (dict(qs=16 * 192 - 8), 1), (dict(qs=16 * 192 + 2), 1), (dict(w=None), 1),
    (dict(w=ODD), 1), (dict(y=None), 1), (dict(y=A), 1), (dict(total=0, q=None), 0), (dict(total=2 ** 30), 2),
])
def test_absorb_refusals(spg, kw, status):
    a = dict(total=4, q=A, qs=16 * 192, w=A, y=B)
    a.update(kw)
    assert spg.LIB.latent_absorb(ctypes.byref(_p(spg)), a["total"], a["q"], a["qs"], a["w"], a["y"], None) == status


@pytest.mark.parametrize("kw, status", [
    (dict(total=-1), 1), (dict(o=None), 1), (dict(o=ODD), 1), (dict(w=None), 1), (dict(w=ODD), 1), (dict(y=None), 1), (dict(y=A), 1),
    (dict(total=0, o=None), 0),
])
def test_project_refusals(spg, kw, status):
    a = dict(total=4, o=A, w=A, y=B)
    a.update(kw)
    assert spg.LIB.latent_project(ctypes.byref(_p(spg)), a["total"], a["o"], a["w"], a["y"], None) == status


def test_binding_refuses_shapes_types_and_host_tensors(spg):
    p, bf = _p(spg), torch.bfloat16
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)  # noqa: E731
    pool, st, pt, sl = z(100, 64, 576), z(3, dt=torch.int32), z(2, 32, dt=torch.int32), z(2, dt=torch.int32)
    ws = z(1, dt=torch.uint8)
    with pytest.raises(ValueError, match="shape"):
        spg.paged_latent_attention(p, z(4, 16, 512), st, pool, pt, sl, z(4, 16, 512), ws=ws)
    with pytest.raises(ValueError, match="shape"):
        spg.paged_latent_attention(p, z(4, 16, 576), st, z(100, 64, 512), pt, sl, z(4, 16, 512), ws=ws)
    with pytest.raises(ValueError):  # host tensors
        spg.paged_latent_attention(p, z(4, 16, 576), st, pool, pt, sl, z(4, 16, 512), ws=ws)
    with pytest.raises(ValueError, match="expected torch.bfloat16"):
        spg.latent_absorb(p, z(4, 16, 192, dt=torch.float16), z(16, 256, 512), z(4, 16, 576))
    with pytest.raises(ValueError, match="shape"):
        spg.latent_project(p, z(4, 16, 512), z(16, 128, 512), z(4, 16, 128))
    with pytest.raises(ValueError):
        spg.latent_project(p, z(4, 16, 512), z(16, 256, 512), z(4, 16, 128))
    with pytest.raises(ValueError, match="contiguous"):
        spg.paged_latent_append(p, None, z(512, 4).t(), z(4, 64), None, 0.0, None, st, pt, sl, pool, ws=ws)
    with pytest.raises(ValueError, match="heads"):
        spg.latent_absorb(p, z(4, 16, 384)[..., :192], z(16, 256, 512), z(4, 16, 576))


def test_reference_forms_agree_with_a_library_routine():
    """Absorbed attention and its projection against torch's attention over the expanded keys and values."""
    c = R.Latent(3, 256, 16, "f16", [37, 5], [9, 5], dn=64, seed=3, poison=0.0)
    y, _ = R.absorb(c)
    c.q_lat = torch.cat([y, c.q_lat[..., c.r :].to(R.F64)], dim=2)
    o, _, lse, _ = R.attention(c)
    out, _ = R.project(c, o)
    w = c.w_kv.to(R.F64)
    for b, L in enumerate(c.lens):
        lo, hi = c.starts[b], c.starts[b + 1]
        kv = c.tokens(b)
        k = torch.cat([torch.einsum("tc,hdc->htd", kv[:, : c.r], w[:, : c.dn]), kv[:, c.r :].expand(3, L, 64)], dim=2)
        v = torch.einsum("tc,hvc->htv", kv[:, : c.r], w[:, c.dn :])
        q = torch.cat([c.q[lo:hi, :, : c.dn].to(R.F64), c.q_lat[lo:hi, :, c.r :]], dim=2).transpose(0, 1)
        see = torch.arange(L)[None] <= torch.arange(L - (hi - lo), L)[:, None]
        ref = torch.nn.functional.scaled_dot_product_attention(q, k, v, attn_mask=see, scale=c.scale)
        assert torch.allclose(out[lo:hi].transpose(0, 1), ref, atol=1e-11)
        z = (q @ k.transpose(1, 2) * c.scale).masked_fill(~see, -math.inf)
        assert torch.allclose(lse[lo:hi].t(), torch.logsumexp(z, dim=2), atol=1e-11)


def test_reference_append_agrees_with_complex_turns():
    c = R.Latent(2, 256, 16, "f16", [30], [5])
    inv, m = R.rope_freqs(64, 1e4, "none", 1.0, 1)
    row, _, q, _ = R.append(c, 64, "half", inv, m, 1e-6)
    turn = torch.polar(torch.tensor(1.0, dtype=R.F64), torch.arange(25, 30)[:, None].double() * torch.tensor(inv, dtype=R.F64))
    x = c.kv[:, 256:].to(R.F64)
    z = torch.complex(x[:, :32], x[:, 32:]) * turn
    assert torch.allclose(row[:, 256:], torch.cat([z.real, z.imag], 1), atol=1e-12)
    y = torch.nn.functional.rms_norm(c.kv[:, :256].to(R.F64), (256,), c.norm.to(R.F64), 1e-6)
    assert torch.allclose(row[:, :256], y, atol=1e-12)


# ---- another device --------------------------------------------------------------------------

from test_paged_devices_host import On  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
CACHE = dict(pool=(BF, 20, 64, 576), page_table=(I32, 3, 5), seq_lens=(I32, 3), q_start=(I32, 4))
CALLS = {
    "paged_latent_append": dict(CACHE, c=(BF, 7, 512), k_pe=(BF, 7, 64), norm_weight=(BF, 512), q=(BF, 7, 8, 192),
                                q_lat=(BF, 7, 8, 576), positions=(I32, 7)),
    "paged_latent_attention": dict(CACHE, q_lat=(BF, 7, 8, 576), o_lat=(BF, 7, 8, 512), lse=(F32, 7, 8)),
    "latent_absorb": dict(q=(BF, 7, 8, 192), w_kv=(BF, 8, 256, 512), q_lat=(BF, 7, 8, 576)),
    "latent_project": dict(o_lat=(BF, 7, 8, 512), w_kv=(BF, 8, 256, 512), out=(BF, 7, 8, 128)),
}


@pytest.mark.parametrize("fn, name", [(f, n) for f, ts in CALLS.items() for n in ts])
@pytest.mark.parametrize("dev", [0, -1])
def test_tensors_of_another_device_are_refused(spg, monkeypatch, fn, name, dev):
    """Every tensor on device 1 but one: refused, and the library is not called."""
    p = spg.make_latent_params(batch=3, num_heads=8, latent_dim=512, page_size=64, num_phys_pages=20, max_pages_per_seq=5)
    monkeypatch.setattr(spg.binding, "LIB", None)
    args = {n: On(1, *t) for n, t in CALLS[fn].items()}
    args[name] = On(dev, *CALLS[fn][name])
    if fn.startswith("paged"):
        args["ws"] = On(1, torch.uint8, 1 << 30)
    extra = dict(rope=None, eps=1e-6) if fn == "paged_latent_append" else {}
    with pytest.raises(ValueError):
        getattr(spg, fn)(p, **args, **extra)
