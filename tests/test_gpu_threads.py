"""Calls from host threads that have done nothing on the GPU before: a serving loop's workers."""

import threading

import pytest
import torch

import latent_ref
import paged_ref
import test_gpu_latent as latent
import test_gpu_paged as paged
from synth import get_workload, make_inputs, scaled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spg():
    import query_aware_sparse_page_gb300 as m

    return m


def in_a_new_thread(f):
    got = []

    def run():
        try:
            f()
        except Exception as e:  # noqa: BLE001 - shown by the assertion
            got.append(repr(e))

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert got == []


def test_latent_calls(spg):
    x = latent.Run(spg, latent_ref.Latent(16, 512, 64, "bf16", [700, 130], [1, 3]))
    rope = spg.make_rope(rot_dim=64)
    latent.layer(x, rope)
    want = [t.clone() for t in (x.out, x.o_lat, x.lse, x.q_lat)]
    for f in (lambda: spg.latent_absorb(x.p, x.q, x.w_kv, x.q_lat), x.attend,
              lambda: spg.latent_project(x.p, x.o_lat, x.w_kv, x.out), lambda: latent.layer(x, rope)):
        in_a_new_thread(f)
    assert x.err() == 0
    for a, b in zip((x.out, x.o_lat, x.lse, x.q_lat), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kv, q", [("bf16", "bf16"), ("i8", "f16")])
def test_chunk_calls(spg, kv, q):
    r = paged.Run(spg, paged_ref.Chunk(8, 2, 128, 64, kv, q, [700, 130], [1, 40]))
    mass = torch.zeros((2, 2, r.page_table.shape[1] * 64), device="cuda")
    in_a_new_thread(r.chunk)
    paged.check_chunk(r)
    in_a_new_thread(lambda: r.mass(r.lse, None, mass, 1.0))
    again = torch.zeros_like(mass)
    r.mass(r.lse, None, again, 1.0)
    assert r.err() == 0 and bool((mass.sum() > 0).all()) and torch.equal(mass, again)


def test_decode_calls(spg):
    w = scaled(get_workload("tiny-quest-gqa4-1k"))
    inp = make_inputs(w, device="cuda")
    p = spg.params_for(inp)
    b = spg.alloc_buffers(p, "cuda")
    spg.sparse_page_meta_update(p, inp.k_pool, None, inp.page_table, inp.seq_lens, 1, b.minmax, None, None, None, b.ws)

    def step():
        spg.sparse_decode_select_attend(p, inp.q, inp.k_pool, inp.v_pool, None, None, inp.page_table, inp.seq_lens, b.minmax,
                                        None, None, None, b.sel, b.sel_cnt, b.out, b.lse, b.ws)

    def dense():
        spg.dense_decode_attention(p, inp.q, inp.k_pool, inp.v_pool, None, None, inp.page_table, inp.seq_lens, b.out, b.lse, b.ws)

    for f in (step, dense):
        f()
        want = b.out.clone(), b.lse.clone()
        b.out.zero_()
        in_a_new_thread(f)
        assert torch.equal(b.out, want[0]) and torch.equal(b.lse, want[1])
    assert spg.spg_read_device_error(b.ws) == 0
