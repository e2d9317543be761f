"""Where the latent-cache operators are easily wrong, beside tests/test_gpu_latent.py."""

import ctypes
import math
import shutil
import subprocess

import pytest
import torch

import latent_exact as X
import latent_ref as R
import paged_ref
import test_gpu_latent as latent
import test_gpu_paged as paged
from synth import get_workload, make_inputs, scaled
from test_gpu_latent import Run, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spg():
    import query_aware_sparse_page_gb300 as m

    return m


# ---- a launch before that lets the next one start at once, and then takes its time -----------------

LATE_COPY = r"""
#include <cuda_runtime.h>
__global__ void k_late_copy(uint4* dst, const uint4* src, long long n, unsigned long long ns) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  unsigned long long t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  for (int i = 0; i < 1 << 20; ++i) {
    __nanosleep(10000);
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (t - t0 > ns) break;
  }
  for (long long i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src[i];
}
extern "C" int late_copy(void* dst, const void* src, long long bytes, unsigned long long ns, void* stream) {
  k_late_copy<<<1, 256, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<uint4*>(dst), static_cast<const uint4*>(src),
                                                                bytes / 16, ns);
  return cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def late_copy(tmp_path_factory):
    """dst = src, 250 ms later, by a launch whose dependents may start at its beginning."""
    d = tmp_path_factory.mktemp("late")
    (d / "late.cu").write_text(LATE_COPY)
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-Xcompiler", "-fPIC", "-o",
                    str(d / "late.so"), str(d / "late.cu")], check=True)
    fn = ctypes.CDLL(str(d / "late.so")).late_copy
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_ulonglong, ctypes.c_void_p]

    def copy(dst, src):
        n = dst.numel() * dst.element_size()
        assert dst.shape == src.shape and dst.dtype == src.dtype and dst.is_contiguous() and src.is_contiguous() and n % 16 == 0
        assert fn(dst.data_ptr(), src.data_ptr(), n, 250_000_000, torch.cuda.current_stream().cuda_stream) == 0

    return copy


@pytest.mark.parametrize("H, T", [(16, 3), (130, 140)])
def test_head_products_wait_out_a_long_launch(spg, late_copy, H, T):
    """2.5 times as long as a bounded wait of theirs: their inputs come from that launch."""
    c = R.Latent(H, 512, 16, "bf16", [T], [T])
    x = Run(spg, c)
    o = (0.1 * torch.randn(T, H, 512, generator=torch.Generator().manual_seed(T))).to(torch.bfloat16)
    q, oc = x.q.clone(), o.cuda()
    x.q.zero_()
    x.o_lat.zero_()
    torch.cuda.synchronize()
    late_copy(x.q, q)
    spg.latent_absorb(x.p, x.q, x.w_kv, x.q_lat)
    late_copy(x.o_lat, oc)
    spg.latent_project(x.p, x.o_lat, x.w_kv, x.out)
    torch.cuda.synchronize()
    y, tol = R.absorb(c)
    close(x.q_lat[..., :512], y, tol, "absorb")
    y, tol = R.project(c, o)
    close(x.out, y, tol, "project")


# ---- head products at the borders of their forms -------------------------------------------------


@pytest.mark.parametrize("H, r, dn, dv, T", [
    # 32 columns a CTA up to 32 rows, 64 up to 128, then tiles of 128 rows
    (4, 512, 128, 128, 31), (4, 256, 64, 64, 32), (4, 512, 128, 128, 33), (3, 256, 128, 128, 64), (3, 512, 64, 128, 257),
    # absorbing with one CTA for all columns: more than 16 rows, their tiles times heads from as many as there are SMs on
    (152, 512, 128, 64, 16), (152, 512, 128, 64, 17), (130, 256, 64, 64, 140), (130, 512, 64, 128, 129), (151, 256, 64, 64, 1), (152, 512, 64, 64, 1), (152, 256, 128, 64, 2),
    (200, 512, 128, 64, 1), (200, 256, 64, 128, 5), (200, 512, 64, 64, 33), (1024, 256, 64, 64, 1), (1024, 256, 64, 64, 3),
])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_head_products_at_borders(spg, H, r, dn, dv, T, dt):
    c = R.Latent(H, r, 16, dt, [T], [T], dn=dn, dv=dv, pad_rows=3)
    x = Run(spg, c)
    x.q_lat.fill_(5.0)
    spg.latent_absorb(x.p, x.q[:T], x.w_kv, x.q_lat[:T])
    y, tol = R.absorb(c)
    close(x.q_lat[:T, :, :r], y[:T], tol[:T], "absorb")
    assert bool((x.q_lat[..., r:] == 5.0).all()) and bool((x.q_lat[T:] == 5.0).all())
    o = (0.1 * torch.randn(T + 3, H, r, generator=torch.Generator().manual_seed(T))).to(R.DT[dt])
    spg.latent_project(x.p, o.cuda()[:T], x.w_kv, x.out[:T])
    y, tol = R.project(c, o)
    close(x.out[:T], y[:T], tol[:T], "project")
    assert bool((x.out[T:] == 7.0).all())


# ---- logits near the end of the 32-bit range ------------------------------------------------------


@pytest.mark.parametrize("dt, q, k, scale", [("bf16", 2.0 ** 60, -(2.0 ** 67), 1.0), ("f16", 2.0 ** 10, -(2.0 ** 10), 2.0 ** 107),
                                             ("bf16", 2.0 ** 60, 2.0 ** 67, 1.0)])
@pytest.mark.parametrize("H, lens, new", [(4, [1, 200], [1, 3]), (70, [1, 200], [1, 3]), (4, [3000, 5], [1, 1])])
def test_logits_near_the_end_of_the_range(spg, H, lens, new, dt, q, k, scale):
    """Logits of 2^127 (2.5e38 in base 2) of either sign, the same for all tokens: the mean of the tokens seen.  Where they
    are above 0, a sequence's first token has the opposite one and so no weight.

    TOLERANCE.  The weights are equal and a power of two, so P is exact; the sums of L terms in 32 bits and one inverse
    cost (2 L + 8) 2^-24 of sum p |c|, the result's rounding e |o| (fp16: and 2^-25)."""
    c = R.Latent(H, 256, 16, dt, lens, new)
    c.q_lat.zero_()
    c.q_lat[..., 0] = q
    live = ~torch.isnan(c.pool)
    c.pool[..., 0] = k
    c.pool[~live] = math.nan
    first = [(int(c.page_table[b, 0]), 0) for b, L in enumerate(lens) if L > 1 and k > 0]
    for pg, sl in first:
        c.pool[pg, sl, 0] = -k
    x = Run(spg, c, softmax_scale=scale)
    x.attend()
    assert x.err() == 0
    want = torch.zeros((c.T, H, 256), dtype=R.F64)
    tol = torch.zeros_like(want)
    e = torch.finfo(R.DT[dt]).eps / 2
    for b, L in enumerate(lens):
        kv = c.tokens(b)[:, :256]
        for i in range(new[b]):
            seen = kv[1 if L > 1 and k > 0 else 0 : L - new[b] + i + 1]
            t = c.starts[b] + i
            want[t] = seen.mean(dim=0)
            tol[t] = 1.01 * e * want[t].abs() + (2 * len(seen) + 8) * 2.0 ** -24 * seen.abs().mean(dim=0) + 2.0 ** -25
    close(x.o_lat, want, tol, "o_lat")
    z = q * k * scale
    close(x.lse, torch.full((c.T, H), z, dtype=R.F64), torch.full((c.T, H), 2.0 ** -21 * abs(z), dtype=R.F64), "lse")


# ---- exact logits ---------------------------------------------------------------------------------


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("H, r, lens, new", X.CASES)
def test_exact_logits_show_both_values_of_p(spg, H, r, lens, new, dt):
    """Within a tolerance that one value of P, or a second one of the wrong sign or place, does not keep (the model in
    tests/test_latent_exact_host.py); with one value within that one's, and not the same."""
    c = X.chunk(H, r, lens, new, dt)
    x = Run(spg, c, softmax_scale=X.SCALE)
    got = {}
    for parts in (1, 2):
        try:
            spg.spg_set_chunk_parts(parts)
            x.attend()
        finally:
            spg.spg_set_chunk_parts(2)
        assert x.err() == 0
        close(x.o_lat, *X.attention(c, parts), f"o_lat, {parts}")
        got[parts] = x.o_lat.clone()
    assert not torch.equal(got[1], got[2])


# ---- a workspace that other entry points use as well ----------------------------------------------


@pytest.mark.parametrize("slack", [0, 16, 1000 * 16])
def test_a_workspace_shared_with_the_other_entry_points(spg, slack):
    """Latent calls in between chunk attention, attention mass and decode steps (each in its kernels), on one workspace of
    both sizes together: everything as on workspaces of their own, and the other calls' part as they left it."""
    w = scaled(get_workload("tiny-quest-gqa4-1k"))
    inp = make_inputs(w, device="cuda")
    p = spg.params_for(inp)
    b = spg.alloc_buffers(p, "cuda")
    ch = paged.Run(spg, paged_ref.Chunk(8, 2, 128, 64, "bf16", "bf16", [3000, 900], [2, 200]))
    few = latent.Run(spg, R.Latent(64, 512, 64, "bf16", [3000, 900], [1, 4], seed=1))
    many = latent.Run(spg, R.Latent(128, 256, 16, "f16", [2000], [2], seed=2))
    mass = torch.zeros((2, 2, ch.page_table.shape[1] * 64), device="cuda")
    spg.sparse_page_meta_update(p, inp.k_pool, None, inp.page_table, inp.seq_lens, 1, b.minmax, None, None, None, b.ws)

    def step(kernel, ws):
        spg.spg_set_step_kernel(kernel)
        try:
            spg.sparse_decode_select_attend(p, inp.q, inp.k_pool, inp.v_pool, None, None, inp.page_table, inp.seq_lens, b.minmax,
                                            None, None, None, b.sel, b.sel_cnt, b.out, b.lse, ws)
        finally:
            spg.spg_set_step_kernel(0)
        return b.out.clone(), b.lse.clone(), b.sel.clone()

    def chunk(ws):
        ch.ws = ws
        ch.out.fill_(7.0)
        ch.chunk()
        ch.mass(ch.lse, None, mass, 1.0)
        return ch.out.clone(), ch.lse.clone(), mass.clone()

    def attend(x, ws):
        x.ws = ws
        x.o_lat.fill_(7.0)
        x.attend()
        return x.o_lat.clone(), x.lse.clone()

    # both geometries' calls on their own workspaces, and a workspace per geometry shared with the latent ones
    calls = [lambda ws: step(1, ws[0]), lambda ws: attend(few, ws[0]), lambda ws: step(2, ws[0]), lambda ws: attend(many, ws[0]),
             lambda ws: step(1, ws[0]), lambda ws: chunk(ws[1]), lambda ws: attend(few, ws[1]), lambda ws: chunk(ws[1]),
             lambda ws: attend(many, ws[1]), lambda ws: chunk(ws[1])]
    zeros = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    n_step, n_chunk = spg.spg_workspace_size(p), spg.spg_chunk_workspace_size(ch.p, ch.c.T)
    n_latent = max(spg.spg_latent_workspace_size(x.p, x.c.T) for x in (few, many))
    want = []
    for i, f in enumerate(calls):
        own = [zeros(n_latent if i in (1, 3) else n_step), zeros(n_latent if i in (6, 8) else n_chunk)]
        want.append(f(own))
    shared = [zeros(n_step + n_latent + slack), zeros(n_chunk + n_latent + slack)]
    for _ in range(3):
        for i, f in enumerate(calls):
            rest = shared[0 if i < 5 else 1][: n_step if i < 5 else n_chunk]
            before = rest.clone()
            got = f(shared)
            if i in (1, 3, 6, 8):
                assert torch.equal(rest, before)
            for x, y in zip(got, want[i]):
                assert torch.equal(x, y)
    for ws in shared:
        assert spg.spg_read_device_error(ws) == 0
