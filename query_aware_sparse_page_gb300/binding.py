"""ctypes binding of libspg.so: argument marshalling only.

Every function here has the name of the C entry point it calls, checks that
the tensors it is given are contiguous CUDA tensors, passes their device
pointers and the current CUDA stream, and turns a non-OK status into
SpgError.  No step of the computation runs in Python, and there is no
fallback: if the library is missing, importing this module fails.
"""

from __future__ import annotations

import ctypes
import functools
import os
from ctypes import POINTER, c_char_p, c_double, c_float, c_int32, c_int64, c_size_t, c_void_p

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libspg.so")

SPG_OK, SPG_EINVAL, SPG_EUNSUPPORTED, SPG_ECUDA, SPG_EWORKSPACE = 0, 1, 2, 3, 4
SEL_QUEST, SEL_SKETCH_INT4, SEL_ALL, SEL_PROBE = 0, 1, 2, 3
F16, BF16, I8 = 0, 1, 2
DEVERR_PAGE_ID, DEVERR_SEQ_LEN, DEVERR_SEL, DEVERR_TIMEOUT, DEVERR_Q_START = 1, 2, 4, 8, 16

_DTYPES = {"f16": F16, "bf16": BF16, "i8": I8}
_SELECTORS = {"quest": SEL_QUEST, "sketch": SEL_SKETCH_INT4, "all": SEL_ALL, "probe": SEL_PROBE}


class SpgError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} (status {status})")


class spg_params(ctypes.Structure):
    _fields_ = [
        ("batch", c_int32),
        ("num_q_heads", c_int32),
        ("num_kv_heads", c_int32),
        ("head_dim", c_int32),
        ("page_size", c_int32),
        ("num_phys_pages", c_int32),
        ("max_pages_per_seq", c_int32),
        ("kv_dtype", c_int32),
        ("q_dtype", c_int32),
        ("selector", c_int32),
        ("token_budget", c_int32),
        ("n_sink_pages", c_int32),
        ("n_recent_pages", c_int32),
        ("sketch_dim", c_int32),
        ("softmax_scale", c_float),
        ("top_p", c_float),
        ("min_pages", c_int32),
        ("n_probe", c_int32),
    ]

    def __repr__(self):
        return "spg_params(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


def make_params(batch, num_q_heads, num_kv_heads, head_dim, page_size, num_phys_pages,
                max_pages_per_seq, kv_dtype="f16", q_dtype=None, selector="quest",
                token_budget=0, n_sink_pages=0, n_recent_pages=0, sketch_dim=16,
                softmax_scale=0.0, top_p=0.0, min_pages=0, n_probe=0) -> spg_params:
    kv = _DTYPES[kv_dtype] if isinstance(kv_dtype, str) else int(kv_dtype)
    if q_dtype is None:
        q_dtype = kv if kv != I8 else F16
    qd = _DTYPES[q_dtype] if isinstance(q_dtype, str) else int(q_dtype)
    sel = _SELECTORS[selector] if isinstance(selector, str) else int(selector)
    return spg_params(batch, num_q_heads, num_kv_heads, head_dim, page_size, num_phys_pages,
                      max_pages_per_seq, kv, qd, sel, token_budget, n_sink_pages, n_recent_pages,
                      sketch_dim, softmax_scale, top_p, min_pages, n_probe)


class spg_rope(ctypes.Structure):
    _fields_ = [
        ("rot_dim", c_int32),
        ("layout", c_int32),
        ("scaling", c_int32),
        ("orig_len", c_int32),
        ("base", c_double),
        ("factor", c_double),
    ]


_ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
_ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def make_rope(rot_dim=0, layout="half", base=10000.0, scaling="none", factor=1.0,
              orig_len=1) -> spg_rope:
    lay = _ROPE_LAYOUTS[layout] if isinstance(layout, str) else int(layout)
    sc = _ROPE_SCALINGS[scaling] if isinstance(scaling, str) else int(scaling)
    return spg_rope(int(rot_dim), lay, sc, int(orig_len), float(base), float(factor))


class spg_latent_params(ctypes.Structure):
    _fields_ = [
        ("batch", c_int32),
        ("num_heads", c_int32),
        ("latent_dim", c_int32),
        ("rope_dim", c_int32),
        ("nope_dim", c_int32),
        ("v_dim", c_int32),
        ("page_size", c_int32),
        ("num_phys_pages", c_int32),
        ("max_pages_per_seq", c_int32),
        ("dtype", c_int32),
        ("softmax_scale", c_float),
    ]

    def __repr__(self):
        return "spg_latent_params(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


def make_latent_params(batch, num_heads, latent_dim, page_size, num_phys_pages, max_pages_per_seq, rope_dim=64,
                       nope_dim=128, v_dim=128, dtype="bf16", softmax_scale=0.0) -> spg_latent_params:
    dt = _DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    return spg_latent_params(batch, num_heads, latent_dim, rope_dim, nope_dim, v_dim, page_size, num_phys_pages,
                             max_pages_per_seq, dt, softmax_scale)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run query_aware_sparse_page_gb300._build.build() "
            "(nvcc for sm_103a).  There is no fallback implementation.")
    lib = ctypes.CDLL(LIB_PATH)
    P, PL = POINTER(spg_params), POINTER(spg_latent_params)
    v = c_void_p
    sigs = {
        "spg_abi_version": ([], c_int32),
        "spg_status_str": ([c_int32], c_char_p),
        "spg_validate": ([P], c_int32),
        "spg_workspace_size": ([P, POINTER(c_size_t)], c_int32),
        "sparse_page_meta_update": ([P, v, v, v, v, c_int32, v, v, v, v, v, c_size_t, v], c_int32),
        "sparse_page_score": ([P, v, v, v, v, v, v, v, v, v, c_size_t, v], c_int32),
        "sparse_page_select": ([P, v, v, v, v, v, v, v, v, v, v, c_size_t, v], c_int32),
        "sparse_decode_attention": ([P, v, v, v, v, v, v, v, v, v, v, v, v, c_size_t, v], c_int32),
        "sparse_decode_select_attend": (
            [P, v, v, v, v, v, v, v, v, v, v, v, v, v, v, v, v, c_size_t, v], c_int32),
        "dense_decode_attention": ([P, v, v, v, v, v, v, v, v, v, v, c_size_t, v], c_int32),
        "sparse_decode_step": (
            [P, v, v, v, v, v, v, v, v, v, v, v, v, v, v, v, v, c_size_t, v], c_int32),
        "sparse_page_sketch_dots": ([P, v, v, v, v, v, v, v, v, c_size_t, v], c_int32),
        "spg_chunk_workspace_size": ([P, c_int32, POINTER(c_size_t)], c_int32),
        "spg_rope_freqs": ([POINTER(spg_rope), c_int32, POINTER(c_double), POINTER(c_double)], c_int32),
        "paged_rope_append": (
            [P, POINTER(spg_rope), c_int32, v, c_int64, v, c_int64, v, c_int64, v, v, v, v, v, v, v, v, v, v,
             c_size_t, v], c_int32),
        "paged_chunk_attention": (
            [P, c_int32, v, v, v, v, v, v, v, v, v, v, v, c_size_t, v], c_int32),
        "paged_attention_mass": (
            [P, c_int32, v, v, v, v, v, v, v, v, v, c_float, v, c_size_t, v], c_int32),
        "paged_cache_evict": (
            [P, v, c_int32, c_int32, c_int32, v, v, v, v, v, v, v, v, v, v, v, c_size_t, v], c_int32),
        "spg_latent_validate": ([PL], c_int32),
        "spg_latent_workspace_size": ([PL, c_int32, POINTER(c_size_t)], c_int32),
        "paged_latent_append": (
            [PL, POINTER(spg_rope), c_int32, v, c_int64, v, c_int64, v, c_float, v, c_int64, v, v, v, v, v, v, v,
             c_size_t, v], c_int32),
        "latent_absorb": ([PL, c_int32, v, c_int64, v, v, v], c_int32),
        "latent_project": ([PL, c_int32, v, v, v, v], c_int32),
        "paged_latent_attention": ([PL, c_int32, v, v, v, v, v, v, v, v, c_size_t, v], c_int32),
        "spg_step_kernel": ([P], c_char_p),
        "spg_prefer_dense": ([P, c_int32, c_float], c_int32),
        "spg_step_launches": ([P], c_int32),
        "spg_set_step_kernel": ([c_int32], c_int32),
        "spg_set_chunk_parts": ([c_int32], c_int32),
        "spg_read_device_error": ([v, POINTER(c_int32), v], c_int32),
        "spg_clear_device_error": ([v, v], c_int32),
        "spg_test_withhold_first_stage": ([v, v], c_int32),
    }
    for name, (args, res) in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


LIB = _load()


# ---- marshalling helpers ----------------------------------------------------
def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libspg takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libspg takes contiguous tensors")
    return c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return c_void_p(int(stream))
    import torch

    return c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(status: int, where: str):
    if status != SPG_OK:
        raise SpgError(status, where)


def _ws(ws):
    return _ptr(ws), c_size_t(ws.numel() * ws.element_size())


# ---- host-only entry points ---------------------------------------------------
def spg_abi_version() -> int:
    return LIB.spg_abi_version()


def status_str(status: int) -> str:
    return LIB.spg_status_str(status).decode()


spg_status_str = status_str


def spg_validate(p: spg_params) -> int:
    return LIB.spg_validate(ctypes.byref(p))


def spg_workspace_size(p: spg_params) -> int:
    n = c_size_t(0)
    _check(LIB.spg_workspace_size(ctypes.byref(p), ctypes.byref(n)), "spg_workspace_size")
    return n.value


def spg_step_kernel(p: spg_params) -> str | None:
    r = LIB.spg_step_kernel(ctypes.byref(p))
    return None if r is None else r.decode()


step_kernel_name = spg_step_kernel


def spg_prefer_dense(p: spg_params, max_seq_len: int, ratio: float = 0.0) -> bool:
    return bool(LIB.spg_prefer_dense(ctypes.byref(p), int(max_seq_len), float(ratio)))


def spg_step_launches(p: spg_params) -> int:
    return LIB.spg_step_launches(ctypes.byref(p))


step_launch_count = spg_step_launches

STEP_KERNEL_AUTO, STEP_KERNEL_CLUSTER, STEP_KERNEL_SCHED = 0, 1, 2


def spg_set_step_kernel(kernel: int):
    _check(LIB.spg_set_step_kernel(int(kernel)), "spg_set_step_kernel")


# ---- device entry points -------------------------------------------------------
def sparse_page_meta_update(p, k_pool, k_scale, page_table, seq_lens, rebuild, minmax=None,
                            sketch=None, sketch_scale=None, proj=None, ws=None, stream=None):
    wp, wn = _ws(ws)
    _check(LIB.sparse_page_meta_update(
        ctypes.byref(p), _ptr(k_pool), _ptr(k_scale), _ptr(page_table), _ptr(seq_lens),
        int(rebuild), _ptr(minmax), _ptr(sketch), _ptr(sketch_scale), _ptr(proj), wp, wn,
        _stream(stream)), "sparse_page_meta_update")


def sparse_page_score(p, q, page_table, seq_lens, minmax=None, sketch=None, sketch_scale=None,
                      proj=None, scores=None, ws=None, stream=None):
    wp, wn = _ws(ws)
    _check(LIB.sparse_page_score(
        ctypes.byref(p), _ptr(q), _ptr(page_table), _ptr(seq_lens), _ptr(minmax), _ptr(sketch),
        _ptr(sketch_scale), _ptr(proj), _ptr(scores), wp, wn, _stream(stream)),
        "sparse_page_score")


def sparse_page_sketch_dots(p, q, seq_lens, sketch, proj, qc, sq, dots, ws, stream=None):
    wp, wn = _ws(ws)
    _check(LIB.sparse_page_sketch_dots(
        ctypes.byref(p), _ptr(q), _ptr(seq_lens), _ptr(sketch), _ptr(proj), _ptr(qc), _ptr(sq),
        _ptr(dots), wp, wn, _stream(stream)), "sparse_page_sketch_dots")


def sparse_page_select(p, q, page_table, seq_lens, minmax=None, sketch=None, sketch_scale=None,
                       proj=None, sel=None, sel_cnt=None, ws=None, stream=None):
    wp, wn = _ws(ws)
    _check(LIB.sparse_page_select(
        ctypes.byref(p), _ptr(q), _ptr(page_table), _ptr(seq_lens), _ptr(minmax), _ptr(sketch),
        _ptr(sketch_scale), _ptr(proj), _ptr(sel), _ptr(sel_cnt), wp, wn, _stream(stream)),
        "sparse_page_select")


def sparse_decode_attention(p, q, k_pool, v_pool, k_scale, v_scale, page_table, seq_lens, sel,
                            sel_cnt, out, lse=None, ws=None, stream=None):
    wp, wn = _ws(ws)
    _check(LIB.sparse_decode_attention(
        ctypes.byref(p), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale),
        _ptr(page_table), _ptr(seq_lens), _ptr(sel), _ptr(sel_cnt), _ptr(out), _ptr(lse), wp, wn,
        _stream(stream)), "sparse_decode_attention")


def sparse_decode_select_attend(p, q, k_pool, v_pool, k_scale, v_scale, page_table, seq_lens,
                                minmax=None, sketch=None, sketch_scale=None, proj=None, sel=None,
                                sel_cnt=None, out=None, lse=None, ws=None, stream=None):
    wp, wn = _ws(ws)
    _check(LIB.sparse_decode_select_attend(
        ctypes.byref(p), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale),
        _ptr(page_table), _ptr(seq_lens), _ptr(minmax), _ptr(sketch), _ptr(sketch_scale),
        _ptr(proj), _ptr(sel), _ptr(sel_cnt), _ptr(out), _ptr(lse), wp, wn, _stream(stream)),
        "sparse_decode_select_attend")


def sparse_decode_step(p, q, k_pool, v_pool, k_scale, v_scale, page_table, seq_lens,
                       minmax=None, sketch=None, sketch_scale=None, proj=None, sel=None,
                       sel_cnt=None, out=None, lse=None, ws=None, stream=None):
    wp, wn = _ws(ws)
    _check(LIB.sparse_decode_step(
        ctypes.byref(p), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale),
        _ptr(page_table), _ptr(seq_lens), _ptr(minmax), _ptr(sketch), _ptr(sketch_scale),
        _ptr(proj), _ptr(sel), _ptr(sel_cnt), _ptr(out), _ptr(lse), wp, wn, _stream(stream)),
        "sparse_decode_step")


def dense_decode_attention(p, q, k_pool, v_pool, k_scale, v_scale, page_table, seq_lens, out,
                           lse=None, ws=None, stream=None):
    wp, wn = _ws(ws)
    _check(LIB.dense_decode_attention(
        ctypes.byref(p), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale),
        _ptr(page_table), _ptr(seq_lens), _ptr(out), _ptr(lse), wp, wn, _stream(stream)),
        "dense_decode_attention")


# ---- chunks of new tokens ----------------------------------------------------------
_ELEM = {F16: torch.float16, BF16: torch.bfloat16, I8: torch.int8}


def _refuse(name, t, shape, dtype, dev):
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {t.dtype}, expected {dtype}")
    if min(t.get_device(), dev) >= 0 and t.get_device() != dev:
        raise ValueError(f"{name}: on device {t.get_device()}, the workspace on device {dev}")
    raise ValueError("libspg takes contiguous device tensors")


def _device(ws):
    """The workspace's device (-1: the host), which every other tensor has to be on: a kernel there takes them as its
    own memory."""
    return -1 if ws is None else ws.get_device()


def _take(dev, name, t, shape, dtype):
    """Device pointer of a tensor that has to be contiguous, of this shape and type, on this device."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(name, t, shape, dtype, dev)
    return t.data_ptr()


def _take_rows(dev, name, t, shape, dtype):
    """Pointer and row stride of a tensor whose rows are contiguous."""
    if t is None:
        return None, 0
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _refuse(name, t, shape, dtype, dev)
    row, head, one = t.stride()
    if t.numel() and (one != 1 or (shape[1] > 1 and head != shape[2])):
        raise ValueError(f"{name}: the heads of one token have to be contiguous")
    return t.data_ptr(), row if shape[0] > 1 else shape[1] * shape[2]


def _take_cache(dev, p, k_pool, v_pool, k_scale, v_scale, page_table, seq_lens, q_start=None):
    pool, kv = (p.num_phys_pages, p.num_kv_heads, p.page_size, p.head_dim), _ELEM[p.kv_dtype]
    return (_take(dev, "k_pool", k_pool, pool, kv), _take(dev, "v_pool", v_pool, pool, kv),
            _take(dev, "k_scale", k_scale, pool[:3], torch.float16), _take(dev, "v_scale", v_scale, pool[:3], torch.float16),
            _take(dev, "page_table", page_table, (p.batch, p.max_pages_per_seq), torch.int32),
            _take(dev, "seq_lens", seq_lens, (p.batch,), torch.int32),
            _take(dev, "q_start", q_start, (p.batch + 1,), torch.int32))


# the current stream's handle, without an object for it where torch has that (0.1 against 1.1 us per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_one_device = functools.lru_cache(None)(lambda: torch.cuda.device_count() == 1)


def _call(dev, fn, where, ws, stream, *args):
    """fn(*args, workspace, its bytes, stream) with the workspace's device current."""
    if dev < 0 or not ws.is_contiguous():
        raise ValueError("a contiguous workspace on the device is needed")
    if stream is None:
        stream = _raw_stream(dev)
    size = ws.numel() * ws.element_size()
    if _one_device() or dev == torch.cuda.current_device():
        _check(fn(*args, ws.data_ptr(), size, stream), where)
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, ws.data_ptr(), size, stream), where)


def spg_chunk_workspace_size(p: spg_params, total_q: int) -> int:
    n = c_size_t(0)
    _check(LIB.spg_chunk_workspace_size(ctypes.byref(p), int(total_q), ctypes.byref(n)),
           "spg_chunk_workspace_size")
    return n.value


def spg_rope_freqs(rope: spg_rope, head_dim: int):
    """(angle per position of every pair, factor on the rotated channels)."""
    f, m = (c_double * max(head_dim, 2))(), c_double(0)
    _check(LIB.spg_rope_freqs(ctypes.byref(rope), int(head_dim), f, ctypes.byref(m)), "spg_rope_freqs")
    return list(f)[: (rope.rot_dim or head_dim) // 2], m.value


def spg_set_chunk_parts(parts: int):
    """16-bit values (2, the default, or 1) in whose sum a probability of chunk attention enters the P V product."""
    _check(LIB.spg_set_chunk_parts(int(parts)), "spg_set_chunk_parts")


def paged_rope_append(p, rope, q, k, v, q_start, page_table, seq_lens, k_pool, v_pool, k_scale=None,
                      v_scale=None, q_out=None, positions=None, ws=None, stream=None):
    dev, T, d, qd = _device(ws), k.shape[0], p.head_dim, _ELEM[p.q_dtype]
    qp, qs = _take_rows(dev, "q", q, (T, p.num_q_heads, d), qd)
    kp, ks = _take_rows(dev, "k", k, (T, p.num_kv_heads, d), qd)
    vp, vs = _take_rows(dev, "v", v, (T, p.num_kv_heads, d), qd)
    kpool, vpool, ksc, vsc, pt, sl, st = _take_cache(dev, p, k_pool, v_pool, k_scale, v_scale, page_table,
                                                     seq_lens, q_start)
    out = _take(dev, "q_out", q_out, (T, p.num_q_heads, d), qd)
    pos = _take(dev, "positions", positions, (T,), torch.int32)
    _call(dev, LIB.paged_rope_append, "paged_rope_append", ws, stream, ctypes.byref(p),
          None if rope is None else ctypes.byref(rope), T, qp, qs, kp, ks, vp, vs, st, pos, pt, sl, kpool, vpool,
          ksc, vsc, out)


def paged_chunk_attention(p, q, q_start, k_pool, v_pool, k_scale, v_scale, page_table, seq_lens, out,
                          lse=None, ws=None, stream=None):
    dev, T, rows, qd = _device(ws), q.shape[0], (q.shape[0], p.num_q_heads, p.head_dim), _ELEM[p.q_dtype]
    qp, op = _take(dev, "q", q, rows, qd), _take(dev, "out", out, rows, qd)
    lp = _take(dev, "lse", lse, rows[:2], torch.float32)
    kpool, vpool, ksc, vsc, pt, sl, st = _take_cache(dev, p, k_pool, v_pool, k_scale, v_scale, page_table,
                                                     seq_lens, q_start)
    _call(dev, LIB.paged_chunk_attention, "paged_chunk_attention", ws, stream, ctypes.byref(p), T, qp, st, kpool, vpool,
          ksc, vsc, pt, sl, op, lp)


def paged_attention_mass(p, q, q_start, k_pool, k_scale, page_table, seq_lens, lse, mass_in, mass_out,
                         decay=1.0, ws=None, stream=None):
    dev, T, rows = _device(ws), q.shape[0], (q.shape[0], p.num_q_heads, p.head_dim)
    m = (p.batch, p.num_kv_heads, p.max_pages_per_seq * p.page_size)
    qp, lp = _take(dev, "q", q, rows, _ELEM[p.q_dtype]), _take(dev, "lse", lse, rows[:2], torch.float32)
    mi, mo = _take(dev, "mass_in", mass_in, m, torch.float32), _take(dev, "mass_out", mass_out, m, torch.float32)
    kpool, _, ksc, _, pt, sl, st = _take_cache(dev, p, k_pool, None, k_scale, None, page_table, seq_lens, q_start)
    _call(dev, LIB.paged_attention_mass, "paged_attention_mass", ws, stream, ctypes.byref(p), T, qp, st, kpool, ksc, pt,
          sl, lp, mi, mo, float(decay))


def paged_cache_evict(p, mass, keep, n_sink, n_recent, k_pool, v_pool, k_scale, v_scale, page_table,
                      dst_page_table, seq_lens, kept, new_lens, mass_out, ws=None, stream=None):
    dev, m, keep = _device(ws), (p.batch, p.num_kv_heads, p.max_pages_per_seq * p.page_size), int(keep)
    mi, mo = _take(dev, "mass", mass, m, torch.float32), _take(dev, "mass_out", mass_out, m, torch.float32)
    kpool, vpool, ksc, vsc, pt, sl, _ = _take_cache(dev, p, k_pool, v_pool, k_scale, v_scale, page_table, seq_lens)
    dst = _take(dev, "dst_page_table", dst_page_table, (p.batch, p.max_pages_per_seq), torch.int32)
    kp = _take(dev, "kept", kept, (p.batch, p.num_kv_heads, keep), torch.int32)
    nl = _take(dev, "new_lens", new_lens, (p.batch,), torch.int32)
    _call(dev, LIB.paged_cache_evict, "paged_cache_evict", ws, stream, ctypes.byref(p), mi, keep, int(n_sink),
          int(n_recent), kpool, vpool, ksc, vsc, pt, dst, sl, kp, nl, mo)


# ---- attention over a paged cache of latent vectors ----------------------------------
def spg_latent_validate(p: spg_latent_params) -> int:
    return LIB.spg_latent_validate(ctypes.byref(p))


def spg_latent_workspace_size(p: spg_latent_params, total_q: int) -> int:
    n = c_size_t(0)
    _check(LIB.spg_latent_workspace_size(ctypes.byref(p), int(total_q), ctypes.byref(n)), "spg_latent_workspace_size")
    return n.value


def _take_latent(dev, p, pool, page_table, seq_lens, q_start):
    return (_take(dev, "pool", pool, (p.num_phys_pages, p.page_size, p.latent_dim + p.rope_dim), _ELEM[p.dtype]),
            _take(dev, "page_table", page_table, (p.batch, p.max_pages_per_seq), torch.int32),
            _take(dev, "seq_lens", seq_lens, (p.batch,), torch.int32),
            _take(dev, "q_start", q_start, (p.batch + 1,), torch.int32))


def _take_2d(dev, name, t, shape, dtype):
    """Pointer and row stride of a matrix whose rows are contiguous."""
    if t is None:
        return None, 0
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _refuse(name, t, shape, dtype, dev)
    row, one = t.stride()
    if t.numel() and one != 1:
        raise ValueError(f"{name}: the channels of one token have to be contiguous")
    return t.data_ptr(), row if shape[0] > 1 else shape[1]


def _call_rows(dev, fn, where, stream, *args):
    """fn(*args, stream) with device `dev` current, for entry points without a workspace."""
    if dev < 0:
        raise ValueError("libspg takes device tensors")
    if stream is None:
        stream = _raw_stream(dev)
    if _one_device() or dev == torch.cuda.current_device():
        _check(fn(*args, stream), where)
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, stream), where)


def paged_latent_append(p, rope, c, k_pe, norm_weight, eps, q, q_start, page_table, seq_lens, pool, q_lat=None,
                        positions=None, ws=None, stream=None):
    dev, T, r, dr, dt = _device(ws), c.shape[0], p.latent_dim, p.rope_dim, _ELEM[p.dtype]
    cp, cs = _take_2d(dev, "c", c, (T, r), dt)
    kp, ks = _take_2d(dev, "k_pe", k_pe, (T, dr), dt)
    wp = _take(dev, "norm_weight", norm_weight, (r,), dt)
    qp, qs = _take_rows(dev, "q", q, (T, p.num_heads, p.nope_dim + dr), dt)
    lp = _take(dev, "q_lat", q_lat, (T, p.num_heads, r + dr), dt)
    pos = _take(dev, "positions", positions, (T,), torch.int32)
    pl, pt, sl, st = _take_latent(dev, p, pool, page_table, seq_lens, q_start)
    _call(dev, LIB.paged_latent_append, "paged_latent_append", ws, stream, ctypes.byref(p),
          None if rope is None else ctypes.byref(rope), T, cp, cs, kp, ks, wp, float(eps), qp, qs, st, pos, pt, sl, pl, lp)


def latent_absorb(p, q, w_kv, q_lat, stream=None):
    dev, T, H, r, dt = q_lat.get_device(), q.shape[0], p.num_heads, p.latent_dim, _ELEM[p.dtype]
    qp, qs = _take_rows(dev, "q", q, (T, H, p.nope_dim + p.rope_dim), dt)
    wp = _take(dev, "w_kv", w_kv, (H, p.nope_dim + p.v_dim, r), dt)
    lp = _take(dev, "q_lat", q_lat, (T, H, r + p.rope_dim), dt)
    _call_rows(dev, LIB.latent_absorb, "latent_absorb", stream, ctypes.byref(p), T, qp, qs, wp, lp)


def paged_latent_attention(p, q_lat, q_start, pool, page_table, seq_lens, o_lat, lse=None, ws=None, stream=None):
    dev, T, H, r, dt = _device(ws), q_lat.shape[0], p.num_heads, p.latent_dim, _ELEM[p.dtype]
    qp = _take(dev, "q_lat", q_lat, (T, H, r + p.rope_dim), dt)
    op, lp = _take(dev, "o_lat", o_lat, (T, H, r), dt), _take(dev, "lse", lse, (T, H), torch.float32)
    pl, pt, sl, st = _take_latent(dev, p, pool, page_table, seq_lens, q_start)
    _call(dev, LIB.paged_latent_attention, "paged_latent_attention", ws, stream, ctypes.byref(p), T, qp, st, pl, pt, sl,
          op, lp)


def latent_project(p, o_lat, w_kv, out, stream=None):
    dev, T, H, r, dt = out.get_device(), o_lat.shape[0], p.num_heads, p.latent_dim, _ELEM[p.dtype]
    ip = _take(dev, "o_lat", o_lat, (T, H, r), dt)
    wp = _take(dev, "w_kv", w_kv, (H, p.nope_dim + p.v_dim, r), dt)
    op = _take(dev, "out", out, (T, H, p.v_dim), dt)
    _call_rows(dev, LIB.latent_project, "latent_project", stream, ctypes.byref(p), T, ip, wp, op)


def spg_read_device_error(ws, stream=None) -> int:
    bits = c_int32(0)
    _check(LIB.spg_read_device_error(_ptr(ws), ctypes.byref(bits), _stream(stream)),
           "spg_read_device_error")
    return bits.value


def spg_clear_device_error(ws, stream=None):
    _check(LIB.spg_clear_device_error(_ptr(ws), _stream(stream)), "spg_clear_device_error")


def spg_test_withhold_first_stage(ws, stream=None):
    _check(LIB.spg_test_withhold_first_stage(_ptr(ws), _stream(stream)), "spg_test_withhold_first_stage")
