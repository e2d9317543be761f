"""The paged-chunk binding takes tensors of one device: the workspace's.  Stand-ins for device tensors, no GPU."""

import pytest
import torch


@pytest.fixture(scope="module")
def spg():
    import __graft_entry__

    __graft_entry__.build()
    import query_aware_sparse_page_gb300 as m

    return m


class On:
    """What the binding asks of a contiguous tensor on device `dev`; its memory is never touched."""

    def __init__(self, dev, dtype, *shape):
        self.dev, self.dtype, self.shape, self.is_cuda = dev, dtype, shape, dev >= 0

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def numel(self):
        return 1

    def element_size(self):
        return 1

    def stride(self):
        return tuple(torch.empty(self.shape, device="meta").stride())

    def data_ptr(self):
        return 1 << 20


F16, F32, I32, I8 = torch.float16, torch.float32, torch.int32, torch.int8
POOL, SCALES, TABLE, MASS = (20, 2, 16, 128), (20, 2, 16), (3, 5), (3, 2, 80)
ROWS, KV_ROWS = (7, 8, 128), (7, 2, 128)
CACHE = dict(k_pool=(I8, *POOL), v_pool=(I8, *POOL), k_scale=(F16, *SCALES), v_scale=(F16, *SCALES), page_table=(I32, *TABLE),
             seq_lens=(I32, 3))
KEYS = {n: CACHE[n] for n in ("k_pool", "k_scale", "page_table", "seq_lens")}
CALLS = {
    "paged_rope_append": dict(CACHE, q=(F16, *ROWS), k=(F16, *KV_ROWS), v=(F16, *KV_ROWS), q_start=(I32, 4), q_out=(F16, *ROWS),
                              positions=(I32, 7)),
    "paged_chunk_attention": dict(CACHE, q=(F16, *ROWS), q_start=(I32, 4), out=(F16, *ROWS), lse=(F32, 7, 8)),
    "paged_attention_mass": dict(KEYS, q=(F16, *ROWS), q_start=(I32, 4), lse=(F32, 7, 8), mass_in=(F32, *MASS),
                                 mass_out=(F32, *MASS)),
    "paged_cache_evict": dict(CACHE, mass=(F32, *MASS), dst_page_table=(I32, *TABLE), kept=(I32, 3, 2, 30), new_lens=(I32, 3),
                              mass_out=(F32, *MASS)),
}
MORE = {"paged_rope_append": dict(rope=None), "paged_cache_evict": dict(keep=30, n_sink=1, n_recent=2)}


@pytest.mark.parametrize("call, name", [(c, n) for c, names in CALLS.items() for n in names])
def test_a_tensor_on_another_device_is_refused(spg, call, name):
    p = spg.make_params(batch=3, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_phys_pages=20,
                        max_pages_per_seq=5, kv_dtype="i8", q_dtype="f16", selector="all")
    args = dict(MORE.get(call, {}), p=p, ws=On(0, torch.uint8, 1))
    for dev, says in ((1, f"{name}: on device 1, the workspace on device 0"), (-1, "device tensors")):
        tensors = {n: On(dev if n == name else 0, *spec) for n, spec in CALLS[call].items()}
        with pytest.raises(ValueError, match=says):
            getattr(spg, call)(**args, **tensors)


@pytest.mark.parametrize("call", list(CALLS))
def test_a_workspace_on_the_host_is_refused(spg, call):
    p = spg.make_params(batch=3, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_phys_pages=20,
                        max_pages_per_seq=5, kv_dtype="i8", q_dtype="f16", selector="all")
    for ws, dev in ((On(-1, torch.uint8, 1), 0), (On(-1, torch.uint8, 1), -1), (None, 0)):
        with pytest.raises(ValueError):
            getattr(spg, call)(**MORE.get(call, {}), p=p, ws=ws, **{n: On(dev, *s) for n, s in CALLS[call].items()})


def test_chunk_parts_are_one_or_two(spg):
    for bad in (0, 3, -1):
        with pytest.raises(spg.SpgError):
            spg.spg_set_chunk_parts(bad)
    spg.spg_set_chunk_parts(1)
    spg.spg_set_chunk_parts(2)
