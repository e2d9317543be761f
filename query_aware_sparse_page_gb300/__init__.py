"""Query-aware sparse-page decode attention for GB300 (sm_103a).

The computation lives in libspg.so (hand-written CUDA, C ABI declared in
include/spg.h); this package is its ctypes binding plus device-buffer
helpers that only allocate (with torch) and never compute.
"""

from .binding import (  # noqa: F401
    BF16, DEVERR_PAGE_ID, DEVERR_Q_START, DEVERR_SEL, DEVERR_SEQ_LEN, DEVERR_TIMEOUT, F16, I8, LIB, LIB_PATH,
    SEL_ALL, SEL_QUEST, SEL_SKETCH_INT4, SpgError, dense_decode_attention, latent_absorb, latent_project, make_latent_params,
    make_params, make_rope, paged_attention_mass, paged_cache_evict, paged_chunk_attention, paged_latent_append,
    paged_latent_attention, paged_rope_append,
    sparse_decode_attention, sparse_decode_select_attend, sparse_decode_step, sparse_page_meta_update,
    sparse_page_score, sparse_page_select, sparse_page_sketch_dots, spg_abi_version, spg_chunk_workspace_size,
    spg_clear_device_error, spg_latent_params, spg_latent_validate, spg_latent_workspace_size, spg_params, spg_rope, spg_rope_freqs,
    spg_read_device_error, spg_status_str, spg_test_withhold_first_stage, spg_validate, spg_workspace_size, status_str,
    STEP_KERNEL_AUTO, STEP_KERNEL_CLUSTER, STEP_KERNEL_SCHED, spg_prefer_dense, spg_set_chunk_parts, spg_set_step_kernel,
    spg_step_kernel, spg_step_launches, step_kernel_name, step_launch_count,
)
from .buffers import DecodeBuffers, alloc_buffers, params_for  # noqa: F401
