// Launchers of the latent-cache operators (spg_latent_append.cu,
// spg_latent_heads.cu, spg_latent_attention.cu), for the C ABI layer.
#pragma once

#include "spg_internal.h"

namespace spg {

struct LatentRows {
  const int32_t *q_start, *page_table, *seq_lens;
  int total_q;
};
struct LatentAppend : LatentRows {
  const void *c, *k_pe, *norm_weight, *q;
  int64_t c_stride, kpe_stride, q_stride;
  const int32_t* positions;
  float eps;
  void *pool, *q_lat;
};

// 16-bit values in whose sum a probability enters the second product (spg_set_chunk_parts)
int chunk_parts();

// encode_tmap of 16-bit elements
bool make_tmap16(CUtensorMap* map, int dtype, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                 const uint32_t* box);

// rope (may be NULL) with what rope_freqs gave for it
cudaError_t launch_latent_append(const spg_latent_params& p, const spg_rope* rope, const double* inv_freq, double mscale,
                                 const LatentAppend& r, int32_t* err, cudaStream_t stream);
// project: x = o_lat [total_q][H][r] times W_uv, else x = q (rows q_stride apart) times W_uk
cudaError_t launch_latent_heads(const spg_latent_params& p, bool project, int total_q, const void* x, int64_t x_stride,
                                const void* w_kv, void* y, cudaStream_t stream);
size_t latent_workspace_bytes(const spg_latent_params& p, int total_q);
cudaError_t launch_latent_attention(const spg_latent_params& p, const LatentRows& r, const void* q_lat, const void* pool,
                                    void* o_lat, float* lse, int parts, void* ws, size_t ws_bytes, cudaStream_t stream);

}  // namespace spg
