// C ABI of the latent-cache operators: parameter and argument checks.  All
// device work is in the kernel files.
#include <cmath>
#include <cstdint>

#include "spg_latent.h"

namespace spg {

bool make_tmap16(CUtensorMap* map, int dtype, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                 const uint32_t* box) {
  return encode_tmap(map, dtype == SPG_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, base,
                     dims, strides, box);
}

}  // namespace spg

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_ptr(const void* p) { return p != nullptr && aligned16(p); }
spg_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SPG_OK : SPG_ECUDA; }

// rows of a chunk, whose heads' rows are counted in 32 bits
spg_status check_rows(const spg_latent_params* p, int32_t total_q) {
  const spg_status s = spg_latent_validate(p);
  if (s != SPG_OK) return s;
  if (total_q < 0) return SPG_EINVAL;
  return static_cast<int64_t>(total_q) * p->num_heads > INT32_MAX - 128 ? SPG_EUNSUPPORTED : SPG_OK;
}
spg_status check_ws(const spg_latent_params* p, int32_t total_q, const void* ws, size_t ws_bytes) {
  if (!ok_ptr(ws)) return SPG_EINVAL;
  return ws_bytes < spg::latent_workspace_bytes(*p, total_q) ? SPG_EWORKSPACE : SPG_OK;
}
int64_t q_row(const spg_latent_params* p) { return static_cast<int64_t>(p->num_heads) * (p->nope_dim + p->rope_dim); }

}  // namespace

extern "C" {

spg_status spg_latent_validate(const spg_latent_params* p) {
  if (!p) return SPG_EINVAL;
  if (p->batch < 1 || p->num_heads < 1) return SPG_EINVAL;
  if (p->latent_dim < 64 || p->latent_dim % 64 || p->rope_dim < 16 || p->rope_dim % 16) return SPG_EINVAL;
  if (p->nope_dim < 16 || p->nope_dim % 16 || p->v_dim < 16 || p->v_dim % 16) return SPG_EINVAL;
  if (p->page_size < 8 || p->page_size > 128 || (p->page_size & (p->page_size - 1))) return SPG_EINVAL;
  if (p->num_phys_pages < 1 || p->max_pages_per_seq < 1) return SPG_EINVAL;
  if (static_cast<int64_t>(p->max_pages_per_seq) * p->page_size > INT32_MAX - 128) return SPG_EINVAL;
  if (p->dtype < SPG_F16 || p->dtype > SPG_I8) return SPG_EINVAL;
  if (!(p->softmax_scale >= 0.f) || std::isinf(p->softmax_scale)) return SPG_EINVAL;
  // valid, but not built
  if (p->num_heads > 1024) return SPG_EUNSUPPORTED;
  if ((p->latent_dim != 256 && p->latent_dim != 512) || p->rope_dim != 64) return SPG_EUNSUPPORTED;
  if ((p->nope_dim != 64 && p->nope_dim != 128) || (p->v_dim != 64 && p->v_dim != 128)) return SPG_EUNSUPPORTED;
  if (p->page_size < 16 || p->dtype == SPG_I8) return SPG_EUNSUPPORTED;
  // the pool's groups of 8 tokens are counted in 32 bits
  if (static_cast<int64_t>(p->num_phys_pages) * (p->page_size / 8) > INT32_MAX) return SPG_EUNSUPPORTED;
  return SPG_OK;
}

spg_status spg_latent_workspace_size(const spg_latent_params* p, int32_t total_q, size_t* bytes) {
  const spg_status s = check_rows(p, total_q);
  if (s != SPG_OK) return s;
  if (!bytes) return SPG_EINVAL;
  *bytes = spg::latent_workspace_bytes(*p, total_q);
  return SPG_OK;
}

spg_status paged_latent_append(const spg_latent_params* p, const spg_rope* rope, int32_t total_q, const void* c,
                               int64_t c_stride, const void* k_pe, int64_t kpe_stride, const void* norm_weight,
                               float eps, const void* q, int64_t q_stride, const int32_t* q_start,
                               const int32_t* positions, const int32_t* page_table, const int32_t* seq_lens, void* pool,
                               void* q_lat, void* ws, size_t ws_bytes, spg_stream_t stream) {
  spg_status s = check_rows(p, total_q);
  if (s != SPG_OK) return s;
  double inv[32], m = 1.0;  // rope_dim / 2 pairs
  if (rope) {
    if (!spg::rope_freqs(*rope, p->rope_dim, inv, &m)) return SPG_EINVAL;
    if (rope->rot_dim % 16) return SPG_EUNSUPPORTED;  // whole 16-byte pieces of both halves
  }
  if (!(eps >= 0.f) || std::isinf(eps)) return SPG_EINVAL;
  if ((s = check_ws(p, total_q, ws, ws_bytes)) != SPG_OK) return s;
  if (total_q == 0) return SPG_OK;
  if (!ok_ptr(c) || !ok_ptr(k_pe) || !aligned16(norm_weight) || !aligned16(q) || !aligned16(q_lat) ||
      (q == nullptr) != (q_lat == nullptr) || (q && q == q_lat) || !ok_ptr(q_start) || !aligned16(positions) ||
      !ok_ptr(page_table) || !ok_ptr(seq_lens) || !ok_ptr(pool))
    return SPG_EINVAL;
  if (c_stride < p->latent_dim || c_stride % 8 || kpe_stride < p->rope_dim || kpe_stride % 8) return SPG_EINVAL;
  if (q && (q_stride < q_row(p) || q_stride % 8)) return SPG_EINVAL;
  spg::LatentAppend r{};
  r.q_start = q_start;
  r.page_table = page_table;
  r.seq_lens = seq_lens;
  r.total_q = total_q;
  r.c = c;
  r.k_pe = k_pe;
  r.norm_weight = norm_weight;
  r.q = q;
  r.c_stride = c_stride;
  r.kpe_stride = kpe_stride;
  r.q_stride = q_stride;
  r.positions = positions;
  r.eps = eps;
  r.pool = pool;
  r.q_lat = q_lat;
  return cuda_status(spg::launch_latent_append(*p, rope, inv, m, r, static_cast<int32_t*>(ws), reinterpret_cast<cudaStream_t>(stream)));
}

spg_status latent_absorb(const spg_latent_params* p, int32_t total_q, const void* q, int64_t q_stride, const void* w_kv,
                         void* q_lat, spg_stream_t stream) {
  const spg_status s = check_rows(p, total_q);
  if (s != SPG_OK) return s;
  if (total_q == 0) return SPG_OK;
  if (!ok_ptr(q) || !ok_ptr(w_kv) || !ok_ptr(q_lat) || q == q_lat) return SPG_EINVAL;
  if (q_stride < q_row(p) || q_stride % 8) return SPG_EINVAL;
  return cuda_status(spg::launch_latent_heads(*p, false, total_q, q, q_stride, w_kv, q_lat, reinterpret_cast<cudaStream_t>(stream)));
}

spg_status latent_project(const spg_latent_params* p, int32_t total_q, const void* o_lat, const void* w_kv, void* out,
                          spg_stream_t stream) {
  const spg_status s = check_rows(p, total_q);
  if (s != SPG_OK) return s;
  if (total_q == 0) return SPG_OK;
  if (!ok_ptr(o_lat) || !ok_ptr(w_kv) || !ok_ptr(out) || o_lat == out) return SPG_EINVAL;
  return cuda_status(spg::launch_latent_heads(*p, true, total_q, o_lat, static_cast<int64_t>(p->num_heads) * p->latent_dim,
                                              w_kv, out, reinterpret_cast<cudaStream_t>(stream)));
}

spg_status paged_latent_attention(const spg_latent_params* p, int32_t total_q, const void* q_lat, const int32_t* q_start,
                                  const void* pool, const int32_t* page_table, const int32_t* seq_lens, void* o_lat,
                                  float* lse, void* ws, size_t ws_bytes, spg_stream_t stream) {
  spg_status s = check_rows(p, total_q);
  if (s != SPG_OK) return s;
  if ((s = check_ws(p, total_q, ws, ws_bytes)) != SPG_OK) return s;
  if (total_q == 0) return SPG_OK;
  if (!ok_ptr(q_lat) || !ok_ptr(q_start) || !ok_ptr(pool) || !ok_ptr(page_table) || !ok_ptr(seq_lens) || !ok_ptr(o_lat) ||
      !aligned16(lse) || q_lat == o_lat)
    return SPG_EINVAL;
  const spg::LatentRows r{q_start, page_table, seq_lens, total_q};
  return cuda_status(spg::launch_latent_attention(*p, r, q_lat, pool, o_lat, lse, spg::chunk_parts(), ws,
                                                  ws_bytes, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
