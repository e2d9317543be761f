// Attention weight received by every cached token (paged_attention_mass).
//
// S^T = K Q^T with 64 tokens as the rows: a lane sums exp(scale s - lse) over
// the query columns it holds, so a token's mass needs no atomics and its
// order of summation is fixed.
#include <cmath>

#include "spg_chunk_common.cuh"
#include "spg_internal.h"

namespace spg {
namespace {

constexpr int kRows = 64;   // rows of a tile
constexpr int kTok = 64;    // tokens per step
constexpr int kThreads = 128;

// Shared tile of 16-bit rows of D channels: 16-byte piece c of row r at c ^ (r % 8).
template <int D>
__device__ __forceinline__ uint32_t tile_at(uint32_t base, int r, int c) {
  return base + r * (D * 2) + ((c ^ (r & 7)) << 4);
}

// `rows` tokens from t0 of one (batch, kv-head) into a tile, int8 codes as
// exact 16-bit values; tokens at or past `end`, or of a bad page, are zeros
// and their mask entry (and scale) says so.
template <typename T, typename TQ, int D, int ROWS, int THREADS>
__device__ __forceinline__ void load_tokens(const T* pool, const __half* scale, const int32_t* pt, int Hkv, int h,
                                            int S, int n_phys, int t0, int end, uint8_t* tile, float* s_scale,
                                            int32_t* err) {
  constexpr int CPR = D / 8;
  for (int i = threadIdx.x; i < ROWS * CPR; i += THREADS) {
    const int r = i / CPR, c = i % CPR, t = t0 + r;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    float sc = 0.f;
    if (t < end) {
      const int page = pt[t / S];
      if (page >= 0 && page < n_phys) {
        const size_t row = (static_cast<size_t>(page) * Hkv + h) * S + t % S;
        sc = 1.f;
        if constexpr (sizeof(T) == 1) {
          if (scale) sc = __half2float(scale[row]);
          float x[8];
          load_cvt<int8_t, 8>(reinterpret_cast<const int8_t*>(pool) + row * D + 8 * c, x);
          w = make_uint4(pack2<TQ>(x[0], x[1]), pack2<TQ>(x[2], x[3]), pack2<TQ>(x[4], x[5]), pack2<TQ>(x[6], x[7]));
        } else {
          w = *reinterpret_cast<const uint4*>(pool + row * D + 8 * c);
        }
      } else if (c == 0) {
        record_error(err, SPG_DEVERR_PAGE_ID);
        sc = -1.f;
      } else {
        sc = -1.f;
      }
    }
    *reinterpret_cast<uint4*>(tile + r * (D * 2) + ((c ^ (r & 7)) << 4)) = w;
    if (c == 0 && s_scale) s_scale[r] = sc;  // negative: bad page
  }
}

struct MassArgs {
  const void *q, *k_pool;
  const __half* k_scale;
  const int32_t *q_start, *page_table, *seq_lens;
  const float *lse, *mass_in;
  float* mass_out;
  int32_t* err;
  int B, Hkv, S, MP, n_phys, total_q;
  float scale_log2, decay;
};

template <typename T, typename TQ, int D, int G>
__global__ void __launch_bounds__(kThreads) k_mass(const __grid_constant__ MassArgs a) {
  constexpr int KS = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* s_k = smem;
  uint8_t* s_q = smem + kTok * D * 2;
  __shared__ float s_ks[kTok], s_lse[kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.y, b = unit / a.Hkv, h = unit % a.Hkv, t0 = blockIdx.x * kTok, Hq = a.Hkv * G;
  pdl_wait();
  int32_t bad = 0;
  const ChunkSeq sq = chunk_seq(a.q_start, a.seq_lens, b, a.total_q, a.MP * a.S, bad);
  if (bad && blockIdx.x == 0 && threadIdx.x == 0) record_error(a.err, bad);
  if (t0 >= sq.L) return;
  load_tokens<T, TQ, D, kTok, kThreads>(static_cast<const T*>(a.k_pool), a.k_scale,
                                        a.page_table + static_cast<size_t>(b) * a.MP, a.Hkv, h, a.S, a.n_phys, t0, sq.L,
                                        s_k, s_ks, a.err);
  __syncthreads();
  const int g = lane >> 2, tq = lane & 3, mi = lane >> 3, r8 = lane & 7;
  uint32_t ka[KS][4];
  const uint32_t kb = smem_u32(s_k), qb = smem_u32(s_q);
#pragma unroll
  for (int j = 0; j < KS; ++j) ldmatrix_x4(ka[j], tile_at<D>(kb, warp * 16 + (mi & 1) * 8 + r8, 2 * j + (mi >> 1)));
  float ks[2], sum[2] = {0.f, 0.f};
  int tok[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    tok[e] = t0 + warp * 16 + g + 8 * e;
    ks[e] = s_ks[warp * 16 + g + 8 * e];
  }
  // rows that see at least the tile's first token
  const int first = max(0, t0 - sq.pos0) * G;
  for (int r0 = first; r0 < sq.n * G; r0 += kRows) {
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * (D / 8); i += kThreads) {
      const int r = i / (D / 8), c = i % (D / 8), rr = r0 + r;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      const size_t row = static_cast<size_t>(sq.start + rr / G) * Hq + h * G + rr % G;
      if (rr < sq.n * G) w = *reinterpret_cast<const uint4*>(static_cast<const TQ*>(a.q) + row * D + 8 * c);
      *reinterpret_cast<uint4*>(s_q + r * (D * 2) + ((c ^ (r & 7)) << 4)) = w;
      if (c == 0) {
        const float e = rr < sq.n * G ? a.lse[row] : -INFINITY;
        s_lse[r] = e == -INFINITY ? INFINITY : e * kLog2e;
      }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kRows / 16; ++n) {
      float s[2][4] = {};
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        uint32_t r[4];
        ldmatrix_x4(r, tile_at<D>(qb, n * 16 + (mi >> 1) * 8 + r8, 2 * j + (mi & 1)));
        mma_16816<TQ>(s[0], ka[j], r[0], r[1]);
        mma_16816<TQ>(s[1], ka[j], r[2], r[3]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = n * 16 + i * 8 + 2 * tq + (e & 1);
          const float k = sizeof(T) == 1 ? ks[e >> 1] * a.scale_log2 : a.scale_log2;
          if (tok[e >> 1] <= sq.pos0 + (r0 + c) / G) sum[e >> 1] += exp2f(fmaf(s[i][e], k, -s_lse[c]));
        }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
    if (tq == 0 && tok[e] < sq.L) {
      const size_t at = static_cast<size_t>(unit) * a.MP * a.S + tok[e];
      float old = 0.f;
      if (a.mass_in && a.decay > 0.f && tok[e] < sq.pos0) old = a.mass_in[at] * a.decay;
      a.mass_out[at] = old + (ks[e] < 0.f ? 0.f : sum[e]);
    }
  }
}

template <typename T, typename TQ, int D, int G>
cudaError_t mass_typed(const spg_params& p, const MassArgs& a, cudaStream_t st) {
  const auto kern = k_mass<T, TQ, D, G>;
  const size_t smem = (kTok + kRows) * D * 2;
  const cudaError_t e = ensure_smem(kern, smem);
  if (e != cudaSuccess) return e;
  const int tiles = static_cast<int>((static_cast<long long>(p.max_pages_per_seq) * p.page_size + kTok - 1) / kTok);
  return launch_pdl(kern, dim3(tiles, p.batch * p.num_kv_heads), dim3(kThreads), smem, st, a);
}

#define SPG_DG(FN, T, TQ)                                            \
  switch (p.head_dim * 16 + p.num_q_heads / p.num_kv_heads) {        \
    case 128 * 16 + 1: return FN<T, TQ, 128, 1>(p, a, stream);       \
    case 128 * 16 + 2: return FN<T, TQ, 128, 2>(p, a, stream);       \
    case 128 * 16 + 4: return FN<T, TQ, 128, 4>(p, a, stream);       \
    case 128 * 16 + 8: return FN<T, TQ, 128, 8>(p, a, stream);       \
    case 64 * 16 + 1: return FN<T, TQ, 64, 1>(p, a, stream);         \
    case 64 * 16 + 2: return FN<T, TQ, 64, 2>(p, a, stream);         \
    case 64 * 16 + 4: return FN<T, TQ, 64, 4>(p, a, stream);         \
    case 64 * 16 + 8: return FN<T, TQ, 64, 8>(p, a, stream);         \
    default: return cudaErrorInvalidValue;                           \
  }
#define SPG_TYPES(FN)                                                \
  if (p.kv_dtype == SPG_F16) { SPG_DG(FN, __half, __half) }          \
  if (p.kv_dtype == SPG_BF16) { SPG_DG(FN, __nv_bfloat16, __nv_bfloat16) } \
  if (p.q_dtype == SPG_F16) { SPG_DG(FN, int8_t, __half) }           \
  SPG_DG(FN, int8_t, __nv_bfloat16)

float scale_log2(const spg_params& p) {
  return (p.softmax_scale > 0.f ? p.softmax_scale : 1.0f / sqrtf(static_cast<float>(p.head_dim))) * kLog2e;
}

}  // namespace

cudaError_t launch_mass(const spg_params& p, const ChunkRows& r, const void* k_pool, const void* k_scale,
                        const float* lse, const float* mass_in, float* mass_out, float decay, const Workspace& ws,
                        cudaStream_t stream) {
  MassArgs a{};
  a.q = r.q;
  a.k_pool = k_pool;
  a.k_scale = static_cast<const __half*>(k_scale);
  a.q_start = r.q_start;
  a.page_table = r.page_table;
  a.seq_lens = r.seq_lens;
  a.lse = lse;
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  a.err = ws.err;
  a.B = p.batch;
  a.Hkv = p.num_kv_heads;
  a.S = p.page_size;
  a.MP = p.max_pages_per_seq;
  a.n_phys = p.num_phys_pages;
  a.total_q = r.total_q;
  a.scale_log2 = scale_log2(p);
  a.decay = decay;
  SPG_TYPES(mass_typed)
}

}  // namespace spg
