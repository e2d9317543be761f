// A chunk's latent vectors and rotary keys into the pages of the cache, and
// the rotated part of its queries beside the absorbed one, one launch
// (paged_latent_append).
//
//   pool row = [ c * (mean(c^2) + eps)^-1/2 * w | k_pe turned ]
//   q_lat[h][r:] = q[h][dn:] turned
//
// The turn is that of paged_rope_append: the angle as a 64-bit fraction of a
// turn, its upper 32 bits to sincospif.
//
// Bound by bytes, and for one token per sequence by latency.  A CTA takes a
// token: its first warp the latent vector (one or two 16-byte pieces a lane,
// one shuffle sum) and the key, the others 16 channels of a query head at a
// time.  No warp waits for another: each finds the token's position by itself
// and has the 32 pairs' cos and sin in its lanes; the values are on their way
// before the position is known (8192 tokens: 20 us, 23 the other way round).
//
// Measured (GB300): 8192 tokens of 32 heads, 86 MB: 20 us, 4.3 TB/s (a copy of
// the same bytes, the queries' pieces of 128 bytes at a stride and the rows in
// two launches: 12.8 + 4.4 us); 16 tokens: 2.3 us back to back.
#include <cmath>

#include "spg_chunk_common.cuh"
#include "spg_latent.h"

namespace spg {
namespace {

constexpr int kThreads = 160;  // a warp for the latent vector and the key, 128 threads for the queries' items
constexpr int kRope = 64, kPairs = kRope / 2;

struct AppendArgs {
  unsigned long long turns[kPairs];  // angle per position, 64-bit fraction of a turn
  const void *c, *k_pe, *w, *q;
  int64_t c_stride, kpe_stride, q_stride;
  const int32_t *q_start, *positions, *page_table, *seq_lens;
  void *pool, *q_lat;
  int32_t* err;
  float mscale, eps;
  int B, H, S, s_log2, MP, n_phys, total_q, rot, nope;
};

template <typename T, int R, bool HALF>
__global__ void __launch_bounds__(kThreads) k_latent_append(const __grid_constant__ AppendArgs a) {
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rot_items = a.rot / 16;
  constexpr int kPieces = R / 256;  // 16-byte pieces of the latent vector a lane has
  uint4 u[kPieces];
  // an item is 16 channels of a head (h = -1: the key), as the two 16-byte pieces that hold both halves of its pairs
  struct Item {
    int h, c0, c1, j;
    uint4 w0, w1;
  };
  const auto load_item = [&](int h, int j) {
    Item it;
    it.h = h;
    it.j = j;
    it.c0 = HALF && j < rot_items ? j : 2 * j;
    it.c1 = HALF && j < rot_items ? j + rot_items : 2 * j + 1;
    const T* src = h < 0 ? static_cast<const T*>(a.k_pe) + t * a.kpe_stride
                         : static_cast<const T*>(a.q) + t * a.q_stride + static_cast<size_t>(h) * (a.nope + kRope) + a.nope;
    it.w0 = *reinterpret_cast<const uint4*>(src + 8 * it.c0);
    it.w1 = *reinterpret_cast<const uint4*>(src + 8 * it.c1);
    return it;
  };
  const int items = a.q ? 4 * a.H : 0;
  pdl_wait();
  // the row's values first: they do not wait for its place
  int i = static_cast<int>(threadIdx.x) - 32;
  Item it{};
  if (warp == 0) {
    const T* src = static_cast<const T*>(a.c) + t * a.c_stride;
#pragma unroll
    for (int x = 0; x < kPieces; ++x) u[x] = *reinterpret_cast<const uint4*>(src + 8 * (lane + 32 * x));
    it = load_item(-1, lane & 3);
  } else if (i < items) {
    it = load_item(i >> 2, i & 3);
  }
  // the sequence with q_start[b] <= t < q_start[b + 1]; an unsorted q_start ends at some b, checked below
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_start[mid] <= t) lo = mid; else hi = mid;
  }
  int32_t bad = 0;
  // empty sequences before the row's own share its start: the last of them is the one found
  const ChunkSeq s = chunk_seq(a.q_start, a.seq_lens, lo, a.total_q, a.MP * a.S, bad);
  const bool mine = t >= s.start && t < s.start + s.n;
  const int pos = s.pos0 + t - s.start;
  int page = -1;
  if (warp == 0 && mine) {
    page = a.page_table[static_cast<size_t>(lo) * a.MP + (pos >> a.s_log2)];
    if (page < 0 || page >= a.n_phys) {
      bad |= SPG_DEVERR_PAGE_ID;
      page = -1;
    }
  }
  if (bad && threadIdx.x == 0) record_error(a.err, bad);
  pdl_trigger();
  if (!mine) return;  // a row of no sequence

  // the 32 pairs' cos and sin, one a lane
  const unsigned long long at = static_cast<unsigned long long>(static_cast<long long>(a.positions ? a.positions[t] : pos));
  const unsigned long long f = at * a.turns[lane];
  // nearest 2^-32 of a turn, as half-turns in [-1, 1)
  const int w = static_cast<int>(static_cast<uint32_t>((f + 0x80000000ull) >> 32));
  float sn, cs;
  sincospif(static_cast<float>(w) * 4.656612873077393e-10f, &sn, &cs);
  sn *= a.mscale;
  cs *= a.mscale;
  const auto turn = [&](const Item& it, T* dst, bool live) {  // a whole warp
    float x[8], y[8];
    unpack8<T>(it.w0, x);
    unpack8<T>(it.w1, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = __shfl_sync(0xffffffffu, cs, 8 * it.j + e), n = __shfl_sync(0xffffffffu, sn, 8 * it.j + e);
      if (it.j < rot_items) {
        // half: (x[e], y[e]); interleaved: neighbours within a piece
        float& p = HALF ? x[e] : (e < 4 ? x[2 * e] : y[2 * e - 8]);
        float& q = HALF ? y[e] : (e < 4 ? x[2 * e + 1] : y[2 * e - 7]);
        const float v = p * c - q * n, z = q * c + p * n;
        p = v;
        q = z;
      }
    }
    if (live) {
      *reinterpret_cast<uint4*>(dst + 8 * it.c0) = pack8<T>(x);
      *reinterpret_cast<uint4*>(dst + 8 * it.c1) = pack8<T>(y);
    }
  };

  if (warp == 0) {
    T* const row = static_cast<T*>(a.pool) + (static_cast<size_t>(page < 0 ? 0 : page) * a.S + (pos & (a.S - 1))) * (R + kRope);
    if (a.w) {
      float x[8], g[8], sum = 0.f;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        unpack8<T>(u[k], x);
        float q = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(x[e], x[e], q);
        sum += q;
      }
      const float r = rsqrtf(warp_sum(sum) * (1.f / R) + a.eps);
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        unpack8<T>(u[k], x);
        unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.w) + 8 * (lane + 32 * k)), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * r * g[e];
        u[k] = pack8<T>(x);
      }
    }
    if (page >= 0) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) *reinterpret_cast<uint4*>(row + 8 * (lane + 32 * k)) = u[k];
    }
    turn(it, row + R, page >= 0 && lane < 4);
    return;
  }
  while (i - lane < items) {
    const bool live = i < items;
    turn(it, static_cast<T*>(a.q_lat) + (static_cast<size_t>(t) * a.H + it.h) * (R + kRope) + R, live);
    i += kThreads - 32;
    if (i < items) it = load_item(i >> 2, i & 3);
  }
}

template <typename T>
cudaError_t append_typed(const spg_latent_params& p, const AppendArgs& a, bool half, cudaStream_t st) {
  const dim3 grid(a.total_q), block(kThreads);
  if (p.latent_dim == 512)
    return half ? launch_pdl(k_latent_append<T, 512, true>, grid, block, 0, st, a)
                : launch_pdl(k_latent_append<T, 512, false>, grid, block, 0, st, a);
  return half ? launch_pdl(k_latent_append<T, 256, true>, grid, block, 0, st, a)
              : launch_pdl(k_latent_append<T, 256, false>, grid, block, 0, st, a);
}

}  // namespace

cudaError_t launch_latent_append(const spg_latent_params& p, const spg_rope* rope, const double* inv_freq, double mscale,
                                 const LatentAppend& r, int32_t* err, cudaStream_t stream) {
  AppendArgs a{};
  a.mscale = 1.f;
  bool half = true;
  if (rope) {
    a.rot = rope->rot_dim == 0 ? kRope : rope->rot_dim;
    for (int i = 0; i < a.rot / 2; ++i)
      a.turns[i] = static_cast<unsigned long long>(std::ldexp(inv_freq[i] / 6.283185307179586476925, 64));
    a.mscale = static_cast<float>(mscale);
    half = rope->layout == SPG_ROPE_HALF;
  }
  a.c = r.c;
  a.k_pe = r.k_pe;
  a.w = r.norm_weight;
  a.q = r.q;
  a.c_stride = r.c_stride;
  a.kpe_stride = r.kpe_stride;
  a.q_stride = r.q_stride;
  a.q_start = r.q_start;
  a.positions = r.positions;
  a.page_table = r.page_table;
  a.seq_lens = r.seq_lens;
  a.pool = r.pool;
  a.q_lat = r.q_lat;
  a.err = err;
  a.eps = r.eps;
  a.B = p.batch;
  a.H = p.num_heads;
  a.S = p.page_size;
  a.s_log2 = log2_of(p.page_size);
  a.MP = p.max_pages_per_seq;
  a.n_phys = p.num_phys_pages;
  a.total_q = r.total_q;
  a.nope = p.nope_dim;
  return p.dtype == SPG_F16 ? append_typed<__half>(p, a, half, stream) : append_typed<__nv_bfloat16>(p, a, half, stream);
}

}  // namespace spg
