// Rotary positions of a ragged chunk of new tokens and their keys and values
// into the pages of the cache, one launch (paged_rope_append).
//
// Pair i of a row at position t turns by the angle t * f_i:
//   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin) * mscale.
// The angle is kept as a fraction of a turn in 64-bit fixed point: with
// F_i = f_i / 2 pi * 2^64, t * F_i mod 2^64 is one integer product whose
// wrap-around is the reduction, so that far positions lose only what F_i
// itself is off by (t * 2^-54 of a turn); its upper 32 bits go to sincospif as
// a float, which rounds them to 2^-26 of a turn.
//
// Bound by bytes: every row of q, k and v is read and written once.  A CTA
// takes a few tokens: one pass computes their cos and sin into shared memory
// (each is used by every head) and resolves their cache slots, then each
// thread takes 16 channels of a head at a time, the two 16-byte pieces that
// hold both halves of its pairs.
//
// Measured (GB300): 8192 tokens of an MHA-32 prompt at d 128, fp16: 71 us for
// 403 MB, 5.7 TB/s; one token of each of 16 sequences: 6 us.
#include <cmath>

#include "spg_chunk_common.cuh"
#include "spg_internal.h"

namespace spg {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64;
constexpr int kMaxTokens = 2;  // tokens of one CTA

struct RopeArgs {
  unsigned long long turns[kMaxPairs];  // f_i / 2 pi, 64-bit fraction of a turn
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *q_start, *positions, *page_table, *seq_lens;
  void *k_pool, *v_pool, *q_out;
  __half *k_scale, *v_scale;
  int32_t* err;
  float mscale;
  int B, Hq, Hkv, S, MP, n_phys, total_q, rot, tokens;
};

template <typename T, bool I8, int D, bool HALF>
__global__ void __launch_bounds__(kThreads) k_rope_append(const __grid_constant__ RopeArgs a) {
  constexpr int IPH = D / 16;  // items of one head
  __shared__ float2 s_cs[kMaxTokens][kMaxPairs];
  __shared__ int s_page[kMaxTokens], s_slot[kMaxTokens], s_pos[kMaxTokens];
  const int t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.total_q - t0);
  pdl_wait();
  if (threadIdx.x < nt) {
    const int t = t0 + threadIdx.x;
    // the sequence with q_start[b] <= t < q_start[b + 1]; an unsorted q_start ends at some b, checked below
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.q_start[mid] <= t) lo = mid; else hi = mid;
    }
    int32_t bad = 0;
    // empty sequences before the row's own share its start: the last of them is the one found
    const ChunkSeq s = chunk_seq(a.q_start, a.seq_lens, lo, a.total_q, a.MP * a.S, bad);
    int page = -1, pos = -1;
    if (t >= s.start && t < s.start + s.n) {
      pos = s.pos0 + t - s.start;
      page = a.page_table[static_cast<size_t>(lo) * a.MP + pos / a.S];
      if (page < 0 || page >= a.n_phys) {
        bad |= SPG_DEVERR_PAGE_ID;
        page = -1;
      }
    }
    if (bad) record_error(a.err, bad);
    s_page[threadIdx.x] = page;
    s_slot[threadIdx.x] = pos < 0 ? -1 : pos % a.S;
    s_pos[threadIdx.x] = a.positions ? a.positions[t] : pos;
  }
  __syncthreads();
  const int pairs = a.rot / 2;
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int tk = i / pairs, j = i % pairs;
    const unsigned long long f = static_cast<unsigned long long>(static_cast<long long>(s_pos[tk])) * a.turns[j];
    // nearest 2^-32 of a turn, as half-turns in [-1, 1)
    const int w = static_cast<int>(static_cast<uint32_t>((f + 0x80000000ull) >> 32));
    float sn, cs;
    sincospif(static_cast<float>(w) * 4.656612873077393e-10f, &sn, &cs);
    s_cs[tk][j] = make_float2(cs * a.mscale, sn * a.mscale);
  }
  __syncthreads();
  pdl_trigger();

  const int h0 = a.q ? 0 : a.Hq;
  const int items = (a.Hq - h0 + 2 * a.Hkv) * IPH, items32 = (items + 31) & ~31;
  const int rot_items = a.rot / 16;
  for (int tk = 0; tk < nt; ++tk) {
    const int slot = s_slot[tk], page = s_page[tk];
    if (slot < 0) continue;  // a row of no sequence
    const size_t t = t0 + tk;
    for (int it = threadIdx.x; it < items32; it += kThreads) {
      const bool live = it < items;
      const int h = live ? h0 + it / IPH : 0, j = it % IPH;
      const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
      const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;  // kv-head
      const bool turn = j < rot_items && !is_v;
      int c0 = 2 * j, c1 = 2 * j + 1;  // the item's two 16-byte pieces
      if (HALF && j < rot_items) {
        c0 = j;
        c1 = j + rot_items;
      }
      float x[8] = {}, y[8] = {};
      if (live) {
        const T* row = is_q   ? static_cast<const T*>(a.q) + t * a.q_stride + static_cast<size_t>(h) * D
                       : is_v ? static_cast<const T*>(a.v) + t * a.v_stride + static_cast<size_t>(hk) * D
                              : static_cast<const T*>(a.k) + t * a.k_stride + static_cast<size_t>(hk) * D;
        const uint4 w0 = *reinterpret_cast<const uint4*>(row + 8 * c0);
        const uint4 w1 = *reinterpret_cast<const uint4*>(row + 8 * c1);
        unpack8<T>(w0, x);
        unpack8<T>(w1, y);
      }
      if (turn) {
        const float2* cs = &s_cs[tk][8 * j];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 r = cs[e];
          // half: (x[e], y[e]); interleaved: neighbours within a piece
          float& u = HALF ? x[e] : (e < 4 ? x[2 * e] : y[2 * e - 8]);
          float& v = HALF ? y[e] : (e < 4 ? x[2 * e + 1] : y[2 * e - 7]);
          const float p = u * r.x - v * r.y, s = v * r.x + u * r.y;
          u = p;
          v = s;
        }
      }
      if (!I8 || is_q) {
        T* dst = nullptr;
        if (is_q)
          dst = static_cast<T*>(a.q_out) + (t * a.Hq + h) * D;
        else if (page >= 0)
          dst = static_cast<T*>(is_v ? a.v_pool : a.k_pool) + ((static_cast<size_t>(page) * a.Hkv + hk) * a.S + slot) * D;
        if (live && dst) {
          *reinterpret_cast<uint4*>(dst + 8 * c0) = pack8<T>(x);
          *reinterpret_cast<uint4*>(dst + 8 * c1) = pack8<T>(y);
        }
      }
      if constexpr (I8) {
        // scale and codes of the head's row: its IPH lanes are neighbours
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(fabsf(x[e]), fabsf(y[e])));
#pragma unroll
        for (int o = 1; o < IPH; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        __half sc = __float2half_rn(fminf(__fdiv_rn(m, 127.f), 65504.f));
        if (!(__half2float(sc) > 0.f)) sc = __float2half_rn(1.f);
        if (live && !is_q && page >= 0) {
          // the code of the quotient x / sc in 32 bits, by one division per
          // row: x * (1 / sc) is off by at most 2^-16 where codes are not
          // clamped and the quotient's own rounding by 2^-18, so that only
          // values within 2^-15 of a border are divided
          const float scale = __half2float(sc), inv = __fdiv_rn(1.f, scale);
          uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float v = e < 8 ? x[e & 7] : y[e & 7], z = v * inv;
            float r = rintf(z);
            if (fabsf(z - r) > 0.5f - 0x1p-15f) r = rintf(__fdiv_rn(v, scale));
            const int c = static_cast<int>(fmaxf(-127.f, fminf(127.f, r)));
            w[e >> 2] |= static_cast<uint32_t>(c & 0xff) << (8 * (e & 3));
          }
          const size_t r = (static_cast<size_t>(page) * a.Hkv + hk) * a.S + slot;
          int8_t* dst = static_cast<int8_t*>(is_v ? a.v_pool : a.k_pool) + r * D;
          *reinterpret_cast<uint2*>(dst + 8 * c0) = make_uint2(w[0], w[1]);
          *reinterpret_cast<uint2*>(dst + 8 * c1) = make_uint2(w[2], w[3]);
          if (j == 0) (is_v ? a.v_scale : a.k_scale)[r] = sc;
        }
      }
    }
  }
}

template <typename T, bool I8>
cudaError_t rope_typed(const spg_params& p, const RopeArgs& a, bool half, cudaStream_t st) {
  const dim3 grid((a.total_q + a.tokens - 1) / a.tokens), block(kThreads);
  if (p.head_dim == 128)
    return half ? launch_pdl(k_rope_append<T, I8, 128, true>, grid, block, 0, st, a)
                : launch_pdl(k_rope_append<T, I8, 128, false>, grid, block, 0, st, a);
  return half ? launch_pdl(k_rope_append<T, I8, 64, true>, grid, block, 0, st, a)
              : launch_pdl(k_rope_append<T, I8, 64, false>, grid, block, 0, st, a);
}

}  // namespace

bool rope_freqs(const spg_rope& r, int head_dim, double* inv, double* mscale) {
  const int rot = r.rot_dim == 0 ? head_dim : r.rot_dim;
  if (rot < 2 || rot > head_dim || rot % 2) return false;
  if (r.layout != SPG_ROPE_HALF && r.layout != SPG_ROPE_INTERLEAVED) return false;
  if (r.scaling < SPG_ROPE_PLAIN || r.scaling > SPG_ROPE_YARN) return false;
  if (!(r.base > 1.0) || std::isinf(r.base)) return false;
  if (r.scaling != SPG_ROPE_PLAIN && (!(r.factor >= 1.0) || std::isinf(r.factor))) return false;
  if (r.scaling == SPG_ROPE_YARN && r.orig_len < 1) return false;
  if (r.scaling == SPG_ROPE_NTK && rot <= 2) return false;
  constexpr double kTwoPi = 6.283185307179586476925;
  const double base = r.scaling == SPG_ROPE_NTK ? r.base * std::pow(r.factor, rot / (rot - 2.0)) : r.base;
  // pair index at which a pair makes `turns` turns over orig_len positions
  const auto at = [&](double turns) { return rot * std::log(r.orig_len / (turns * kTwoPi)) / (2.0 * std::log(base)); };
  double lo = 0.0, hi = 1.0;
  if (r.scaling == SPG_ROPE_YARN) {
    lo = std::fmax(std::floor(at(32.0)), 0.0);
    hi = std::fmin(std::ceil(at(1.0)), rot - 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot);
    if (r.scaling == SPG_ROPE_LINEAR) {
      inv[i] = f / r.factor;
    } else if (r.scaling == SPG_ROPE_YARN) {
      const double ramp = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 1e-3)));
      inv[i] = f / r.factor * ramp + f * (1.0 - ramp);
    } else {
      inv[i] = f;
    }
  }
  *mscale = r.scaling == SPG_ROPE_YARN ? 0.1 * std::log(r.factor) + 1.0 : 1.0;
  return true;
}

cudaError_t launch_rope_append(const spg_params& p, const spg_rope* rope, const RopeRows& r, void* k_pool, void* v_pool,
                               void* k_scale, void* v_scale, int32_t* err, cudaStream_t stream) {
  RopeArgs a{};
  a.mscale = 1.f;
  bool half = true;
  if (rope) {
    double inv[kMaxPairs], m = 1.0;
    if (!rope_freqs(*rope, p.head_dim, inv, &m)) return cudaErrorInvalidValue;
    a.rot = rope->rot_dim == 0 ? p.head_dim : rope->rot_dim;
    for (int i = 0; i < a.rot / 2; ++i)
      a.turns[i] = static_cast<unsigned long long>(std::ldexp(inv[i] / 6.283185307179586476925, 64));
    a.mscale = static_cast<float>(m);
    half = rope->layout == SPG_ROPE_HALF;
  }
  a.q = r.q;
  a.k = r.k;
  a.v = r.v;
  a.q_stride = r.q_stride;
  a.k_stride = r.k_stride;
  a.v_stride = r.v_stride;
  a.q_start = r.q_start;
  a.positions = r.positions;
  a.page_table = r.page_table;
  a.seq_lens = r.seq_lens;
  a.q_out = r.q_out;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.k_scale = static_cast<__half*>(k_scale);
  a.v_scale = static_cast<__half*>(v_scale);
  a.err = err;
  a.B = p.batch;
  a.Hq = p.num_q_heads;
  a.Hkv = p.num_kv_heads;
  a.S = p.page_size;
  a.MP = p.max_pages_per_seq;
  a.n_phys = p.num_phys_pages;
  a.total_q = r.total_q;
  // A token per CTA while they are few, then two (cold caches, one by one and
  // in pairs: MHA-32 fp16 512 tokens 13.5 and 15.5 us, 2048 27.8 and 29.9, 3000
  // 36.0 and 35.0, 8192 79.0 and 77.0; int8 GQA 32/8 8192 74.9 and 64.7)
  a.tokens = r.total_q > 2048 ? 2 : 1;
  const bool i8 = p.kv_dtype == SPG_I8;
  if (p.q_dtype == SPG_F16)
    return i8 ? rope_typed<__half, true>(p, a, half, stream) : rope_typed<__half, false>(p, a, half, stream);
  return i8 ? rope_typed<__nv_bfloat16, true>(p, a, half, stream) : rope_typed<__nv_bfloat16, false>(p, a, half, stream);
}

}  // namespace spg
