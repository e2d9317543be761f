// Eviction from the paged cache by accumulated attention weight
// (StreamingLLM/H2O: sinks, a recent window, heavy hitters), per (batch,
// kv-head): choose, then compact (paged_cache_evict).
//
// Choosing is an exact selection of the keep - forced heaviest of the
// unforced tokens.  Masses map to order-preserving 32-bit keys (NaN lowest);
// the key of the last one kept is found by histograms of the range that the
// keys still in question span, 2048 bins a pass, at most three passes; one
// more pass writes the kept positions in order, the first of the equal ones
// by position.  The kept masses move along in the same pass: a position
// never moves up, and a tile is read before anything is written at or before
// its end, so mass_out may be mass.
//
// Compacting moves rows of d channels.  To pages of its own it is a gather,
// split over tokens.  Within the same pages a destination slot j is also the
// source of some later destination, so the order matters: sources ascend
// with their destinations and never lie before them, hence a CTA that takes
// the tokens in order and reads a tile (and the next) before it writes the
// first never loses one.  CTAs of one (batch, kv-head) then split the row's
// channels (and K from V), which never meet.
#include <algorithm>

#include "spg_chunk_common.cuh"
#include "spg_internal.h"

namespace spg {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;
constexpr int kPer = 4;  // keys of a thread per tile of the ordered pass

struct EvictArgs {
  const float* mass;
  float* mass_out;
  const int32_t *page_table, *dst_table, *seq_lens;
  int32_t *kept, *new_lens, *err;
  uint8_t *k_pool, *v_pool;
  __half *k_scale, *v_scale;
  int Hkv, S, MP, n_phys, keep, n_sink, n_recent, row_bytes, slices, lpr_log2, in_place;
};

__device__ __forceinline__ uint32_t mass_key(float m) { return m != m ? 0u : score_key(m); }

// exclusive prefix of v over the block, and the total; s: one int per warp + 1
__device__ __forceinline__ int block_scan(int v, int* s, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) s[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = lane < nw ? s[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    if (lane < nw) s[lane] = w;
  }
  __syncthreads();
  total = s[nw - 1];
  const int base = warp ? s[warp - 1] : 0;
  __syncthreads();
  return base + incl - v;
}

__global__ void __launch_bounds__(kSelThreads) k_evict_select(const __grid_constant__ EvictArgs a) {
  __shared__ int s_hist[kBins];
  __shared__ int s_scan[33];
  __shared__ uint32_t s_lo, s_hi;
  __shared__ int s_bin, s_need;
  pdl_wait();
  const int unit = blockIdx.x, b = unit / a.Hkv, tid = threadIdx.x;
  int L = a.seq_lens[b];
  if (L < 0 || L > a.MP * a.S) {
    if (tid == 0) record_error(a.err, SPG_DEVERR_SEQ_LEN);
    L = 0;
  }
  const size_t N = static_cast<size_t>(a.MP) * a.S;
  const float* mass = a.mass + unit * N;
  float* mass_out = a.mass_out + unit * N;
  int32_t* kept = a.kept + static_cast<size_t>(unit) * a.keep;
  const int new_len = min(L, a.keep);
  if (tid == 0 && unit % a.Hkv == 0) a.new_lens[b] = new_len;
  for (int j = new_len + tid; j < a.keep; j += kSelThreads) kept[j] = -1;

  // the unforced tokens [lo_t, hi_t), `need` of them kept
  const int lo_t = min(a.n_sink, L), hi_t = max(lo_t, L - a.n_recent);
  int need = L <= a.keep ? hi_t - lo_t : a.keep - (L - (hi_t - lo_t));
  uint32_t thr = 0;     // keys above thr are kept, and the first `need` equal to it
  const bool all = need >= hi_t - lo_t;
  if (all) {
    need = hi_t - lo_t;
  } else if (need > 0) {
    if (tid == 0) {
      s_lo = 0xffffffffu;
      s_hi = 0u;
    }
    __syncthreads();
    uint32_t mn = 0xffffffffu, mx = 0u;
    for (int t = lo_t + tid; t < hi_t; t += kSelThreads) {
      const uint32_t k = mass_key(mass[t]);
      mn = min(mn, k);
      mx = max(mx, k);
    }
    mn = __reduce_min_sync(0xffffffffu, mn);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if ((tid & 31) == 0) {
      atomicMin(&s_lo, mn);
      atomicMax(&s_hi, mx);
    }
    __syncthreads();
    uint32_t lo = s_lo, hi = s_hi;
    while (lo < hi) {
      // bins of 2^shift keys over [lo, hi]
      const int shift = max(0, 32 - __clz(hi - lo) - 11);
      for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
      __syncthreads();
      for (int t = lo_t + tid; t < hi_t; t += kSelThreads) {
        const uint32_t k = mass_key(mass[t]);
        if (k >= lo && k <= hi) atomicAdd(&s_hist[(k - lo) >> shift], 1);
      }
      __syncthreads();
      // from the top: the bin in which the need-th key lies (threads take two bins each, descending)
      const int c0 = s_hist[kBins - 1 - 2 * tid], c1 = s_hist[kBins - 2 - 2 * tid];
      int total;
      const int before = block_scan(c0 + c1, s_scan, total);
      if (before < need && before + c0 >= need) {
        s_bin = kBins - 1 - 2 * tid;
        s_need = need - before;
      } else if (before + c0 < need && before + c0 + c1 >= need) {
        s_bin = kBins - 2 - 2 * tid;
        s_need = need - before - c0;
      }
      __syncthreads();
      need = s_need;
      const uint32_t first = lo + (static_cast<uint32_t>(s_bin) << shift);
      const uint32_t last = min(hi, first + ((1u << shift) - 1u));
      lo = first;
      hi = last;
      __syncthreads();
    }
    thr = lo;
  }

  // the kept positions in order
  int out = 0, equal = 0;
  for (int t0 = 0; t0 < L; t0 += kSelThreads * kPer) {
    float m[kPer];
    bool above[kPer], eq[kPer];
    int n_above = 0, n_eq = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int t = t0 + tid * kPer + e;
      m[e] = 0.f;
      above[e] = eq[e] = false;
      if (t < L) {
        m[e] = mass[t];
        const uint32_t k = mass_key(m[e]);
        above[e] = all || t < lo_t || t >= hi_t || (need > 0 && k > thr);
        eq[e] = !above[e] && need > 0 && k == thr;
      }
      n_above += above[e];
      n_eq += eq[e];
    }
    int total_eq, total;
    int e0 = equal + block_scan(n_eq, s_scan, total_eq);
    int n = n_above;
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (eq[e] && e0++ < need) {
        above[e] = true;
        ++n;
      }
    int o = out + block_scan(n, s_scan, total);  // a barrier: every mass of the tile is in registers
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (above[e]) {
        kept[o] = t0 + tid * kPer + e;
        mass_out[o] = m[e];
        ++o;
      }
    out += total;
    equal += total_eq;
  }
  pdl_trigger();
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;  // rows of a thread per step

// CTA (x, y, z): tokens of chunk x, slice y (K's, then V's, then the scales) of unit z
__global__ void __launch_bounds__(kMoveThreads) k_evict_move(const __grid_constant__ EvictArgs a) {
  pdl_wait();
  const int unit = blockIdx.z, b = unit / a.Hkv, h = unit % a.Hkv, tid = threadIdx.x;
  const int n = a.new_lens[b];
  const int32_t* kept = a.kept + static_cast<size_t>(unit) * a.keep;
  const int32_t* src_pt = a.page_table + static_cast<size_t>(b) * a.MP;
  const int32_t* dst_pt = a.dst_table + static_cast<size_t>(b) * a.MP;
  const bool scales = static_cast<int>(blockIdx.y) == 2 * a.slices;
  const bool is_v = static_cast<int>(blockIdx.y) >= a.slices;
  uint8_t* pool = is_v ? a.v_pool : a.k_pool;
  const int lpr = scales ? 0 : a.lpr_log2;  // log2 of the threads of one row slice
  const int slice = scales ? 0 : blockIdx.y % a.slices;
  const size_t col = (static_cast<size_t>(slice) << (lpr + 4)) + 16 * (tid & ((1 << lpr) - 1));
  const int per_step = (kMoveThreads >> lpr) * kMoveRows;
  const int steps = (n + per_step - 1) / per_step;
  const int s0 = static_cast<int>(static_cast<long long>(blockIdx.x) * steps / gridDim.x);
  const int s1 = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * steps / gridDim.x);

  uint4 w[2][kMoveRows];
  const auto slot = [&](const int32_t* pt, int t) -> long long {
    const int page = pt[t / a.S];
    if (page < 0 || page >= a.n_phys) {
      record_error(a.err, SPG_DEVERR_PAGE_ID);
      return -1;
    }
    return (static_cast<long long>(page) * a.Hkv + h) * a.S + t % a.S;
  };
  long long dst[2][kMoveRows];
  const auto load = [&](int step, uint4 (&v)[kMoveRows], long long (&d)[kMoveRows]) {
#pragma unroll
    for (int r = 0; r < kMoveRows; ++r) {
      const int j = step * per_step + r * (kMoveThreads >> lpr) + (tid >> lpr);
      d[r] = -1;
      if (j < n) {
        const int t = kept[j];
        const long long from = slot(src_pt, t);
        if (from >= 0 && !(a.in_place && t == j)) {
          d[r] = slot(dst_pt, j);
          if (scales)
            v[r].x = static_cast<uint32_t>(__half_as_ushort(a.k_scale[from])) |
                     (static_cast<uint32_t>(__half_as_ushort(a.v_scale[from])) << 16);
          else
            v[r] = *reinterpret_cast<const uint4*>(pool + from * a.row_bytes + col);
        }
      }
    }
  };
  const auto store = [&](const uint4 (&v)[kMoveRows], const long long (&d)[kMoveRows]) {
#pragma unroll
    for (int r = 0; r < kMoveRows; ++r)
      if (d[r] >= 0) {
        if (scales) {
          a.k_scale[d[r]] = __ushort_as_half(static_cast<unsigned short>(v[r].x & 0xffffu));
          a.v_scale[d[r]] = __ushort_as_half(static_cast<unsigned short>(v[r].x >> 16));
        } else {
          *reinterpret_cast<uint4*>(pool + d[r] * a.row_bytes + col) = v[r];
        }
      }
  };
  if (s0 < s1) load(s0, w[0], dst[0]);
  for (int s = s0; s < s1; s += 2) {
    if (s + 1 < s1) load(s + 1, w[1], dst[1]);
    if (a.in_place) __syncthreads();  // every row of this step (and the next) is in registers
    store(w[0], dst[0]);
    if (s + 1 >= s1) break;
    if (s + 2 < s1) load(s + 2, w[0], dst[0]);
    if (a.in_place) __syncthreads();
    store(w[1], dst[1]);
  }
}

}  // namespace

cudaError_t launch_evict(const spg_params& p, const float* mass, int keep, int n_sink, int n_recent, void* k_pool,
                         void* v_pool, void* k_scale, void* v_scale, const int32_t* page_table,
                         const int32_t* dst_table, const int32_t* seq_lens, int32_t* kept, int32_t* new_lens,
                         float* mass_out, int32_t* err, cudaStream_t stream) {
  EvictArgs a{};
  a.mass = mass;
  a.mass_out = mass_out;
  a.page_table = page_table;
  a.in_place = dst_table == nullptr || dst_table == page_table;
  a.dst_table = a.in_place ? page_table : dst_table;
  a.seq_lens = seq_lens;
  a.kept = kept;
  a.new_lens = new_lens;
  a.err = err;
  a.k_pool = static_cast<uint8_t*>(k_pool);
  a.v_pool = static_cast<uint8_t*>(v_pool);
  a.k_scale = static_cast<__half*>(k_scale);
  a.v_scale = static_cast<__half*>(v_scale);
  a.Hkv = p.num_kv_heads;
  a.S = p.page_size;
  a.MP = p.max_pages_per_seq;
  a.n_phys = p.num_phys_pages;
  a.keep = keep;
  a.n_sink = n_sink;
  a.n_recent = n_recent;
  a.row_bytes = p.head_dim * (p.kv_dtype == SPG_I8 ? 1 : 2);
  // within the same pages the rows' 64-byte pieces, to pages of its own whole rows
  const int slice_bytes = a.in_place ? 64 : a.row_bytes;
  a.slices = a.row_bytes / slice_bytes;
  a.lpr_log2 = 0;
  while ((16 << a.lpr_log2) < slice_bytes) ++a.lpr_log2;
  const int units = p.batch * p.num_kv_heads;
  cudaError_t e = launch_pdl(k_evict_select, dim3(units), dim3(kSelThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  int chunks = 1;
  if (!a.in_place) {
    const int per_step = (kMoveThreads >> a.lpr_log2) * kMoveRows;
    const long long most = static_cast<long long>(p.max_pages_per_seq) * p.page_size;
    const int steps = static_cast<int>((std::min<long long>(keep, most) + per_step - 1) / per_step);
    chunks = std::max(1, std::min(steps, (8 * device_sm_count() + 2 * units - 1) / (2 * units)));
  }
  const int y = 2 * a.slices + (p.kv_dtype == SPG_I8 ? 1 : 0);
  return launch_pdl(k_evict_move, dim3(chunks, y, units), dim3(kMoveThreads), 0, stream, a);
}

}  // namespace spg
