// Eviction from the paged cache by accumulated attention weight
// (StreamingLLM/H2O: sinks, a recent window, heavy hitters), per (batch,
// kv-head): choose, then compact (paged_cache_evict).
//
// Choosing is an exact selection of the keep - forced heaviest of the
// unforced tokens.  Masses map to order-preserving 32-bit keys (NaN lowest);
// the key of the last one kept is found by histograms of the range that the
// keys still in question span, 2048 bins a pass, at most three passes; one
// more pass writes the kept positions in order, the first of the equal ones
// by position, and their masses.  A cluster of up to 8 CTAs shares one
// (batch, kv-head): each reads its tokens' masses once, into shared memory
// (all of them before any is written, so mass_out may be mass), and the
// passes meet in the first CTA's histogram over distributed shared memory.
// Under a page table of more than 384K tokens they do not fit and every pass
// reads them again: the cluster does, or with mass_out = mass one CTA, since
// a later CTA's writes would meet an earlier one's reads (512K tokens of two
// kv-heads to a quarter: 0.18 ms the whole call with the cluster, 1.1 ms with
// one CTA; 4096 tokens of 32 kv-heads under such a table 31 and 33 us).
//
// Compacting moves rows of d channels.  To pages of its own it is a gather:
// a CTA resolves the pages of 128 kept tokens, then streams their K and V
// rows with all loads independent.  Within the same pages a destination slot
// j is also the source of some later destination, so the order matters:
// sources ascend with their destinations and never lie before them, hence a
// CTA that takes the tokens in order and reads a step (and the next) before
// it writes the first never loses one.  The CTAs of one (batch, kv-head)
// then split the row's channels (and K from V), which never meet.
//
// Measured (GB300): four caches of 128K tokens, GQA 32/8 bf16, to a quarter:
// selection 48 us (16.8 MB of masses; its passes over shared memory and the
// cluster barriers between them), gather 161 us (1.07 GB, 6.7 TB/s).  Within
// the same pages the call takes 0.70 ms: few CTAs move rows, each in order.
#include <algorithm>

#include "spg_chunk_common.cuh"
#include "spg_internal.h"

namespace spg {
namespace {

constexpr int kSelThreads = 512;
constexpr int kBins = 2048;
constexpr int kPer = 8;  // tokens of a thread per tile of the ordered pass
constexpr int kMaxCluster = 8;
// masses of one CTA that stay in shared memory (else they are read again)
constexpr int kMaxResident = 48 * 1024;

struct EvictArgs {
  const float* mass;
  float* mass_out;
  const int32_t *page_table, *dst_table, *seq_lens;
  int32_t *kept, *new_lens, *err;
  uint8_t *k_pool, *v_pool;
  __half *k_scale, *v_scale;
  int Hkv, S, MP, n_phys, keep, n_sink, n_recent, row_bytes, resident;
  int cluster, tiles;  // CTAs of a unit: of its cluster, and that move its rows
};

// atomics on another CTA's shared memory
__device__ __forceinline__ void red_cluster_add(uint32_t addr, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void red_cluster_min(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.min.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void red_cluster_max(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

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

// Units run along x (batch * kv-heads may be more than 65535, a grid's limit in
// y): a cluster of a.cluster CTAs per unit; CTA r has the r-th share of the
// sequence's tokens.
__global__ void __launch_bounds__(kSelThreads) k_evict_select(const __grid_constant__ EvictArgs a) {
  extern __shared__ float s_mass[];  // the CTA's masses, where they fit
  __shared__ int s_hist[kBins];
  __shared__ int s_scan[33];
  __shared__ uint32_t s_range[2];            // of the unforced keys: min, max (whole cluster, in the first CTA)
  __shared__ int s_bin, s_need;              // found by the first CTA
  __shared__ int s_count[kMaxCluster][2];    // per CTA: tokens above the threshold, and equal to it
  const int tid = threadIdx.x, C = a.cluster, rank = blockIdx.x % C, unit = blockIdx.x / C,
            b = unit / a.Hkv;
  if (tid == 0) {
    s_range[0] = 0xffffffffu;
    s_range[1] = 0u;
  }
  pdl_wait();
  int L = a.seq_lens[b];
  if (L < 0 || L > a.MP * a.S) {
    if (tid == 0 && rank == 0) record_error(a.err, SPG_DEVERR_SEQ_LEN);
    L = 0;
  }
  const size_t N = static_cast<size_t>(a.MP) * a.S;
  const float* mass = a.mass + unit * N;
  float* mass_out = a.mass_out + unit * N;
  int32_t* kept = a.kept + static_cast<size_t>(unit) * a.keep;
  const int new_len = min(L, a.keep);
  if (tid == 0 && rank == 0 && unit % a.Hkv == 0) a.new_lens[b] = new_len;
  for (int j = new_len + rank * kSelThreads + tid; j < a.keep; j += C * kSelThreads) kept[j] = -1;

  // this CTA's tokens
  const int share = (L + C - 1) / C, t_lo = min(rank * share, L), t_hi = min(t_lo + share, L);
  const auto at = [&](int t) { return a.resident ? s_mass[t - t_lo] : mass[t]; };
  // the unforced tokens [f_lo, f_hi), `need` of them kept
  const int f_lo = min(a.n_sink, L), f_hi = max(f_lo, L - a.n_recent);
  int need = L <= a.keep ? f_hi - f_lo : a.keep - (L - (f_hi - f_lo));
  const bool all = need >= f_hi - f_lo;
  const int u_lo = max(t_lo, f_lo), u_hi = min(t_hi, f_hi);  // this CTA's unforced ones
  uint32_t mn = 0xffffffffu, mx = 0u;
  for (int t = t_lo + tid; t < t_hi; t += kSelThreads) {
    const float v = mass[t];
    if (a.resident) s_mass[t - t_lo] = v;
    if (t >= f_lo && t < f_hi) {
      const uint32_t k = mass_key(v);
      mn = min(mn, k);
      mx = max(mx, k);
    }
  }
  cluster_sync();  // the first CTA's range is set up, every mass has been read
  uint32_t thr = 0;  // keys above thr are kept, and the first `need` equal to it
  if (!all && need > 0) {
    mn = __reduce_min_sync(0xffffffffu, mn);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if ((tid & 31) == 0 && mn <= mx) {
      atomicMin(&s_range[0], mn);
      atomicMax(&s_range[1], mx);
    }
    __syncthreads();
    if (rank != 0 && tid == 0) {
      red_cluster_min(map_rank(&s_range[0], 0), s_range[0]);
      red_cluster_max(map_rank(&s_range[1], 0), s_range[1]);
    }
    cluster_sync();
    uint32_t lo = static_cast<uint32_t>(ld_cluster_s32(map_rank(&s_range[0], 0)));
    uint32_t hi = static_cast<uint32_t>(ld_cluster_s32(map_rank(&s_range[1], 0)));
    while (lo < hi) {  // the same in every CTA
      // bins of 2^shift keys over [lo, hi]
      const int shift = max(0, 32 - __clz(hi - lo) - 11);
      for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
      cluster_sync();
      for (int t = u_lo + tid; t < u_hi; t += kSelThreads) {
        const uint32_t k = mass_key(at(t));
        if (k >= lo && k <= hi) atomicAdd(&s_hist[(k - lo) >> shift], 1);
      }
      __syncthreads();
      if (rank != 0)
        for (int i = tid; i < kBins; i += kSelThreads)
          if (s_hist[i]) red_cluster_add(map_rank(&s_hist[i], 0), s_hist[i]);
      cluster_sync();
      if (rank == 0) {
        // from the top: the bin in which the need-th key lies (threads take four bins each, descending)
        int c[4], sum = 0, total;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += c[i] = s_hist[kBins - 1 - 4 * tid - i];
        int before = block_scan(sum, s_scan, total);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (before < need && before + c[i] >= need) {
            s_bin = kBins - 1 - 4 * tid - i;
            s_need = need - before;
          }
          before += c[i];
        }
      }
      cluster_sync();
      need = ld_cluster_s32(map_rank(&s_need, 0));
      const uint32_t first = lo + (static_cast<uint32_t>(ld_cluster_s32(map_rank(&s_bin, 0))) << shift);
      hi = min(hi, first + ((1u << shift) - 1u));
      lo = first;
    }
    thr = lo;
  }

  // the kept positions in order: how many this CTA's tokens follow
  const auto above = [&](int t, uint32_t k) { return all || t < f_lo || t >= f_hi || (need > 0 && k > thr); };
  int n_above = 0, n_equal = 0;
  for (int t = t_lo + tid; t < t_hi; t += kSelThreads) {
    const uint32_t k = mass_key(at(t));
    if (above(t, k)) ++n_above;
    else if (need > 0 && k == thr) ++n_equal;
  }
  int all_above, all_equal;
  block_scan(n_above, s_scan, all_above);
  block_scan(n_equal, s_scan, all_equal);
  if (tid < C) {
    st_cluster_u32(map_rank(&s_count[rank][0], tid), all_above);
    st_cluster_u32(map_rank(&s_count[rank][1], tid), all_equal);
  }
  cluster_sync();  // (nothing remote is touched after it)
  int out = 0, equal = 0;
  for (int r = 0; r < rank; ++r) {
    out += s_count[r][0];
    equal += s_count[r][1];
  }
  out += min(equal, max(need, 0));
  for (int t0 = t_lo; t0 < t_hi; t0 += kSelThreads * kPer) {
    float m[kPer];
    unsigned take = 0, eq = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int t = t0 + tid * kPer + e;
      m[e] = 0.f;
      if (t < t_hi) {
        m[e] = at(t);
        const uint32_t k = mass_key(m[e]);
        if (above(t, k)) take |= 1u << e;
        else if (need > 0 && k == thr) eq |= 1u << e;
      }
    }
    int total_eq, total;
    int e0 = equal + block_scan(__popc(eq), s_scan, total_eq);
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if ((eq >> e & 1u) && e0++ < need) take |= 1u << e;
    int o = out + block_scan(__popc(take), s_scan, total);  // a barrier: every mass of the tile is in registers
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (take >> e & 1u) {
        kept[o] = t0 + tid * kPer + e;
        mass_out[o] = m[e];
        ++o;
      }
    out += total;
    equal += total_eq;
  }
  pdl_trigger();
}

// row of the pool that holds token t of kv-head h (-1: a bad page)
__device__ __forceinline__ long long pool_row(const EvictArgs& a, const int32_t* pt, int h, int t) {
  const int page = pt[t / a.S];
  if (page < 0 || page >= a.n_phys) {
    record_error(a.err, SPG_DEVERR_PAGE_ID);
    return -1;
  }
  return (static_cast<long long>(page) * a.Hkv + h) * a.S + t % a.S;
}

// ---- to pages of its own ---------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 128;  // kept tokens of a CTA

// CTA x of a unit's `tiles`: kept tokens 128 x .., K and V
template <int ROW>  // bytes
__global__ void __launch_bounds__(kMoveThreads) k_evict_gather(const __grid_constant__ EvictArgs a) {
  __shared__ long long s_from[kMoveRows], s_to[kMoveRows];
  pdl_wait();
  const int unit = blockIdx.x / a.tiles, b = unit / a.Hkv, h = unit % a.Hkv, tid = threadIdx.x;
  const int j0 = blockIdx.x % a.tiles * kMoveRows;
  const int n = min(kMoveRows, a.new_lens[b] - j0);
  if (n <= 0) return;
  if (tid < n) {
    const long long from = pool_row(a, a.page_table + static_cast<size_t>(b) * a.MP, h,
                                    a.kept[static_cast<size_t>(unit) * a.keep + j0 + tid]);
    const long long to = pool_row(a, a.dst_table + static_cast<size_t>(b) * a.MP, h, j0 + tid);
    s_from[tid] = from;
    s_to[tid] = from < 0 ? -1 : to;
    if (a.k_scale && from >= 0 && to >= 0) {
      a.k_scale[to] = a.k_scale[from];
      a.v_scale[to] = a.v_scale[from];
    }
  }
  __syncthreads();
  constexpr int LPR = ROW / 16, PER = kMoveThreads / LPR;  // threads of a row, rows at a time
  constexpr int STEPS = kMoveRows / PER, U = STEPS < 8 ? STEPS : 8;
  const int r0 = tid / LPR, col = tid % LPR * 16;
#pragma unroll 1
  for (int kv = 0; kv < 2; ++kv) {
    uint8_t* pool = (kv ? a.v_pool : a.k_pool) + col;
#pragma unroll 1
    for (int s = 0; s < STEPS; s += U) {
      uint4 w[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int r = r0 + (s + i) * PER;
        if (r < n && s_to[r] >= 0) w[i] = __ldcs(reinterpret_cast<const uint4*>(pool + s_from[r] * ROW));
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int r = r0 + (s + i) * PER;
        if (r < n && s_to[r] >= 0) *reinterpret_cast<uint4*>(pool + s_to[r] * ROW) = w[i];
      }
    }
  }
}

// ---- within the same pages ---------------------------------------------------------
constexpr int kShiftRows = 8;        // rows of a thread per step
constexpr int kSliceBytes = 32;      // a CTA's channels

// CTA x of a unit's `tiles`: slice x (K's, then V's, then the scales)
__global__ void __launch_bounds__(kMoveThreads) k_evict_shift(const __grid_constant__ EvictArgs a) {
  pdl_wait();
  const int unit = blockIdx.x / a.tiles, x = blockIdx.x % a.tiles, b = unit / a.Hkv, h = unit % a.Hkv, tid = threadIdx.x;
  const int n = a.new_lens[b], slices = a.row_bytes / kSliceBytes, slice = x % slices;
  const int32_t* kept = a.kept + static_cast<size_t>(unit) * a.keep;
  const int32_t* pt = a.page_table + static_cast<size_t>(b) * a.MP;
  const bool scales = x == 2 * slices;
  uint8_t* pool = x >= slices ? a.v_pool : a.k_pool;
  const int lpr = scales ? 1 : kSliceBytes / 16;  // threads of a row's slice
  const int col = slice * kSliceBytes + tid % lpr * 16, rows = kMoveThreads / lpr;
  const int per_step = rows * kShiftRows, steps = (n + per_step - 1) / per_step;
  uint4 w[2][kShiftRows];
  long long dst[2][kShiftRows];
  const auto load = [&](int step, uint4 (&v)[kShiftRows], long long (&d)[kShiftRows]) {
#pragma unroll
    for (int r = 0; r < kShiftRows; ++r) {
      const int j = step * per_step + r * rows + tid / lpr;
      d[r] = -1;
      if (j >= n) continue;
      const int t = kept[j];
      if (t == j) continue;  // already there
      const long long from = pool_row(a, pt, h, t);
      if (from < 0) continue;
      d[r] = pool_row(a, pt, h, j);
      if (scales)
        v[r].x = static_cast<uint32_t>(__half_as_ushort(a.k_scale[from])) |
                 (static_cast<uint32_t>(__half_as_ushort(a.v_scale[from])) << 16);
      else
        v[r] = *reinterpret_cast<const uint4*>(pool + from * a.row_bytes + col);
    }
  };
  const auto store = [&](const uint4 (&v)[kShiftRows], const long long (&d)[kShiftRows]) {
#pragma unroll
    for (int r = 0; r < kShiftRows; ++r)
      if (d[r] >= 0) {
        if (scales) {
          a.k_scale[d[r]] = __ushort_as_half(static_cast<unsigned short>(v[r].x & 0xffffu));
          a.v_scale[d[r]] = __ushort_as_half(static_cast<unsigned short>(v[r].x >> 16));
        } else {
          *reinterpret_cast<uint4*>(pool + d[r] * a.row_bytes + col) = v[r];
        }
      }
  };
  if (steps > 0) load(0, w[0], dst[0]);
  for (int s = 0; s < steps; s += 2) {
    if (s + 1 < steps) load(s + 1, w[1], dst[1]);
    __syncthreads();  // every row of this step (and the next) is in registers
    store(w[0], dst[0]);
    if (s + 1 >= steps) break;
    if (s + 2 < steps) load(s + 2, w[0], dst[0]);
    __syncthreads();
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
  a.dst_table = dst_table;
  const bool in_place = dst_table == nullptr || dst_table == page_table;
  a.seq_lens = seq_lens;
  a.kept = kept;
  a.new_lens = new_lens;
  a.err = err;
  a.k_pool = static_cast<uint8_t*>(k_pool);
  a.v_pool = static_cast<uint8_t*>(v_pool);
  if (p.kv_dtype == SPG_I8) {
    a.k_scale = static_cast<__half*>(k_scale);
    a.v_scale = static_cast<__half*>(v_scale);
  }
  a.Hkv = p.num_kv_heads;
  a.S = p.page_size;
  a.MP = p.max_pages_per_seq;
  a.n_phys = p.num_phys_pages;
  a.keep = keep;
  a.n_sink = n_sink;
  a.n_recent = n_recent;
  a.row_bytes = p.head_dim * (p.kv_dtype == SPG_I8 ? 1 : 2);
  const int units = p.batch * p.num_kv_heads;
  const long long most = static_cast<long long>(p.max_pages_per_seq) * p.page_size;
  // one CTA up to 2048 tokens, then as many as keep that share, up to 8
  int C = 1;
  while (C < kMaxCluster && most > 2048ll * C) C *= 2;
  const long long share = (most + C - 1) / C;
  a.resident = share <= kMaxResident ? 1 : 0;
  if (!a.resident && mass_out == mass) C = 1;
  a.cluster = C;
  const size_t smem = a.resident ? sizeof(float) * share : 0;
  cudaError_t e = ensure_smem(k_evict_select, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(C) * units);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, k_evict_select, a);
  if (e != cudaSuccess) return e;
  if (in_place) {
    a.tiles = 2 * (a.row_bytes / kSliceBytes) + (p.kv_dtype == SPG_I8 ? 1 : 0);
    return launch_pdl(k_evict_shift, dim3(static_cast<unsigned>(a.tiles) * units), dim3(kMoveThreads), 0, stream, a);
  }
  a.tiles = static_cast<int>((std::min<long long>(keep, most) + kMoveRows - 1) / kMoveRows);
  const dim3 grid(static_cast<unsigned>(a.tiles) * units);
  switch (a.row_bytes) {
    case 256: return launch_pdl(k_evict_gather<256>, grid, dim3(kMoveThreads), 0, stream, a);
    case 128: return launch_pdl(k_evict_gather<128>, grid, dim3(kMoveThreads), 0, stream, a);
    default: return launch_pdl(k_evict_gather<64>, grid, dim3(kMoveThreads), 0, stream, a);
  }
}

}  // namespace spg
