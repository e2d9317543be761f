// Attention weight received by every cached token (paged_attention_mass), on
// the tcgen05 tensor cores.
//
// An item is 256 tokens of one (batch, kv-head), two tiles of 128; a step is
// 128 rows (head r % G of new token r / G) that see them:
//   S^T = K Q^T   tokens are TMEM lanes, rows its columns
//   sum of exp2(scale s - lse) along a lane, by the thread that owns the token
// so that a token's sum needs no exchange between threads, no atomics, and
// has a fixed order.  The keys of an item stay in shared memory while the
// rows pass by; with few rows (a decode step) the keys pass by and the rows
// stay.  One exponential per (row, token) and one product of the head_dim:
// with 128 channels the tensor cores and the exponentials take about the
// same time, so two accumulators per tile keep both going.
//
// The steps of all items are dealt out evenly (spg_deal.cuh).  A part of an
// item leaves its 256 sums in the workspace, and the part that arrives last
// adds them in order.
//
// Measured (GB300): 2048 rows over 32K, GQA 32/8, 606 to 618 us, 0.87 PFLOP/s
// of 1.90.  A summing warp takes 1770 cycles for its 128 columns and 600 to hand
// the accumulator back, against 1024 of products for both tiles.  Four
// summing warpgroups instead of two, half the columns each, took 913 us (the
// 80 registers that leaves spill in the loading warps); keeping whole rows of
// 128 columns in registers 724.
//
// Nothing is rounded to fewer than 32 bits.
#include <algorithm>
#include <cmath>

#include "spg_deal.cuh"
#include "spg_internal.h"
#include "spg_tile_load.cuh"

namespace spg {
namespace {

constexpr int kItemTokens = 2 * kTile;
constexpr uint32_t kTmemCols = 512;  // two accumulators of 128 columns for each of the two tiles

struct TokenItems : ChunkShape {
  static constexpr int kLeast = 1, kExtra = 0;
  __device__ int items(const ChunkSeq& s) const { return (s.L + kItemTokens - 1) / kItemTokens; }
  // row tiles of the sequence, and the first that sees token t
  __device__ int row_tiles(const ChunkSeq& s) const { return ((s.n << g_log2) + kTile - 1) / kTile; }
  __device__ int first_tile(const ChunkSeq& s, int t) const { return t > s.pos0 ? ((t - s.pos0) << g_log2) / kTile : 0; }
  __device__ int item_steps(const ChunkSeq& s, int i) const { return s.n == 0 ? 1 : row_tiles(s) - first_tile(s, i * kItemTokens); }
  // item k is seen by the row tiles from floor((256 k - pos0) G / 128) on: 2 k G - ceil(pos0 G / 128)
  // past pos0 (an item without rows still counts one step, its decay)
  __device__ long long steps(const ChunkSeq& s, int m) const {
    if (s.n == 0) return m;
    const long long rt = row_tiles(s);
    const int early = min(m, s.pos0 / kItemTokens + 1);
    long long sum = early * rt;
    if (m > early) {
      const long long c = ((static_cast<long long>(s.pos0) << g_log2) + kTile - 1) / kTile, cnt = m - early;
      sum += cnt * (rt + c) - ((2ll * (cnt * (early + m - 1) / 2)) << g_log2);
    }
    return sum;
  }
};

struct MassArgs {
  TokenItems sh;
  CUtensorMap tmq;
  const void* k_pool;
  const __half* k_scale;
  const int32_t* page_table;
  const float *lse, *mass_in;
  float* mass_out;
  int32_t *err, *counters;
  float* part;  // [2 * CTAs][256]
  int Hkv, S, s_log2, MP, n_phys;
  float scale_log2, decay;
};

// A part of an item with the rows it takes.
struct Seg : Part {
  int tile0, tiles;  // row tiles [tile0, tile0 + tiles)
};
struct SegIter : PartIter<TokenItems> {
  using PartIter::PartIter;
  __device__ bool next(Seg& s) {
    if (!PartIter::next(s)) return false;
    s.tile0 = sh.first_tile(s.sq, s.item * kItemTokens) + s.k0;
    s.tiles = s.sq.n == 0 ? 0 : s.k1 - s.k0;
    return true;
  }
};
// Which tile of rows is in shared memory: it stays while the next step wants
// the same one.  Every role follows the same rule.
struct RowRing {
  int b = -1, h = -1, tile = -1;
  __device__ bool same(const Seg& s, int t) const { return s.b == b && s.h == h && t == tile; }
  __device__ void set(const Seg& s, int t) { b = s.b, h = s.h, tile = t; }
};

template <int D>
struct Layout {
  static constexpr uint32_t kTileBytes = D / 64 * kTile * 128;
  static constexpr int QST = 3;
  static constexpr uint32_t k_off = 0, q_off = 4 * kTileBytes, misc = q_off + QST * kTileBytes;
};
template <int QST>
struct Misc {
  uint64_t k_full[2][2], k_empty[2][2], q_full[QST], q_empty[QST], s_full[2][2], s_empty[2][2], drain[2];
  Plan plan;
  uint32_t tmem;
  int last;
  int gaps[QST];  // the tile has rows that count nothing
  alignas(16) float neg_lse[QST][kTile];  // -lse in the log2 domain; -inf for rows that count nothing
};

template <typename T, typename TQ, int D>
struct Kernel {
  static constexpr bool I8 = sizeof(T) == 1;
  using Lay = Layout<D>;
  using M = Misc<Lay::QST>;
  using Tiles = TileLoader<T, TQ, D>;
  static constexpr int QST = Lay::QST;
  // warps 0-7 sums, 8-11 keys, 12 and 13 issue for one tile each, 14 rows
  static constexpr int kThreads = 512, kLoadWarp = 8, kMmaWarp = 12, kRowWarp = 14;

  // ---- products of one tile's keys with every row tile (whole warp, one lane issues) ------
  static __device__ bool issue(const MassArgs& a, M& m, uint32_t smem, uint32_t tmem, int t) {
    const auto wait = [&](uint64_t* bar, uint32_t phase) {
      return __all_sync(0xffffffffu, Waiter{a.err}(bar, phase)) != 0;
    };
    const auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    constexpr uint32_t kStep = Lay::kTileBytes >> 4, kHalf = kTile * 128;
    tmem = uniform(tmem) + t * 256;
    const uint32_t dk = desc_k_major(smem + Lay::k_off) + t * kStep, dq = desc_k_major(smem + Lay::q_off);
    uint32_t kc = 0, qi = 0, qr = 0, sc = 0;
    bool have = false;  // a row tile in use
    RowRing ring;
    SegIter it(a.sh, m.plan);
    Seg s;
    while (uniform(it.next(s))) {
      const int tiles = uniform(s.tiles);
      if (tiles == 0) continue;
      if (!wait(&m.k_full[kc & 1][t], kc >> 1)) return false;
      fence_proxy_async();
      for (int j = 0; j < tiles; ++j) {
        const int tile = s.tile0 + j;
        if (!uniform(ring.same(s, tile))) {
          if (have) {
            if (elect_one()) mma_commit(&m.q_empty[qi]);
            __syncwarp();
            if (++qi == QST) qi = 0, ++qr;
          }
          have = true;
          ring.set(s, tile);
          if (!wait(&m.q_full[qi], qr)) return false;
        }
        const uint32_t buf = sc & 1;
        if (sc >= 2 && !wait(&m.s_empty[t][buf], (sc >> 1) - 1)) return false;
        tc_fence_after();
        // columns in use, in sixteens
        const int cols = min(kTile, ((s.sq.n << a.sh.g_log2) - tile * kTile + 15) & ~15);
        const uint32_t id = instr_desc<TQ>(kTile, uniform(cols), false);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32u) >> 4;
            mma_ss(tmem + buf * 128, dk + (kc & 1) * 2 * kStep + off, dq + qi * kStep + off, id, ks > 0);
          }
          mma_commit(&m.s_full[t][buf]);
          if (j == tiles - 1) mma_commit(&m.k_empty[kc & 1][t]);
        }
        __syncwarp();
        ++sc;
      }
      ++kc;
    }
    return true;
  }

  // ---- rows: their tile by TMA, their lse by hand, read one tile ahead (whole warp) ---------
  static __device__ void load_rows(const MassArgs& a, M& m, uint8_t* smem, int lane) {
    const int g_log2 = a.sh.g_log2;
    RowRing ring;
    SegIter it(a.sh, m.plan);
    Seg s;
    int j = 0;
    s.tiles = 0;
    float v[kTile / 32];
    const auto next = [&] {  // the next tile that is not there yet, its lse on their way
      for (;; ++j) {
        while (j >= s.tiles) {
          if (!it.next(s)) return false;
          j = 0;
        }
        if (!ring.same(s, s.tile0 + j)) break;
      }
      ring.set(s, s.tile0 + j);
#pragma unroll
      for (int i = 0; i < kTile / 32; ++i) {
        const int r = ring.tile * kTile + lane + 32 * i;
        v[i] = r < s.sq.n << g_log2 ? a.lse[(static_cast<size_t>(s.sq.start + (r >> g_log2)) * a.Hkv << g_log2) + (s.h << g_log2) +
                                        (r & ((1 << g_log2) - 1))]
                                : -INFINITY;
      }
      return true;
    };
    bool more = next();
    for (uint32_t qi = 0, qr = 0; more; qr += qi == QST - 1, qi = qi == QST - 1 ? 0 : qi + 1) {
      if (!__all_sync(0xffffffffu, qr == 0 || Waiter{a.err}(&m.q_empty[qi], qr - 1))) return;
#pragma unroll
      for (int i = 0; i < kTile / 32; ++i) m.neg_lse[qi][lane + 32 * i] = v[i] == -INFINITY ? -INFINITY : -v[i] * kLog2e;
      bool gap = false;
#pragma unroll
      for (int i = 0; i < kTile / 32; ++i) gap |= v[i] == -INFINITY;
      gap = __any_sync(0xffffffffu, gap);
      __syncwarp();
      if (lane == 0) {
        m.gaps[qi] = gap;
        mbar_arrive_expect_tx(&m.q_full[qi], Lay::kTileBytes);
        for (int hf = 0; hf < D / 64; ++hf)
          tma_tile_4d(smem + Lay::q_off + qi * Lay::kTileBytes + hf * kTile * 128, &a.tmq, hf * 64, 0, s.h,
                      s.sq.start + (ring.tile * kTile >> g_log2), &m.q_full[qi]);
      }
      more = next();
    }
  }

  // ---- keys: a ring of four tiles, the two of an item after those of the last --------------
  static __device__ void load_keys(const MassArgs& a, M& m, uint8_t* smem, int tid, int lane) {
    bool dead = false;  // after a wait that ran out the others are skipped
    const auto wait = [&](uint64_t* bar, uint32_t phase) {
      if (!dead && !Waiter{a.err}(bar, phase)) dead = true;
    };
    const int s_log2 = a.s_log2;
    uint32_t kc = 0, copied = 0, done = 0;  // items; tiles
    const auto finish = [&] {               // int8: the oldest of the tiles in flight
      const uint32_t x = done++ & 3;
      Tiles::widen(smem + Lay::k_off + x * Lay::kTileBytes, tid, 3);
      fence_proxy_async();
      mbar_arrive(&m.k_full[x >> 1][x & 1]);
    };
    SegIter it(a.sh, m.plan);
    Seg s, ahead;
    int page[2], page_ahead[2];
    const auto next = [&] {  // the next item with rows, its pages on their way
      do
        if (!it.next(ahead)) return false;
      while (ahead.tiles == 0);
      const int32_t* pt = a.page_table + static_cast<size_t>(ahead.b) * a.MP;
#pragma unroll
      for (int t = 0; t < 2; ++t)
        page_ahead[t] = Tiles::page_of(pt, ahead.item * kItemTokens + t * kTile, ahead.sq.L, s_log2, a.n_phys, lane);
      return true;
    };
    bool more = next();
    while (more) {
      s = ahead;
      page[0] = page_ahead[0];
      page[1] = page_ahead[1];
      more = next();
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t x = 2 * (kc & 1) + t;
        if (kc >= 2) wait(&m.k_empty[kc & 1][t], (kc >> 1) - 1);
        Tiles::copy(a.k_pool, a.Hkv, s.h, s_log2, s.item * kItemTokens + t * kTile, s.sq.L, page[t], tid,
                    smem_u32(smem) + Lay::k_off + x * Lay::kTileBytes);
        ++copied;
        if constexpr (I8) {
          copy_commit();
          // two tiles in flight: a third would be widened only after the one
          // before it was used
          if (copied - done > 2) {
            copy_wait<2>();
            finish();
          }
        } else {
          copy_arrive(&m.k_full[kc & 1][t]);
        }
      }
      ++kc;
    }
    copy_commit();
    copy_wait<0>();
    if constexpr (I8)
      while (done < copied) finish();
  }

  // ---- sums -----------------------------------------------------------------------------------------
  static __device__ void sums(const MassArgs& a, M& m, uint32_t tmem, int warp, int lane) {
    bool dead = false;
    const auto wait = [&](uint64_t* bar, uint32_t phase) {
      if (!dead && !Waiter{a.err}(bar, phase)) dead = true;
    };
    const int t = warp >> 2, tid = threadIdx.x;
    const uint32_t tS = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + t * 256;
    uint32_t sc = 0, qi = 0, qr = 0;
    bool have = false;
    RowRing ring;
    SegIter it(a.sh, m.plan);
    Seg s, ahead;
    // the page of the thread's token, one item ahead; its scale and its old
    // mass follow when the item begins, while its products are on their way
    int page = 0, page_ahead = 0;
    const auto next = [&] {
      if (!it.next(ahead)) return false;
      const int tok = ahead.item * kItemTokens + tid;
      if (tok < ahead.sq.L) page_ahead = a.page_table[static_cast<size_t>(ahead.b) * a.MP + (tok >> a.s_log2)];
      return true;
    };
    bool more = next();
    while (more) {
      s = ahead;
      page = page_ahead;
      const int tok = s.item * kItemTokens + tid;  // threads 0-127: tile 0, 128-255: tile 1
      const size_t at = (static_cast<size_t>(s.b) * a.Hkv + s.h) * a.MP * a.S + tok;
      const bool live = tok < s.sq.L, ok = live && page >= 0 && page < a.n_phys;
      float k = a.scale_log2, old = 0.f;
      if (live && !ok && s.tiles > 0) record_error(a.err, SPG_DEVERR_PAGE_ID);
      if constexpr (I8)
        if (ok) k *= __half2float(a.k_scale[(static_cast<size_t>(page) * a.Hkv + s.h) * a.S + (tok & (a.S - 1))]);
      if (live && a.mass_in && a.decay > 0.f && tok < s.sq.pos0 && s.k0 == 0) old = a.mass_in[at] * a.decay;
      more = next();
      const uint64_t k2 = f32x2(k, k);
      uint64_t sum0 = f32x2(0.f, 0.f), sum1 = sum0;
      for (int j = 0; j < s.tiles; ++j) {
        const int tile = s.tile0 + j;
        if (!ring.same(s, tile)) {
          if (have) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&m.q_empty[qi]);
            if (++qi == QST) qi = 0, ++qr;
          }
          have = true;
          ring.set(s, tile);
          wait(&m.q_full[qi], qr);
        }
        const float* nl = m.neg_lse[qi];
        const uint32_t buf = sc & 1;
        wait(&m.s_full[t][buf], sc >> 1);
        ++sc;
        tc_fence_after();
        const int cols = min(kTile, (s.sq.n << a.sh.g_log2) - tile * kTile);
        // rows from which on the token is seen (its own is the first)
        const int from = ((tok - s.sq.pos0) << a.sh.g_log2) - tile * kTile;
        // (rows behind the sequence's last are gaps too)
        const bool masked = m.gaps[qi] || (s.item + 1) * kItemTokens - 1 > s.sq.pos0 + (tile * kTile >> a.sh.g_log2);
        // half a row in registers at a time; the accumulator goes back with the second
        uint32_t x[kTile / 2];
        if (masked) {
          for (int c = 0; c < cols; c += 32) {
            tmem_ld32(x, tS + buf * 128 + c);
            tmem_wait_ld();
#pragma unroll
            for (int g = 0; g < 32; g += 8)
              if (c + g < cols) {  // the same for the whole block
#pragma unroll
                for (int i = g; i < g + 8; i += 2) {
                  // rows without a log-sum-exp are left out, whatever their products are
                  const float n0 = nl[c + i], n1 = nl[c + i + 1];
                  const float p = c + i < from || n0 == -INFINITY ? 0.f : ex2(fmaf(__uint_as_float(x[i]), k, n0));
                  const float q = c + i + 1 < from || n1 == -INFINITY ? 0.f : ex2(fmaf(__uint_as_float(x[i + 1]), k, n1));
                  sum0 = add_f32x2(sum0, f32x2(p, q));
                }
              }
          }
          tc_fence_before();
          mbar_arrive(&m.s_empty[t][buf]);
        } else {
#pragma unroll
          for (int hf = 0; hf < kTile; hf += kTile / 2) {
            tmem_ld32(x, tS + buf * 128 + hf);
            tmem_ld32(x + 32, tS + buf * 128 + hf + 32);
            tmem_wait_ld();
            if (hf) {
              tc_fence_before();
              mbar_arrive(&m.s_empty[t][buf]);
            }
#pragma unroll
            for (int i = 0; i < kTile / 2; i += 4) {
              const ulonglong2 e = *reinterpret_cast<const ulonglong2*>(nl + hf + i);
              const float2 p = unpack_f32x2(fma_f32x2(f32x2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), k2, e.x));
              const float2 q = unpack_f32x2(fma_f32x2(f32x2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), k2, e.y));
              sum0 = add_f32x2(sum0, f32x2(ex2(p.x), ex2(p.y)));
              sum1 = add_f32x2(sum1, f32x2(ex2(q.x), ex2(q.y)));
            }
          }
        }
      }
      const float2 p = unpack_f32x2(sum0), q = unpack_f32x2(sum1);
      const float sum = ok ? (p.x + p.y) + (q.x + q.y) : 0.f;
      if (s.whole()) {
        if (live) a.mass_out[at] = old + sum;
      } else {
        __stcg(a.part + own_slot(s) * kItemTokens + tid, sum);
        join(a, m, s, tid, at, live);
      }
    }
  }

  // Counts a part of an item in; the last to arrive adds them up.
  static __device__ void join(const MassArgs& a, M& m, const Seg& s, int tid, size_t at, bool live) {
    const PartRange pr(m.plan, s);
    __threadfence();
    bar_sync(1, 256);
    if (tid == 0) m.last = atomicAdd(&a.counters[pr.c0], 1) == pr.c1 - pr.c0;
    bar_sync(2, 256);
    if (!m.last) return;
    __threadfence();
    float sum = 0.f;
    for (int c = pr.c0; c <= pr.c1; ++c) sum += __ldcg(a.part + pr.slot(c) * kItemTokens + tid);
    if (live) {
      float old = 0.f;
      if (a.mass_in && a.decay > 0.f && s.item * kItemTokens + tid < s.sq.pos0) old = a.mass_in[at] * a.decay;
      a.mass_out[at] = old + sum;
    }
    if (tid == 0) a.counters[pr.c0] = 0;  // ready for the next call
  }
};

template <typename T, typename TQ, int D>
__global__ void __launch_bounds__(512, 1) k_mass(const __grid_constant__ MassArgs a) {
  using K = Kernel<T, TQ, D>;
  using M = typename K::M;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  M& m = *reinterpret_cast<M*>(smem + K::Lay::misc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m.drain[i], 1);
      for (int j = 0; j < 2; ++j) {
        mbar_init(&m.k_full[i][j], K::Tiles::kThreads);
        mbar_init(&m.k_empty[i][j], 1);
        mbar_init(&m.s_full[i][j], 1);
        mbar_init(&m.s_empty[i][j], kTile);
      }
    }
    for (int i = 0; i < K::QST; ++i) {
      mbar_init(&m.q_full[i], 1);
      mbar_init(&m.q_empty[i], 2 + 8);  // the issuing warps and the summing ones
    }
    mbar_fence_init();
  }
  if (warp == K::kMmaWarp) tmem_alloc(&m.tmem, kTmemCols);
  pdl_wait();
  if (warp == 0) make_plan(a.sh, &m.plan, a.err, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem;
  if (warp < K::kLoadWarp) {
    K::sums(a, m, tmem, warp, lane);
  } else {
    if (warp < K::kMmaWarp) {
      K::load_keys(a, m, smem, threadIdx.x - K::kLoadWarp * 32, lane);
    } else if (warp < K::kRowWarp) {
      const int t = warp - K::kMmaWarp;
      if (!K::issue(a, m, smem_u32(smem), tmem, t)) {
        if (elect_one()) mma_commit(&m.drain[t]);  // products in flight end before TMEM goes back
        __syncwarp();
        mbar_wait_bounded(&m.drain[t], 0);
      }
    } else if (warp == K::kRowWarp) {
      K::load_rows(a, m, smem, lane);
    }
  }
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  if (warp == K::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <typename T, typename TQ, int D>
cudaError_t mass_typed(const spg_params& p, MassArgs& a, const void* q, cudaStream_t st) {
  using K = Kernel<T, TQ, D>;
  // (without rows the map is not used; any readable address describes it)
  if (a.sh.total_q > 0 && !make_q_tmap(&a.tmq, q, p, a.sh.total_q, kTile)) return cudaErrorNotSupported;
  const auto kern = k_mass<T, TQ, D>;
  const size_t smem = 1024 + K::Lay::misc + sizeof(typename K::M);
  const cudaError_t e = ensure_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(std::min(device_sm_count(), kMaxCtas)), dim3(K::kThreads), smem, st, a);
}

}  // namespace

static_assert(kPartCounterBytes >= sizeof(int32_t) * kMaxCtas, "a counter per CTA");
size_t mass_workspace_bytes() { return sizeof(float) * 2 * kMaxCtas * kItemTokens; }

cudaError_t launch_mass(const spg_params& p, const ChunkRows& r, const void* k_pool, const void* k_scale,
                        const float* lse, const float* mass_in, float* mass_out, float decay, const Workspace& ws,
                        cudaStream_t stream) {
  // A decode step has one row per sequence: the keys' bytes bound the work and
  // the page stream reads them faster (one token of each of 16 sequences at
  // 10K, GQA 32/8, cold caches: bf16 keys in 16-token pages 70 us there and 83
  // here, int8 keys in 64-token pages 60 and 87).  With more rows than
  // sequences one of them may have nearly all, and the tiles take them better:
  // 127 tokens and a piece of 129 over 2K to 4K 246 us there and 187 here, 31
  // tokens and a piece of 33 over 32K 244 and 93 (two drafted tokens of each of
  // 16 sequences would be 70 and 83).  Where other sequences have none, a piece
  // of 256 rows beside 255 empty ones, 474 and 271, stays there: the host
  // cannot tell it from a decode step.
  if (r.total_q <= p.batch) {
    const cudaError_t e = launch_mass_few(p, r, k_pool, k_scale, lse, mass_in, mass_out, decay, ws.err, stream);
    if (e != cudaErrorNotSupported) return e;
  }
  MassArgs a{};
  a.sh.q_start = r.q_start;
  a.sh.seq_lens = r.seq_lens;
  a.sh.B = p.batch;
  a.sh.Hkv = p.num_kv_heads;
  a.sh.g_log2 = log2_of(p.num_q_heads / p.num_kv_heads);
  a.sh.total_q = r.total_q;
  a.sh.max_tokens = p.max_pages_per_seq * p.page_size;
  a.k_pool = k_pool;
  a.k_scale = static_cast<const __half*>(k_scale);
  a.page_table = r.page_table;
  a.lse = lse;
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  a.err = ws.err;
  a.counters = ws.part_counters;
  a.part = ws.mass_part;
  a.Hkv = p.num_kv_heads;
  a.S = p.page_size;
  a.s_log2 = log2_of(p.page_size);
  a.MP = p.max_pages_per_seq;
  a.n_phys = p.num_phys_pages;
  a.scale_log2 = (p.softmax_scale > 0.f ? p.softmax_scale : 1.0f / sqrtf(static_cast<float>(p.head_dim))) * kLog2e;
  a.decay = decay;
#define SPG_MASS(T, TQ) \
  return p.head_dim == 128 ? mass_typed<T, TQ, 128>(p, a, r.q, stream) : mass_typed<T, TQ, 64>(p, a, r.q, stream)
  if (p.kv_dtype == SPG_F16) SPG_MASS(__half, __half);
  if (p.kv_dtype == SPG_BF16) SPG_MASS(__nv_bfloat16, __nv_bfloat16);
  if (p.q_dtype == SPG_F16) SPG_MASS(int8_t, __half);
  SPG_MASS(int8_t, __nv_bfloat16);
#undef SPG_MASS
}

}  // namespace spg
