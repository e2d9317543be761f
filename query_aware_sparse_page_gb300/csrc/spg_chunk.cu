// Attention of a ragged chunk of new tokens over the paged cache
// (paged_chunk_attention), on the tcgen05 tensor cores.
//
// An item is up to 256 rows of one (batch, kv-head): the group's query heads
// share their kv-head's keys, so row r is head r % G of new token r / G, at
// cache position pos0 + r / G, and sees the tokens up to there.  A step is
// 128 tokens of an item:
//   S = Q K^T      both from shared memory, S in TMEM
//   P = exp2(scale S - m)  by the softmax warps, one row per thread, written
//                  back over S as 16-bit pairs
//   O += P V       A from TMEM, V from shared memory (its rows are the
//                  contraction: MN-major), O in TMEM
// with the running maximum m and sum l of the softmax per row.  m is only
// raised when a logit exceeds it by more than 2^kSlack: p stays at most
// 2^kSlack, O is rescaled in the rare step that raises it, and out = O / l
// does not depend on m.
//
// One CTA per SM: two softmax warpgroups, one issuing thread, and the
// warps that fill the K and V rings.  With more than 128 rows the two
// warpgroups have 128 rows each (streams of Q tiles 0 and 1 over the same
// keys); with fewer they share the rows and take alternate steps, and their
// two (m, l, O) are joined at the end of the item.  While one stream is in
// its softmax the tensor cores work for the other.
//
// The steps of all items, in the order (sequence, kv-head, rows), are dealt
// out to the CTAs in equal contiguous shares, whatever the lengths: an item
// that crosses a border leaves (m, l, O) of its parts in the workspace, and
// the part that arrives last joins them in a fixed order.  No CTA waits for
// another.
//
// Keys and values of 16-bit pools come by TMA, one copy per page and 64
// channels (K: the pages' rows of a half follow one another, so that 128
// tokens are one operand) or per page (V).  int8 pages are turned into exact
// 16-bit codes by four warps; the key scales then multiply the logits and the
// value scales (times 16, undone at the end) the probabilities.
//
// Roundings: P to the 16-bit type (as the products take it) and the result;
// everything else is fp32.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "spg_chunk_common.cuh"
#include "spg_internal.h"
#include "spg_tcgen05.cuh"

namespace spg {
namespace {

constexpr int kTile = 128;           // rows of a Q tile, tokens of a step
constexpr int kItemRows = 2 * kTile;
constexpr int kMaxCtas = 160;        // shares of the plan (one per SM)
constexpr int kMaxParts = 32;        // most parts an average item is split into
constexpr uint32_t kTmemCols = 512;  // S0 S1 O0 O1, 128 columns each

struct ChunkArgs {
  CUtensorMap tmq, tmk, tmv;
  int v_whole;  // tmv takes a whole page per copy
  const void *k_pool, *v_pool;
  const __half *k_scale, *v_scale;
  const int32_t *q_start, *page_table, *seq_lens;
  void* out;
  float* lse;
  int32_t *err, *counters;
  float* part;  // [2 * CTAs][D + 2][part_rows]: O by channel, then m and l, so that a warp's rows are neighbours
  int B, Hkv, G, S, MP, n_phys, total_q, part_rows;
  float scale_log2;
};

// ---- the plan -----------------------------------------------------------------------
// sum of ceil((pos0 + i q) / 128) for i = 1 .. m: the steps of a sequence's
// first m full items, q = 256 / G new tokens each
__device__ __forceinline__ long long full_item_steps(int pos0, int q, int m) {
  if (q >= kTile) return static_cast<long long>(m) * ((pos0 + kTile - 1) / kTile) + static_cast<long long>(q / kTile) * m * (m + 1) / 2;
  long long sum = 0;
  const int per = kTile / q;
  for (int r = 1; r <= per && r <= m; ++r) {
    const long long cnt = (m - r) / per + 1;
    sum += cnt * ((pos0 + r * q + kTile - 1) / kTile) + cnt * (cnt - 1) / 2;
  }
  return sum;
}
// steps of the sequence's first `items` items (one kv-head)
__device__ __forceinline__ long long item_steps(const ChunkSeq& s, int q, int items) {
  const int full = min(items, s.n / q);
  long long sum = full_item_steps(s.pos0, q, full);
  if (items > full) sum += (s.L + kTile - 1) / kTile;
  return sum;
}

struct Plan {
  long long total, lo, hi;  // steps in all, and this CTA's
  long long item_first;     // first step of the item that lo lies in
  int ctas, b, h, item;
};

// one whole warp
__device__ void make_plan(const ChunkArgs& a, Plan* out, int lane) {
  const int q = kItemRows / a.G;
  long long total = 0, items = 0;
  int32_t bad = 0;
  for (int b = lane; b < a.B; b += 32) {
    const ChunkSeq s = chunk_seq(a.q_start, a.seq_lens, b, a.total_q, a.MP * a.S, bad);
    const int ni = (s.n + q - 1) / q;
    total += a.Hkv * item_steps(s, q, ni);
    items += static_cast<long long>(a.Hkv) * ni;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    items += __shfl_xor_sync(0xffffffffu, items, o);
  }
  if (bad && blockIdx.x == 0) record_error(a.err, bad);
  Plan p{};
  p.total = total;
  long long n = min(static_cast<long long>(gridDim.x), total);
  n = min(n, items * kMaxParts);
  p.ctas = static_cast<int>(n);
  const int c = blockIdx.x;
  if (c >= n) {
    if (lane == 0) *out = p;  // lo = hi = 0: nothing to do
    return;
  }
  p.lo = c * total / n;
  p.hi = (c + 1) * total / n;
  long long base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    long long w = 0;
    ChunkSeq s{};
    if (b < a.B) {
      s = chunk_seq(a.q_start, a.seq_lens, b, a.total_q, a.MP * a.S, bad);
      w = a.Hkv * item_steps(s, q, (s.n + q - 1) / q);
    }
    long long incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const long long first = base + incl - w;
    if (p.lo >= first && p.lo < first + w) {  // one lane
      const long long per_head = w / a.Hkv;
      p.b = b;
      p.h = static_cast<int>((p.lo - first) / per_head);
      const long long rest = (p.lo - first) % per_head;
      int x = 0, y = (s.n + q - 1) / q - 1;  // the last item that starts at or before rest
      while (x < y) {
        const int mid = (x + y + 1) >> 1;
        if (item_steps(s, q, mid) <= rest) x = mid; else y = mid - 1;
      }
      p.item = x;
      p.item_first = first + p.h * per_head + item_steps(s, q, x);
      *out = p;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
    if (base > p.lo) break;
  }
}

// A CTA's share of one item: steps [k0, k1) of its nk.
struct Seg {
  ChunkSeq sq;
  int b, h, row0, n_rows, last, k0, k1, nk;
  long long item_first;
};
struct SegIter {
  long long pos, hi, item_first;
  int b, h, item;
  ChunkSeq sq;
  __device__ SegIter(const ChunkArgs& a, const Plan& p) : pos(p.lo), hi(p.hi), item_first(p.item_first), b(p.b), h(p.h), item(p.item) {
    if (pos < hi) load(a);
  }
  __device__ void load(const ChunkArgs& a) {
    int32_t bad = 0;
    sq = chunk_seq(a.q_start, a.seq_lens, b, a.total_q, a.MP * a.S, bad);
  }
  __device__ bool next(const ChunkArgs& a, Seg& s) {
    if (pos >= hi) return false;
    const int q = kItemRows / a.G;
    s.sq = sq;
    s.b = b;
    s.h = h;
    s.row0 = item * kItemRows;
    s.n_rows = min(kItemRows, sq.n * a.G - s.row0);
    s.last = sq.pos0 + min((item + 1) * q, sq.n) - 1;  // the last token any row sees
    s.nk = s.last / kTile + 1;
    s.item_first = item_first;
    s.k0 = static_cast<int>(pos - item_first);
    s.k1 = static_cast<int>(min(static_cast<long long>(s.nk), hi - item_first));
    pos = item_first + s.k1;
    if (s.k1 == s.nk) {
      item_first += s.nk;
      if (++item * q >= sq.n) {
        item = 0;
        if (++h == a.Hkv) {
          h = 0;
          if (pos < hi) do { ++b; load(a); } while (sq.n == 0);
        }
      }
    }
    return true;
  }
};

// ---- shared memory ---------------------------------------------------------------------
template <int D, bool I8>
struct Layout {
  static constexpr int NH = D / 64;  // 64-channel halves
  static constexpr uint32_t kHalf = kTile * 128;
  static constexpr uint32_t kTileBytes = NH * kHalf;
  static constexpr int KST = D == 128 ? (I8 ? 2 : 3) : 4, VST = D == 128 ? 2 : 4;
  static constexpr uint32_t q_off = 0, k_off = 2 * kTileBytes, v_off = k_off + KST * kTileBytes;
  static constexpr uint32_t misc = v_off + VST * kTileBytes;
};
template <int KST, int VST, bool I8>
struct Misc {
  uint64_t q_full, q_empty, k_full[KST], k_empty[KST], v_full[VST], v_empty[VST], s_full[2], p_full[2][2], o_full[2], drain;
  Plan plan;
  uint32_t tmem;
  int last;
  float ml[kTile][2];                            // stream 1's m and l, joined by stream 0
  alignas(16) float scales[I8 ? VST : 1][2][I8 ? kTile : 1];  // int8: scale * key scale, 16 * value scale of a step's tokens
};

// A wait: false, and recorded, when it ran out (as mbar_wait_bounded, in few
// instructions: the issuing warp's path has five of them per step).
struct Waiter {
  int32_t* err;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t phase) const {
    if (mbar_try_wait(bar, phase & 1)) return true;
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
#pragma unroll 1
    for (int i = 0; i < (1 << 22); ++i) {
      if (mbar_try_wait(bar, phase & 1)) return true;
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
      if (t - t0 > 100ull * 1000 * 1000) break;
    }
    record_error(err, SPG_DEVERR_TIMEOUT);
    return false;
  }
};

template <typename T, typename TQ, int D>
struct Kernel {
  static constexpr bool I8 = sizeof(T) == 1;
  using Lay = Layout<D, I8>;
  static constexpr int KST = Lay::KST, VST = Lay::VST, NH = Lay::NH;
  using M = Misc<KST, VST, I8>;
  // warpgroups 0, 1: softmax; then, 16-bit: the issuing warp, the K and the V
  // warp and an idle one; int8: four converting warps, then the issuing warp
  // and three idle ones
  static constexpr int kWarps = I8 ? 16 : 12, kThreads = kWarps * 32;
  static constexpr int kMmaWarp = I8 ? 12 : 8, kFillWarp = I8 ? 8 : 9;
  // registers per thread: at launch (65536 / kThreads, a multiple of 8), then
  // each warpgroup's share of the same total; a softmax thread holds a whole
  // row of 128 logits
  static constexpr int kRegs = I8 ? 128 : 168, kRegsSoftmax = I8 ? 184 : 208, kRegsFill = I8 ? 88 : 88, kRegsMma = I8 ? 56 : 88;
  static_assert(2 * kRegsSoftmax + kRegsFill + (I8 ? kRegsMma : 0) <= (I8 ? 4 : 3) * kRegs, "the block's registers");
  static constexpr int kFillThreads = 128;
  // fp16 holds p * 16 * (value scale) for scales up to 255
  static constexpr float kSlack = I8 ? 4.f : 8.f;
  static constexpr float kVScale = I8 ? 16.f : 1.f;

  // ---- the issuing warp: all of it waits, one elected lane issues --------------------------
  static __device__ bool issue(const ChunkArgs& a, M& m, uint32_t smem, uint32_t tmem) {
    const auto wait = [&](uint64_t* bar, uint32_t phase) {  // the whole warp goes on, or none of it
      return __all_sync(0xffffffffu, Waiter{a.err}(bar, phase)) != 0;
    };
    constexpr uint32_t idS = instr_desc<TQ>(kTile, kTile, false), idO = instr_desc<TQ>(kTile, D, true);
    constexpr uint32_t kStep = Lay::kTileBytes >> 4;  // descriptors count 16 bytes
    // what the whole warp agrees on, taken from one lane so that it can be kept once per warp
    const auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    tmem = uniform(tmem);
    const uint32_t dq = desc_k_major(smem + Lay::q_off), dk = desc_k_major(smem + Lay::k_off);
    // V blocks of 64 columns: within a page (TMA), or over the whole tile (converted)
    const uint32_t dv = desc_mn_major(smem + Lay::v_off, I8 ? Lay::kHalf : static_cast<uint32_t>(a.S) * 128u);
    uint32_t v_at[kTile / 16];  // the tile's tokens 16 ks
#pragma unroll
    for (int ks = 0; ks < kTile / 16; ++ks) {
      const uint32_t tok = 16 * ks, S = a.S;
      v_at[ks] = (I8 ? tok * 128u : (tok / S) * (S * D * 2) + (tok % S) * 128u) >> 4;
    }
    uint32_t sc[2] = {0, 0}, qc = 0;          // rounds of the barriers
    uint32_t ki = 0, vi = 0, kr = 0, vr = 0;          // stage and round of the rings
    const auto next_k = [&] {
      if (++ki == KST) ki = 0, ++kr;
    };
    const auto next_v = [&] {
      if (++vi == VST) vi = 0, ++vr;
    };
    const auto S = [&](int t, int qt) {
      const uint32_t q = dq + qt * kStep, k = dk + ki * kStep;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = ((ks >> 2) * Lay::kHalf + (ks & 3) * 32u) >> 4;
        mma_ss(tmem + t * 128, q + off, k + off, idS, ks > 0);
      }
      mma_commit(&m.s_full[t]);
    };
    // half the step's tokens: the first half starts while the second is in its softmax
    const auto PV = [&](int t, int half, bool acc) {
      const uint32_t v = dv + vi * kStep;
#pragma unroll
      for (int i = 0; i < kTile / 32; ++i) {
        const int ks = half * (kTile / 32) + i;
        mma_ts(tmem + 256 + t * 128, tmem + t * 128 + 8 * ks, v + v_at[ks], idO, acc || ks > 0);
      }
    };
    SegIter it(a, m.plan);
    Seg s;
    while (uniform(it.next(a, s))) {
      const int n = uniform(s.k1 - s.k0);
      if (!wait(&m.q_full, qc++)) return false;
      if (uniform(s.n_rows) > kTile) {  // two tiles of rows over the same keys
        if (!wait(&m.k_full[ki], kr)) return false;
        tc_fence_after();
        if (elect_one()) {
          S(0, 0);
          S(1, 1);
          mma_commit(&m.k_empty[ki]);
        }
        __syncwarp();
        next_k();
        for (int j = 0; j < n; ++j) {
          if (!wait(&m.v_full[vi], vr)) return false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t == 0 && j + 1 < n && !wait(&m.k_full[ki], kr)) return false;
            if (!wait(&m.p_full[t][0], sc[t])) return false;
            tc_fence_after();
            if (elect_one()) PV(t, 0, j > 0);
            __syncwarp();
            if (!wait(&m.p_full[t][1], sc[t]++)) return false;
            tc_fence_after();
            if (elect_one()) {
              PV(t, 1, true);
              if (j + 1 < n) S(t, t);
              if (t == 1) {
                mma_commit(&m.v_empty[vi]);
                if (j + 1 < n) mma_commit(&m.k_empty[ki]);
              }
            }
            __syncwarp();
          }
          next_v();
          if (j + 1 < n) next_k();
        }
      } else {  // one tile of rows, the streams take alternate steps
        for (int j = 0; j < min(n, 2); ++j) {
          if (!wait(&m.k_full[ki], kr)) return false;
          tc_fence_after();
          if (elect_one()) {
            S(j, 0);
            mma_commit(&m.k_empty[ki]);
          }
          __syncwarp();
          next_k();
        }
        for (int j = 0; j < n; ++j) {
          const int t = j & 1;
          if (!wait(&m.v_full[vi], vr)) return false;
          if (!wait(&m.p_full[t][0], sc[t])) return false;
          tc_fence_after();
          if (elect_one()) PV(t, 0, j > 1);
          __syncwarp();
          if (!wait(&m.p_full[t][1], sc[t]++)) return false;
          tc_fence_after();
          if (elect_one()) {
            PV(t, 1, true);
            mma_commit(&m.v_empty[vi]);
          }
          __syncwarp();
          next_v();
          if (j + 2 < n) {
            if (!wait(&m.k_full[ki], kr)) return false;
            tc_fence_after();
            if (elect_one()) {
              S(t, 0);
              mma_commit(&m.k_empty[ki]);
            }
            __syncwarp();
            next_k();
          }
        }
      }
      if (elect_one()) {
        mma_commit(&m.q_empty);
        mma_commit(&m.o_full[0]);
        mma_commit(&m.o_full[1]);
      }
      __syncwarp();
    }
    return true;
  }

  // Q tiles of a segment (one thread)
  static __device__ bool load_q(const ChunkArgs& a, M& m, uint8_t* smem, const Seg& s, uint32_t count) {
    if (count > 0 && !Waiter{a.err}(&m.q_empty, count - 1)) return false;
    const int tiles = s.n_rows > kTile ? 2 : 1;
    mbar_arrive_expect_tx(&m.q_full, tiles * Lay::kTileBytes);
    for (int t = 0; t < tiles; ++t)
      for (int hf = 0; hf < NH; ++hf)
        tma_tile_4d(smem + Lay::q_off + t * Lay::kTileBytes + hf * Lay::kHalf, &a.tmq, hf * 64, 0, s.h,
                    s.sq.start + (s.row0 + t * kTile) / a.G, &m.q_full);
    return true;
  }

  // ---- 16-bit pools: one warp fills the K ring, one the V ring -----------------------------
  static __device__ bool fill(const ChunkArgs& a, M& m, uint8_t* smem, bool is_v, int lane) {
    const Waiter wait{a.err};
    const int S = a.S, ppt = kTile / S;
    const uint32_t page_bytes = static_cast<uint32_t>(S) * D * 2;
    uint32_t c = 0, qc = 0;
    SegIter it(a, m.plan);
    Seg s;
    while (it.next(a, s)) {
      const int32_t* pt = a.page_table + static_cast<size_t>(s.b) * a.MP;
      bool ok = true;
      if (!is_v) {
        if (lane == 0) ok = load_q(a, m, smem, s, qc);
        ++qc;
        if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) return false;
      }
      const auto page_of = [&](int k) {  // the lane's page of step k; -1: none, or a bad one
        const int lp = k * ppt + lane;
        if (lane >= ppt || k >= s.k1 || lp * S > s.last) return -1;
        const int page = pt[lp];
        return page >= 0 && page < a.n_phys ? page : -1;
      };
      int page = page_of(s.k0);
      for (int k = s.k0; k < s.k1; ++k) {
        const int ahead = page_of(k + 1);
        const uint32_t stage = is_v ? c % VST : c % KST;
        uint64_t* full = is_v ? &m.v_full[stage] : &m.k_full[stage];
        const uint32_t round = is_v ? c / VST : c / KST;
        if (lane == 0 && round > 0) ok = wait(is_v ? &m.v_empty[stage] : &m.k_empty[stage], round - 1);
        if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) return false;
        uint8_t* dst = smem + (is_v ? Lay::v_off : Lay::k_off) + stage * Lay::kTileBytes;
        const int lp = k * ppt + lane;
        // V rows that hold no token must be zeros (p = 0 there, and 0 times
        // what the pool holds could be NaN); K rows may be anything, their
        // logits are masked
        const bool part = is_v && page >= 0 && (lp + 1) * S > s.sq.L;
        const bool copy = page >= 0 && !part;
        const unsigned by_hand = __ballot_sync(0xffffffffu, is_v && lane < ppt && !copy);
        if (by_hand) {
          for (unsigned left = by_hand; left; left &= left - 1) {
            const int l = __ffs(left) - 1;
            const int pg = __shfl_sync(0xffffffffu, page, l);
            const int rows = pg >= 0 ? min(S, s.sq.L - (k * ppt + l) * S) : 0;
            const uint8_t* src = static_cast<const uint8_t*>(a.v_pool) + (static_cast<size_t>(max(pg, 0)) * a.Hkv + s.h) * page_bytes;
            for (int i = lane; i < S * D / 8; i += 32) {
              const int r = i / (D / 8), x = i % (D / 8);
              uint4 w = make_uint4(0u, 0u, 0u, 0u);
              if (r < rows) w = *reinterpret_cast<const uint4*>(src + r * (D * 2) + x * 16);
              *reinterpret_cast<uint4*>(dst + l * page_bytes + (x >> 3) * (S * 128) + r * 128 + (((x & 7) ^ (r & 7)) << 4)) = w;
            }
          }
          fence_proxy_async();
        }
        const int copies = __popc(__ballot_sync(0xffffffffu, copy));
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full, copies * page_bytes);
        __syncwarp();
        if (copy) {
          const int row = (page * a.Hkv + s.h) * S;
          if (is_v && a.v_whole) {
            tma_tile_3d(dst + lane * page_bytes, &a.tmv, 0, row, 0, full);
          } else {
#pragma unroll
            for (int hf = 0; hf < NH; ++hf) {
              if (is_v)
                tma_tile_2d(dst + lane * page_bytes + hf * S * 128, &a.tmv, hf * 64, row, full);
              else
                tma_tile_2d(dst + hf * Lay::kHalf + lane * S * 128, &a.tmk, hf * 64, row, full);
            }
          }
        }
        ++c;
        page = ahead;
      }
    }
    // copies still in flight land before the CTA leaves: their consumers wait for them
    return true;
  }

  // ---- int8 pools: four warps turn codes into 16-bit tiles -----------------------------------
  // four bytes -> two pairs, exact
  static __device__ __forceinline__ void widen4(uint32_t r, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = r ^ 0x80808080u;
    if constexpr (std::is_same<TQ, __half>::value) {
      // the byte under an exponent byte is 1024 + code + 128
      uint32_t x, y;
      asm("prmt.b32 %0, %1, %2, 0x4140;" : "=r"(x) : "r"(u), "r"(0x64646464u));
      asm("prmt.b32 %0, %1, %2, 0x4342;" : "=r"(y) : "r"(u), "r"(0x64646464u));
      const __half2 bias = __floats2half2_rn(1152.f, 1152.f);
      const __half2 hx = __hsub2(*reinterpret_cast<const __half2*>(&x), bias);
      const __half2 hy = __hsub2(*reinterpret_cast<const __half2*>(&y), bias);
      lo = *reinterpret_cast<const uint32_t*>(&hx);
      hi = *reinterpret_cast<const uint32_t*>(&hy);
    } else {
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)  // 2^23 + code + 128
        f[i] = __uint_as_float(0x4b000000u | ((u >> (8 * i)) & 0xffu)) - 8388736.f;
      lo = pack2<TQ>(f[0], f[1]);
      hi = pack2<TQ>(f[2], f[3]);
    }
  }

  static constexpr int kCpt = D / 16;                          // 16-byte pieces of a row of codes
  static constexpr int kPieces = kTile * kCpt / kFillThreads;  // of one tile, per thread

  static __device__ __forceinline__ void fetch(const ChunkArgs& a, const Seg& s, const void* pool, int k, int tid, uint4 (&w)[kPieces]) {
    const int32_t* pt = a.page_table + static_cast<size_t>(s.b) * a.MP;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int x = tid + kFillThreads * i, t = k * kTile + x / kCpt;
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (k < s.k1 && t <= s.last) {
        const int page = pt[t / a.S];
        if (page >= 0 && page < a.n_phys)
          w[i] = *reinterpret_cast<const uint4*>(static_cast<const int8_t*>(pool) +
                                                 ((static_cast<size_t>(page) * a.Hkv + s.h) * a.S + t % a.S) * D + 16 * (x % kCpt));
      }
    }
  }
  static __device__ __forceinline__ void widen(uint8_t* dst, int tid, const uint4 (&w)[kPieces]) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int x = tid + kFillThreads * i, r = x / kCpt, c = 2 * (x % kCpt);  // two 16-byte pieces of 16-bit values
      uint4 lo, hi;
      widen4(w[i].x, lo.x, lo.y);
      widen4(w[i].y, lo.z, lo.w);
      widen4(w[i].z, hi.x, hi.y);
      widen4(w[i].w, hi.z, hi.w);
      uint8_t* row = dst + (c >> 3) * Lay::kHalf + r * 128;
      *reinterpret_cast<uint4*>(row + (((c & 7) ^ (r & 7)) << 4)) = lo;
      *reinterpret_cast<uint4*>(row + ((((c & 7) + 1) ^ (r & 7)) << 4)) = hi;
    }
  }
  static __device__ bool convert(const ChunkArgs& a, M& m, uint8_t* smem, int tid) {
    const Waiter wait{a.err};
    uint32_t c = 0, qc = 0;
    SegIter it(a, m.plan);
    Seg s;
    uint4 wk[kPieces], wv[kPieces];
    while (it.next(a, s)) {
      if (tid == 0 && !load_q(a, m, smem, s, qc)) return false;  // the others run out at the next empty stage
      ++qc;
      const int32_t* pt = a.page_table + static_cast<size_t>(s.b) * a.MP;
      fetch(a, s, a.k_pool, s.k0, tid, wk);
      fetch(a, s, a.v_pool, s.k0, tid, wv);
      for (int k = s.k0; k < s.k1; ++k) {
        const uint32_t ks = c % KST, vs = c % VST;
        float sk = 0.f, sv = 0.f;  // of the step's token tid
        {
          const int t = k * kTile + tid;
          if (t <= s.last) {
            const int page = pt[t / a.S];
            if (page >= 0 && page < a.n_phys) {
              const size_t at = (static_cast<size_t>(page) * a.Hkv + s.h) * a.S + t % a.S;
              sk = __half2float(a.k_scale[at]) * a.scale_log2;
              sv = __half2float(a.v_scale[at]) * kVScale;
            }
          }
        }
        if (c >= KST && !wait(&m.k_empty[ks], c / KST - 1)) return false;
        widen(smem + Lay::k_off + ks * Lay::kTileBytes, tid, wk);
        fence_proxy_async();
        mbar_arrive(&m.k_full[ks]);
        fetch(a, s, a.k_pool, k + 1, tid, wk);
        if (c >= VST && !wait(&m.v_empty[vs], c / VST - 1)) return false;
        m.scales[vs][0][tid] = sk;
        m.scales[vs][1][tid] = sv;
        widen(smem + Lay::v_off + vs * Lay::kTileBytes, tid, wv);
        fence_proxy_async();
        mbar_arrive(&m.v_full[vs]);
        fetch(a, s, a.v_pool, k + 1, tid, wv);
        ++c;
      }
    }
    return true;
  }

  // ---- softmax ------------------------------------------------------------------------------------
  // A thread's row over the steps of one stream; m in the log2 domain.
  struct Row {
    float m, l;
  };

  // channel 0 of a row in a slot; the next channel is part_rows further
  static __device__ __forceinline__ float* part_at(const ChunkArgs& a, int slot, int row) {
    return a.part + static_cast<size_t>(slot) * (D + 2) * a.part_rows + row;
  }

  // out and lse of a row from its unnormalised O (element i by o(i)), m and l
  static __device__ __forceinline__ size_t out_row(const ChunkArgs& a, const Seg& s, int r) {
    const int rr = s.row0 + r;
    return static_cast<size_t>(s.sq.start + rr / a.G) * (a.Hkv * a.G) + s.h * a.G + rr % a.G;
  }

  static __device__ void softmax(const ChunkArgs& a, M& m, uint32_t tmem, int warp, int lane) {
    // after a wait that ran out the others are skipped: every thread still
    // reaches every named barrier (the results are not valid then)
    bool dead = false;
    const auto wait = [&](uint64_t* bar, uint32_t phase) {
      if (!dead && !Waiter{a.err}(bar, phase)) dead = true;
    };
    const int t = warp >> 2, tid = threadIdx.x;  // stream, 0 .. 255
    const int tile_row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tS = lanes + t * 128, tO = lanes + 256 + t * 128;
    uint32_t sc = 0, oc = 0, vc = 0;
    SegIter it(a, m.plan);
    Seg s;
    while (it.next(a, s)) {
      const bool two = s.n_rows > kTile;
      const int r = two ? t * kTile + tile_row : tile_row;  // row of the item
      const int pos = s.sq.pos0 + (s.row0 + r) / a.G;
      const int pos_first = s.sq.pos0 + (s.row0 + (two ? t * kTile : 0)) / a.G;
      const int32_t* pt = a.page_table + static_cast<size_t>(s.b) * a.MP;
      // does the segment have a bad page at all?
      bool any_bad = false;
      {
        const int p1 = min(s.k1 * kTile - 1, s.last) / a.S;
        for (int lp = s.k0 * kTile / a.S + lane; lp <= p1; lp += 32) {
          const int page = pt[lp];
          any_bad |= page < 0 || page >= a.n_phys;
        }
        any_bad = __any_sync(0xffffffffu, any_bad);
        if (any_bad && warp == 0 && lane == 0) record_error(a.err, SPG_DEVERR_PAGE_ID);
      }
      Row row{-INFINITY, 0.f};
      const int step = two ? 1 : 2;
      for (int k = s.k0 + (two ? 0 : t); k < s.k1; k += step) {
        uint32_t stage = 0;
        if constexpr (I8) {
          const uint32_t c = vc + (k - s.k0);
          stage = c % VST;
          wait(&m.v_full[stage], c / VST);
        }
        wait(&m.s_full[t], sc);
        ++sc;
        tc_fence_after();
        uint32_t x[kTile];
#pragma unroll
        for (int c = 0; c < kTile; c += 32) tmem_ld32(x + c, tS + c);
        tmem_wait_ld();
        const auto f = [&](int c) { return __uint_as_float(x[c]); };
        if constexpr (I8) {
          const float* ks = m.scales[stage][0];
#pragma unroll
          for (int c = 0; c < kTile; c += 4) {
            const float4 w = *reinterpret_cast<const float4*>(ks + c);
            const float2 u = unpack_f32x2(mul_f32x2(f32x2(f(c), f(c + 1)), f32x2(w.x, w.y)));
            const float2 v = unpack_f32x2(mul_f32x2(f32x2(f(c + 2), f(c + 3)), f32x2(w.z, w.w)));
            x[c] = __float_as_uint(u.x);
            x[c + 1] = __float_as_uint(u.y);
            x[c + 2] = __float_as_uint(v.x);
            x[c + 3] = __float_as_uint(v.y);
          }
        }
        const int t0 = k * kTile;
        if (t0 + kTile - 1 > pos_first || any_bad) {
          // the step's last tokens are hidden from some row, or a page is bad (per 16 tokens)
          unsigned bad16 = 0;
          if (any_bad)
            for (int c = 0; c < kTile; c += 16)
              if (t0 + c <= s.last) {
                const int page = pt[(t0 + c) / a.S];
                if (page < 0 || page >= a.n_phys) bad16 |= 1u << (c / 16);
              }
          const int lim = pos - t0;
#pragma unroll
          for (int c = 0; c < kTile; ++c)
            if (c > lim || ((bad16 >> (c / 16)) & 1u)) x[c] = 0xff800000u;  // -inf
        }
        float mx[4];  // chains that do not wait for one another
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = fmaxf(f(c), f(c + 4));
#pragma unroll
        for (int c = 8; c < kTile; c += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = fmaxf(fmaxf(mx[i], f(c + i)), f(c + 4 + i));
        float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if constexpr (!I8) top *= a.scale_log2;
        const bool raise = top > row.m + kSlack;  // -inf + kSlack = -inf: the first finite logit
        if (__any_sync(0xffffffffu, raise)) {
          const float mn = raise ? top : row.m;
          const float factor = row.m == -INFINITY ? (raise ? 0.f : 1.f) : ex2(row.m - mn);
          row.m = mn;
          row.l *= factor;
          if (k >= s.k0 + step) {  // O holds earlier steps (all done: S of this step was issued after them)
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(o, tO + c);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
              tmem_st32(tO + c, o);
            }
          }
        }
        const float mm = row.m == -INFINITY ? 0.f : row.m;
        const uint64_t nm = f32x2(-mm, -mm), sc2 = f32x2(a.scale_log2, a.scale_log2);
        uint64_t l0 = f32x2(0.f, 0.f), l1 = l0;
#pragma unroll
        for (int c0 = 0; c0 < kTile; c0 += 32) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c = c0 + 2 * i;
            const uint64_t z = f32x2(f(c), f(c + 1));
            const float2 e = unpack_f32x2(I8 ? add_f32x2(z, nm) : fma_f32x2(z, sc2, nm));
            float2 p = make_float2(ex2(e.x), ex2(e.y));
            if (i & 1) l1 = add_f32x2(l1, f32x2(p.x, p.y)); else l0 = add_f32x2(l0, f32x2(p.x, p.y));
            if constexpr (I8) {
              const float2 vs = *reinterpret_cast<const float2*>(&m.scales[stage][1][c]);
              p.x *= vs.x;
              p.y *= vs.y;
            }
            w[i] = pack2<TQ>(p.x, p.y);
          }
          tmem_st16(tS + c0 / 2, w);
          if (c0 % (kTile / 2)) {
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&m.p_full[t][c0 / (kTile / 2)]);
          }
        }
        const float2 s0 = unpack_f32x2(l0), s1 = unpack_f32x2(l1);
        row.l += (s0.x + s0.y) + (s1.x + s1.y);
      }
      vc += s.k1 - s.k0;

      // ---- the segment's end ----
      const bool whole = s.k0 == 0 && s.k1 == s.nk;
      wait(&m.o_full[t], oc);
      float f0 = 1.f, f1 = 0.f;
      if (!two) {  // the rows' two streams
        if (t == 1) {
          m.ml[tile_row][0] = row.m;
          m.ml[tile_row][1] = row.l;
        } else {
          wait(&m.o_full[1], oc);
        }
        bar_sync(1, 256);
        if (t == 0) {
          const float m1 = m.ml[tile_row][0], l1 = m.ml[tile_row][1];
          const float mm = fmaxf(row.m, m1);
          f0 = row.m == -INFINITY ? 0.f : ex2(row.m - mm);
          f1 = m1 == -INFINITY ? 0.f : ex2(m1 - mm);
          row.l = row.l * f0 + l1 * f1;
          row.m = mm;
        }
      }
      ++oc;
      tc_fence_after();
      if (two || t == 0) {
        const bool live = r < s.n_rows;
        const bool both = !two && s.k1 - s.k0 > 1;  // stream 1 has had a step
        const float inv = row.l > 0.f ? (1.f / kVScale) / row.l : 0.f;
        if (whole) {
          f0 *= inv;
          f1 *= inv;
        }
        const size_t orow = live ? out_row(a, s, r) : 0;
        const int c_slot = 2 * blockIdx.x + (s.k0 > 0 ? 0 : 1);
        float* part = part_at(a, c_slot, live ? r : 0);
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(o, tO + c);
          tmem_wait_ld();
          // f0 = 0 stands for rows that saw nothing: their O may not be trusted to be finite
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(f0 == 0.f ? 0.f : __uint_as_float(o[i]) * f0);
          if (both) {
            uint32_t o1[32];
            tmem_ld32(o1, tO + 128 + c);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (f1 != 0.f) o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), f1, __uint_as_float(o[i])));
          }
          if (live && whole) {
            TQ* dst = static_cast<TQ*>(a.out) + orow * D + c;
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(dst + i) = make_uint4(pack2<TQ>(__uint_as_float(o[i]), __uint_as_float(o[i + 1])),
                                                             pack2<TQ>(__uint_as_float(o[i + 2]), __uint_as_float(o[i + 3])),
                                                             pack2<TQ>(__uint_as_float(o[i + 4]), __uint_as_float(o[i + 5])),
                                                             pack2<TQ>(__uint_as_float(o[i + 6]), __uint_as_float(o[i + 7])));
          } else if (live) {
#pragma unroll
            for (int i = 0; i < 32; ++i) __stcg(part + (c + i) * a.part_rows, __uint_as_float(o[i]));
          }
        }
        if (live && whole && a.lse) a.lse[orow] = row.l > 0.f ? (row.m + log2f(row.l)) * kLn2 : -INFINITY;
        if (live && !whole) {
          __stcg(part + D * a.part_rows, row.m);
          __stcg(part + (D + 1) * a.part_rows, row.l);
        }
      }
      tc_fence_before();  // the loads of O come before the next segment's first product
      if (!two) bar_sync(2, 256);
      if (!whole) join(a, m, s, tid);
    }
  }

  // Counts a part of an item in; the last to arrive joins them all.
  static __device__ void join(const ChunkArgs& a, M& m, const Seg& s, int tid) {
    const long long n = m.plan.ctas, total = m.plan.total;
    const int c0 = static_cast<int>(((s.item_first + 1) * n - 1) / total);
    const int c1 = static_cast<int>(((s.item_first + s.nk) * n - 1) / total);
    __threadfence();
    bar_sync(1, 256);
    if (tid == 0) m.last = atomicAdd(&a.counters[c0], 1) == c1 - c0;
    bar_sync(2, 256);
    if (!m.last) return;
    __threadfence();
    // a thread per row, or two with half the channels each
    const bool two = s.n_rows > kTile;
    const int r = two ? tid : tid % kTile, d0 = two ? 0 : tid / kTile * (D / 2), d1 = two ? D : d0 + D / 2;
    if (r < s.n_rows) {
      const auto at = [&](int c) { return part_at(a, c == c0 ? 2 * c + 1 : 2 * c, r); };
      float mm = -INFINITY, l = 0.f;
#pragma unroll 4
      for (int c = c0; c <= c1; ++c) mm = fmaxf(mm, __ldcg(at(c) + D * a.part_rows));
      if (mm == -INFINITY) mm = 0.f;  // every part's weight is 0
#pragma unroll 4
      for (int c = c0; c <= c1; ++c)
        l = fmaf(__ldcg(at(c) + (D + 1) * a.part_rows), ex2(__ldcg(at(c) + D * a.part_rows) - mm), l);
      const float inv = l > 0.f ? (1.f / kVScale) / l : 0.f;
      const size_t orow = out_row(a, s, r);
      TQ* dst = static_cast<TQ*>(a.out) + orow * D;
      for (int d = d0; d < d1; d += 32) {
        float o[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0.f;
        for (int c = c0; c <= c1; ++c) {
          const float* p = at(c);
          const float f = ex2(__ldcg(p + D * a.part_rows) - mm);
          p += d * a.part_rows;
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = fmaf(__ldcg(p + i * a.part_rows), f, o[i]);
        }
#pragma unroll
        for (int i = 0; i < 32; i += 8)
          *reinterpret_cast<uint4*>(dst + d + i) =
              make_uint4(pack2<TQ>(o[i] * inv, o[i + 1] * inv), pack2<TQ>(o[i + 2] * inv, o[i + 3] * inv),
                         pack2<TQ>(o[i + 4] * inv, o[i + 5] * inv), pack2<TQ>(o[i + 6] * inv, o[i + 7] * inv));
      }
      if (d0 == 0 && a.lse) a.lse[orow] = l > 0.f ? (mm + log2f(l)) * kLn2 : -INFINITY;
    }
    if (tid == 0) a.counters[c0] = 0;  // ready for the next call
  }
};

template <typename T, typename TQ, int D>
__global__ void __launch_bounds__((Kernel<T, TQ, D>::kThreads), 1) k_chunk(const __grid_constant__ ChunkArgs a) {
  using K = Kernel<T, TQ, D>;
  using Lay = typename K::Lay;
  using M = typename K::M;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  M& m = *reinterpret_cast<M*>(smem + Lay::misc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    const uint32_t fill = K::I8 ? K::kFillThreads : 1;
    mbar_init(&m.q_full, 1);
    mbar_init(&m.q_empty, 1);
    for (int i = 0; i < K::KST; ++i) {
      mbar_init(&m.k_full[i], fill);
      mbar_init(&m.k_empty[i], 1);
    }
    for (int i = 0; i < K::VST; ++i) {
      mbar_init(&m.v_full[i], fill);
      mbar_init(&m.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m.s_full[i], 1);
      mbar_init(&m.p_full[i][0], 128);
      mbar_init(&m.p_full[i][1], 128);
      mbar_init(&m.o_full[i], 1);
    }
    mbar_init(&m.drain, 1);
    mbar_fence_init();
  }
  if (warp == K::kMmaWarp) tmem_alloc(&m.tmem, kTmemCols);
  pdl_wait();
  if (warp == 0) make_plan(a, &m.plan, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem;

  if (warp < 8) {
    regs_up<K::kRegsSoftmax>();
    K::softmax(a, m, tmem, warp, lane);
  } else {
    if (K::I8 && warp >= 12) regs_down<K::kRegsMma>(); else regs_down<K::kRegsFill>();  // whole warpgroups
    if (warp == K::kMmaWarp) {
      const bool ok = K::issue(a, m, smem_u32(smem), tmem);
      if (!ok) {
        // products in flight end before TMEM goes back
        if (elect_one()) mma_commit(&m.drain);
        __syncwarp();
        mbar_wait_bounded(&m.drain, 0);
      }
    } else if constexpr (K::I8) {
      if (warp < 12) K::convert(a, m, smem, threadIdx.x - K::kFillWarp * 32);
    } else if (warp <= K::kFillWarp + 1) {
      K::fill(a, m, smem, warp == K::kFillWarp + 1, lane);
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

// ---- host ------------------------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// q as [total_q][Hkv][G][d]; a box is 64 channels of 128 rows (token, head of the group)
bool make_q_tmap(CUtensorMap* map, const void* q, const spg_params& p, int total_q) {
  const auto fn = encoder();
  if (!fn) return false;
  const cuuint64_t d = p.head_dim, G = p.num_q_heads / p.num_kv_heads, Hkv = p.num_kv_heads;
  const cuuint64_t dims[4] = {d, G, Hkv, static_cast<cuuint64_t>(total_q)};
  const cuuint64_t strides[3] = {d * 2, G * d * 2, Hkv * G * d * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(G), 1, static_cast<cuuint32_t>(kTile / G)};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, p.q_dtype == SPG_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// K pool: 64 channels of one page of one kv-head per box
bool make_half_tmap(CUtensorMap* map, const void* pool, const spg_params& p) {
  const auto fn = encoder();
  const long long rows = static_cast<long long>(p.num_phys_pages) * p.num_kv_heads * p.page_size;
  if (!fn || rows > 0x7fffffffLL) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.head_dim), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.head_dim) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(p.page_size)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, p.kv_dtype == SPG_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(pool), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int part_rows(const spg_params& p, int total_q) {
  const long long rows = static_cast<long long>(total_q) * (p.num_q_heads / p.num_kv_heads);
  return static_cast<int>(std::min<long long>(kItemRows, rows));
}

template <typename T, typename TQ, int D>
cudaError_t chunk_typed(const spg_params& p, ChunkArgs& a, const void* q, cudaStream_t st) {
  using K = Kernel<T, TQ, D>;
  if (!make_q_tmap(&a.tmq, q, p, a.total_q)) return cudaErrorNotSupported;
  if constexpr (!K::I8) {
    const long long rows = static_cast<long long>(p.num_phys_pages) * p.num_kv_heads * p.page_size;
    bool whole = false;
    if (!make_half_tmap(&a.tmk, a.k_pool, p) || !make_kv_tmap(&a.tmv, a.v_pool, p.kv_dtype, rows, D, p.page_size, &whole))
      return cudaErrorNotSupported;
    a.v_whole = whole ? 1 : 0;
  }
  const auto kern = k_chunk<T, TQ, D>;
  const size_t smem = 1024 + K::Lay::misc + sizeof(typename K::M);
  const cudaError_t e = ensure_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(std::min(device_sm_count(), kMaxCtas)), dim3(K::kThreads), smem, st, a);
}

}  // namespace

size_t chunk_workspace_bytes(const spg_params& p, int total_q) {
  return round256(workspace_bytes(p)) + round256(sizeof(int32_t) * kMaxCtas) +
         round256(sizeof(float) * 2 * kMaxCtas * part_rows(p, total_q) * (p.head_dim + 2));
}

cudaError_t launch_chunk(const spg_params& p, const ChunkRows& r, const void* k_pool, const void* v_pool,
                         const void* k_scale, const void* v_scale, void* out, float* lse, void* ws,
                         cudaStream_t stream) {
  ChunkArgs a{};
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.k_scale = static_cast<const __half*>(k_scale);
  a.v_scale = static_cast<const __half*>(v_scale);
  a.q_start = r.q_start;
  a.page_table = r.page_table;
  a.seq_lens = r.seq_lens;
  a.out = out;
  a.lse = lse;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.err = reinterpret_cast<int32_t*>(base);
  base += round256(workspace_bytes(p));
  a.counters = reinterpret_cast<int32_t*>(base);
  a.part = reinterpret_cast<float*>(base + round256(sizeof(int32_t) * kMaxCtas));
  a.B = p.batch;
  a.Hkv = p.num_kv_heads;
  a.G = p.num_q_heads / p.num_kv_heads;
  a.S = p.page_size;
  a.MP = p.max_pages_per_seq;
  a.n_phys = p.num_phys_pages;
  a.total_q = r.total_q;
  a.part_rows = part_rows(p, r.total_q);
  a.scale_log2 = (p.softmax_scale > 0.f ? p.softmax_scale : 1.0f / sqrtf(static_cast<float>(p.head_dim))) * kLog2e;
#define SPG_CHUNK(T, TQ) \
  return p.head_dim == 128 ? chunk_typed<T, TQ, 128>(p, a, r.q, stream) : chunk_typed<T, TQ, 64>(p, a, r.q, stream)
  if (p.kv_dtype == SPG_F16) SPG_CHUNK(__half, __half);
  if (p.kv_dtype == SPG_BF16) SPG_CHUNK(__nv_bfloat16, __nv_bfloat16);
  if (p.q_dtype == SPG_F16) SPG_CHUNK(int8_t, __half);
  SPG_CHUNK(int8_t, __nv_bfloat16);
#undef SPG_CHUNK
}

}  // namespace spg
