// Attention of a ragged chunk of new tokens over the paged cache
// (paged_chunk_attention), on the tcgen05 tensor cores.
//
// An item is up to 256 rows of one (batch, kv-head): the group's query heads
// share their kv-head's keys, so row r is head r % G of new token r / G, at
// cache position pos0 + r / G, and sees the tokens up to there.  A step is
// 128 tokens of an item:
//   S = Q K^T      both from shared memory, S in TMEM
//   P = exp2(scale S - m)  by the softmax warps, written back over S as the
//                  sum of two 16-bit values: 16 logits become 8 columns of
//                  the first and 8 of what its rounding left
//   O += P V       A from TMEM, V from shared memory (its rows are the
//                  contraction: MN-major), a product for each of the two
//                  values, O in TMEM
// with the running maximum m and sum l of the softmax per row.  m is only
// raised when a (base 2) logit exceeds it by more than kTop, and then set
// kHead below that logit: p stays at most 2^kTop, O is rescaled in the rare
// step that raises it, and out = O / l does not depend on m.  kHead keeps the
// weights of a long tail out of fp16's subnormal range.
//
// One CTA per SM, two streams.  With more than 128 rows each has a Q tile of
// 128 rows over the same keys; with fewer they share the rows and take
// alternate steps, and their two (m, l, O) are joined at the end of the item.
// While one stream is in its softmax the tensor cores work for the other.  A
// stream has an issuing warp and two softmax warpgroups: a thread has one row
// and half of the step's tokens, and the two threads of a row agree on its
// maximum through shared memory (one thread per row: 302 against 284 us for
// a ragged batch to 16K, with P as one value).
//
// Measured (GB300): 2048 tokens at the end of 32K, MHA-32 fp16, 16-token
// pages: 1.24 to 1.26 ms.  With P as one value (spg_set_chunk_parts) 0.93 to
// 0.97 ms, 1.10 to 1.14 PFLOP/s of 1.90 measured: products alone take 0.53 ms
// (0.80 with the second part's); the rest is the hand-over between the streams
// (with one value a chain of softmax, issue and products of 3400 cycles per
// step against 2048 of products) and the copies into shared memory beside
// them.  Few rows over long caches: 8 sequences of 4K to 32K with up to 8
// drafted tokens 161 us, 4.5 TB/s (one value: 141).
//
// The steps of all items, in the order (sequence, kv-head, rows), are dealt
// out to the CTAs in equal contiguous shares, whatever the lengths: an item
// that crosses a border leaves (m, l, O) of its parts in the workspace, and
// the part that arrives last joins them in a fixed order.  No CTA waits for
// another.
//
// Four warps fill the K and V rings, 16 bytes per thread and copy, straight
// into the swizzled tiles: pages of 16 tokens are too small for TMA (24 tile
// copies per step kept its unit busy for 3200 cycles, 1.5 times what the
// products take), and tokens that are not there become zeros on the way.
// Larger pages take the same path; TMA was not timed with them.
// int8 codes land in the upper half of their tile's own space and are widened
// in place to exact 16-bit values; the key scales then multiply the logits
// and the value scales the probabilities.  What enters the product is p times
// the value scale, so with int8 m follows the largest logit plus log2 of its
// value scale: the largest weight of a row has the same size whatever the
// scales are, and the sum of p (larger or smaller by what the scales are)
// needs no more than fp32's range.
//
// Roundings: P (int8: times the value scale) to two values of the 16-bit type,
// 2^-16 (bf16) or 2^-22 of it, and the result; everything else is fp32.  The
// caller may ask for one value, and then has the error of 16-bit weights, 1.4
// times that of the result's rounding alone.
#include <algorithm>
#include <cmath>

#include "spg_deal.cuh"
#include "spg_internal.h"
#include "spg_tile_load.cuh"

namespace spg {
namespace {

constexpr int kItemRows = 2 * kTile;  // rows of a Q tile, and tokens of a step: kTile
constexpr uint32_t kTmemCols = 512;  // S0 S1 O0 O1, 128 columns each
constexpr float kLeastVScale = 5.9604644775390625e-8f;  // fp16's smallest but 0, which counts as that one

// ---- the plan -----------------------------------------------------------------------
// An item is 256 rows, a step 128 of the tokens its rows see.
struct RowItems : ChunkShape {
  // joining a part costs about as much as a step
  static constexpr int kLeast = 2;
  // a short item of 256 rows takes 14000 cycles beside its steps of 3400
  static constexpr int kExtra = 4;
  __device__ int log2_tokens() const { return 8 - g_log2; }  // new tokens of an item: 256 / G
  __device__ int items(const ChunkSeq& s) const { return (s.n + (1 << log2_tokens()) - 1) >> log2_tokens(); }
  // one past the last token that item i sees
  __device__ int seen(const ChunkSeq& s, int i) const { return s.pos0 + min((i + 1) << log2_tokens(), s.n); }
  __device__ int item_steps(const ChunkSeq& s, int i) const { return (seen(s, i) + kTile - 1) / kTile; }
  // the first m items: sum of ceil((pos0 + i q) / 128), the last one ends with the sequence
  __device__ long long steps(const ChunkSeq& s, int m) const {
    const int lq = log2_tokens(), q = 1 << lq, full = min(m, s.n >> lq);
    long long sum = 0;
    if (q >= kTile) {
      sum = static_cast<long long>(full) * ((s.pos0 + kTile - 1) / kTile) + static_cast<long long>(q / kTile) * full * (full + 1) / 2;
    } else {
      const int lp = 7 - lq;  // 128 / q items to a step
      for (int r = 1; r <= 1 << lp && r <= full; ++r) {
        const long long cnt = ((full - r) >> lp) + 1;
        sum += cnt * ((s.pos0 + r * q + kTile - 1) / kTile) + cnt * (cnt - 1) / 2;
      }
    }
    if (m > full) sum += (s.L + kTile - 1) / kTile;
    return sum + static_cast<long long>(m) * kExtra;
  }
};
static_assert(kItemRows == 256 && kTile == 128, "the shifts above");
struct Seg : Part {
  int row0, n_rows, last;  // rows of the sequence; the last token any of them sees
  int rot;
  // Step i of the part.  They may come in any order, so they start where a CTA
  // that had walked one item after another from the start of the launch would
  // be by now: CTAs with items of the same kv-head then read the same keys
  // and values at about the same time, once from memory and else from L2
  // (MHA at 32K, where the heads' caches are four times the L2).
  __device__ int at(int i) const {
    const int k = k0 + rot + i;
    return k < k1 ? k : k - (k1 - k0);
  }
};
struct SegIter : PartIter<RowItems> {
  long long lo;
  __device__ SegIter(const RowItems& shape, const Plan& p) : PartIter(shape, p), lo(p.lo) {}
  __device__ bool next(Seg& s) {
    if (!PartIter::next(s)) return false;
    const int by_now = static_cast<int>(s.item_first + s.k0 - lo) % s.nk;
    s.rot = by_now >= s.k0 && by_now < s.k1 ? by_now - s.k0 : 0;
    s.row0 = s.item * kItemRows;
    s.n_rows = min(kItemRows, (s.sq.n << sh.g_log2) - s.row0);
    s.last = sh.seen(s.sq, s.item) - 1;
    return true;
  }
};

struct ChunkArgs {
  RowItems sh;
  CUtensorMap tmq;
  const void *k_pool, *v_pool;
  const __half *k_scale, *v_scale;
  const int32_t* page_table;
  void* out;
  float* lse;
  int32_t *err, *counters;
  float* part;  // [2 * CTAs][D + 2][part_rows]: O by channel, then m and l, so that a warp's rows are neighbours
  int Hkv, S, s_log2, MP, n_phys, part_rows;
  float scale_log2;
};

// ---- shared memory ---------------------------------------------------------------------
template <int D, bool I8>
struct Layout {
  static constexpr int NH = D / 64;  // 64-channel halves
  static constexpr uint32_t kHalf = kTile * 128;
  static constexpr uint32_t kTileBytes = NH * kHalf;
  static constexpr int KST = D == 128 ? 2 : 4, VST = D == 128 ? 2 : 4;
  static constexpr uint32_t q_off = 0, k_off = 2 * kTileBytes, v_off = k_off + KST * kTileBytes;
  static constexpr uint32_t misc = v_off + VST * kTileBytes;
};
template <int KST, int VST, bool I8>
struct Misc {
  uint64_t q_full, q_empty, k_full[KST], k_empty[KST], v_full[VST], v_empty[VST], s_full[2], p_full[2][2], o_full[2], turn[2], drain[2];
  Plan plan;
  uint32_t tmem;
  int last;
  float top[2][2][2][kTile];  // largest logit of a step, per stream and half of the tokens
  float sum[2][2][kTile], max[2][kTile];  // a segment's sums per stream and half, and its m
  alignas(16) float ones[I8 ? kTile : 1];
  // int8, of a step's tokens: scale * key scale, value scale, log2 of its size
  alignas(16) float scales[I8 ? VST : 1][3][I8 ? kTile : 1];
};

// PARTS: 16-bit values in whose sum a weight enters the P V product
template <typename T, typename TQ, int D, int PARTS>
struct Kernel {
  static constexpr bool I8 = sizeof(T) == 1;
  using Lay = Layout<D, I8>;
  static constexpr int KST = Lay::KST, VST = Lay::VST, NH = Lay::NH;
  using M = Misc<KST, VST, I8>;
  // warpgroups 0-3: softmax, two for each stream; 4: loads; 5: the two
  // issuing warps, the warp that loads Q, an idle one
  static constexpr int kThreads = 768, kSoftmax = 512, kLoadWarp = 16, kMmaWarp = 20, kQWarp = 22;
  // registers per thread: 80 at launch, then each warpgroup's share of the
  // same total
  static constexpr int kRegsSoftmax = 96, kRegsLoad = 56, kRegsIssue = 40;
  static_assert(4 * kRegsSoftmax + kRegsLoad + kRegsIssue <= 6 * 80, "the block's registers");
  static constexpr int kLoadThreads = 128;
  // the weights of a row are at most 2^15, under fp16's 65504
  static constexpr float kHead = 7.f, kTop = 15.f;

  // ---- the issuing warps, one per stream: all of a warp waits, one elected lane issues -----
  // One warp's waits and issues for both streams took longer than their
  // products.  The streams' batches (P V of a step, S of the next) go to the
  // tensor cores strictly in turn: left to themselves the two fall into step,
  // both in their softmax while the tensor cores idle, then both in line
  // (1478 against 1257 us for a prompt piece at 32K; with int8 pages, whose
  // widening sets the pace, the turns only cost: 747 against 656 us).
  static __device__ bool issue(const ChunkArgs& a, M& m, uint32_t smem, uint32_t tmem, int t) {
    const auto wait = [&](uint64_t* bar, uint32_t phase) {  // the whole warp goes on, or none of it
      return __all_sync(0xffffffffu, Waiter{a.err}(bar, phase)) != 0;
    };
    constexpr uint32_t idS = instr_desc<TQ>(kTile, kTile, false), idO = instr_desc<TQ>(kTile, D, true);
    constexpr uint32_t kStep = Lay::kTileBytes >> 4;  // descriptors count 16 bytes
    // what the whole warp agrees on, taken from one lane so that it can be kept once per warp
    const auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    tmem = uniform(tmem);
    t = uniform(t);
    const uint32_t tS = tmem + t * 128, tO = tmem + 256 + t * 128;
    const uint32_t dq = desc_k_major(smem + Lay::q_off), dk = desc_k_major(smem + Lay::k_off);
    const uint32_t dv = desc_mn_major(smem + Lay::v_off, Lay::kHalf);
    uint32_t sc = 0, qc = 0, tc = 0;          // rounds of the barriers
    uint32_t ki = 0, vi = 0, kr = 0, vr = 0;  // stage and round of the rings
    const auto next_k = [&] {
      if (++ki == KST) ki = 0, ++kr;
    };
    const auto next_v = [&] {
      if (++vi == VST) vi = 0, ++vr;
    };
    // S of the next key tile; its stage is free (for this stream) once that is done
    const auto S = [&](int qt) {
      const uint32_t q = dq + qt * kStep, k = dk + ki * kStep;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = ((ks >> 2) * Lay::kHalf + (ks & 3) * 32u) >> 4;
        mma_ss(tS, q + off, k + off, idS, ks > 0);
      }
      mma_commit(&m.s_full[t]);
      mma_commit(&m.k_empty[ki]);
    };
    // half the step's tokens, each half's P from a warpgroup of its own
    const auto PV = [&](int half, bool acc) {
      const uint32_t v = dv + vi * kStep;
#pragma unroll
      for (int i = 0; i < kTile / 32; ++i) {
        const int ks = half * (kTile / 32) + i;
        mma_ts(tO, tS + 64 * half + 16 * i, v + ks * (16 * 128 >> 4), idO, acc || ks > 0);
        if (PARTS == 2) mma_ts(tO, tS + 64 * half + 16 * i + 8, v + ks * (16 * 128 >> 4), idO, true);
      }
    };
    SegIter it(a.sh, m.plan);
    Seg s;
    while (uniform(it.next(s))) {
      const int n = uniform(s.k1 - s.k0);
      // two tiles of rows: both streams take every step; one: alternate ones
      const int step = uniform(s.n_rows) > kTile ? 1 : 2, qt = step == 1 ? t : 0;
      if (!wait(&m.q_full, qc++)) return false;
      int j = step == 1 ? 0 : t, jk = 0;  // next step of P V, next key tile
      // stream 0's first S, stream 1's, stream 0's first P V and next S, ...
      // (with one tile of rows the streams' batches differ in number, and the
      // keys' bytes bound them anyway)
      const auto take_turn = [&] {
        if (I8 || step == 2) return true;
        const uint32_t round = tc++;
        return t == 1 ? wait(&m.turn[1], round) : round == 0 || wait(&m.turn[0], round - 1);
      };
      const auto pass_turn = [&] {
        if (!I8 && step == 1 && elect_one()) mbar_arrive(&m.turn[t ^ 1]);
        __syncwarp();
      };
      // the key tile of this stream's step j, past those that are the other stream's alone
      const auto next_s = [&](int j) {
        for (; jk <= j && jk < n; ++jk) {
          if (step == 2 || jk == 0) {
            if (!wait(&m.k_full[ki], kr)) return false;
            fence_proxy_async();
          }
          tc_fence_after();
          if (elect_one()) {
            if (jk == j) S(qt); else mbar_arrive(&m.k_empty[ki]);
          }
          __syncwarp();
          next_k();
        }
        return true;
      };
      if (!take_turn() || !next_s(j)) return false;
      pass_turn();
      for (int jv = 0; jv < n; ++jv) {
        if (!wait(&m.v_full[vi], vr)) return false;
        // (and the next keys, which follow while the turn is held)
        if (step == 1 && jk < n && !wait(&m.k_full[ki], kr)) return false;
        fence_proxy_async();  // the tiles were written with plain copies
        if (jv == j) {
          if (!wait(&m.p_full[t][0], sc) || !take_turn()) return false;
          tc_fence_after();
          if (elect_one()) PV(0, j >= step);
          __syncwarp();
          if (!wait(&m.p_full[t][1], sc++)) return false;
          tc_fence_after();
          if (elect_one()) {
            PV(1, true);
            mma_commit(&m.v_empty[vi]);
          }
          __syncwarp();
          j += step;
          if (!next_s(j)) return false;
          pass_turn();
        } else if (elect_one()) {
          mbar_arrive(&m.v_empty[vi]);
        }
        next_v();
      }
      while (jk < n)  // key tiles behind this stream's last step
        if (!next_s(n)) return false;
      if (elect_one()) {
        mma_commit(&m.q_empty);
        mma_commit(&m.o_full[t]);
      }
      __syncwarp();
    }
    return true;
  }

  // ---- Q tiles (one thread), as soon as the products are done with the last ones ---------
  static __device__ void load_q(const ChunkArgs& a, M& m, uint8_t* smem) {
    const Waiter wait{a.err};
    uint32_t c = 0;
    SegIter it(a.sh, m.plan);
    Seg s;
    for (; it.next(s); ++c) {
      if (c > 0 && !wait(&m.q_empty, c - 1)) return;
      const int tiles = s.n_rows > kTile ? 2 : 1;
      mbar_arrive_expect_tx(&m.q_full, tiles * Lay::kTileBytes);
      for (int t = 0; t < tiles; ++t)
        for (int hf = 0; hf < NH; ++hf)
          tma_tile_4d(smem + Lay::q_off + t * Lay::kTileBytes + hf * Lay::kHalf, &a.tmq, hf * 64, 0, s.h,
                      s.sq.start + ((s.row0 + t * kTile) >> a.sh.g_log2), &m.q_full);
    }
  }

  // ---- loads ----------------------------------------------------------------------------------
  using Tiles = TileLoader<T, TQ, D>;
  static __device__ void load(const ChunkArgs& a, M& m, uint8_t* smem, int tid, int lane) {
    // as in softmax(): after a wait that ran out the others are skipped
    bool dead = false;
    const auto wait = [&](uint64_t* bar, uint32_t phase) {
      if (!dead && !Waiter{a.err}(bar, phase)) dead = true;
    };
    const uint32_t sm = smem_u32(smem);
    const int s_log2 = a.s_log2;
    uint32_t ki = 0, vi = 0, kr = 0, vr = 0;  // stage and round of the rings
    // int8: tiles copied, not yet widened (at most two: a K and a V)
    uint32_t kw = 0, vw = 0;
    int open = 0;
    const auto finish = [&](bool is_v) {
      uint8_t* tile = smem + (is_v ? Lay::v_off + vw * Lay::kTileBytes : Lay::k_off + kw * Lay::kTileBytes);
      Tiles::widen(tile, tid, 3);  // a thread widens what it copied
      fence_proxy_async();
      mbar_arrive(is_v ? &m.v_full[vw] : &m.k_full[kw]);
      uint32_t& w = is_v ? vw : kw;
      if (++w == static_cast<uint32_t>(is_v ? VST : KST)) w = 0;
    };
    SegIter it(a.sh, m.plan);
    Seg s;
    while (it.next(s)) {
      const int32_t* pt = a.page_table + static_cast<size_t>(s.b) * a.MP;
      const int n = s.k1 - s.k0;
      const auto pages = [&](int i) {
        return i < n ? Tiles::page_of(pt, s.at(i) * kTile, s.last + 1, s_log2, a.n_phys, lane) : -1;
      };
      int page = pages(0);
      for (int i = 0; i < n; ++i) {
        const int k = s.at(i), ahead = pages(i + 1);
        if (kr > 0) wait(&m.k_empty[ki], kr - 1);
        Tiles::copy(a.k_pool, a.Hkv, s.h, s_log2, k * kTile, s.sq.L, page, tid, sm + Lay::k_off + ki * Lay::kTileBytes);
        if constexpr (I8) {
          copy_commit();
          if (open == 2) {  // the K of the step before
            copy_wait<2>();
            finish(false);
            --open;
          }
          ++open;
        } else {
          copy_arrive(&m.k_full[ki]);
        }
        if (++ki == KST) ki = 0, ++kr;
        __half sk = __ushort_as_half(0), sv = sk;  // int8: scales of the step's token tid
        if constexpr (I8) {
          const int pg = __shfl_sync(0xffffffffu, page, tid >> s_log2);
          if (pg >= 0 && k * kTile + tid < s.sq.L) {
            const size_t at = ((static_cast<size_t>(pg) * a.Hkv + s.h) << s_log2) + (tid & (a.S - 1));
            sk = a.k_scale[at];
            sv = a.v_scale[at];
          }
        }
        if (vr > 0) wait(&m.v_empty[vi], vr - 1);
        Tiles::copy(a.v_pool, a.Hkv, s.h, s_log2, k * kTile, s.sq.L, page, tid, sm + Lay::v_off + vi * Lay::kTileBytes);
        if constexpr (I8) {
          copy_commit();
          const float v = __half2float(sv);
          m.scales[vi][0][tid] = __half2float(sk) * a.scale_log2;
          m.scales[vi][1][tid] = v;
          m.scales[vi][2][tid] = __log2f(fmaxf(fabsf(v), kLeastVScale));
          if (open == 2) {
            copy_wait<2>();
            finish(true);
            --open;
          }
          ++open;
        } else {
          copy_arrive(&m.v_full[vi]);
        }
        if (++vi == VST) vi = 0, ++vr;
        page = ahead;
      }
    }
    if constexpr (I8) {
      if (open == 2) {
        copy_wait<1>();
        finish(false);
        copy_wait<0>();
        finish(true);
      }
    }
    copy_commit();
    copy_wait<0>();  // nothing is in flight when the CTA leaves
  }

  // ---- softmax ------------------------------------------------------------------------------------
  // A thread has a row, over half of a step's tokens, and of the output half
  // of the channels; m in the log2 domain, the same in both threads.
  struct Row {
    float m, l;
  };

  // Rows that saw nothing have l = 0, out 0 and lse -inf.  A NaN among the
  // logits passes the maximum by and stays in l: out and lse are NaN, from a
  // whole item as from its parts.
  static __device__ __forceinline__ float reciprocal(float l) { return l == 0.f ? 0.f : 1.f / l; }
  static __device__ __forceinline__ float log_sum(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }

  // channel 0 of a row in a slot; the next channel is part_rows further
  static __device__ __forceinline__ float* part_at(const ChunkArgs& a, int slot, int row) {
    return a.part + static_cast<size_t>(slot) * (D + 2) * a.part_rows + row;
  }

  // out and lse of a row from its unnormalised O (element i by o(i)), m and l
  static __device__ __forceinline__ size_t out_row(const ChunkArgs& a, const Seg& s, int r) {
    const int rr = s.row0 + r, lg = a.sh.g_log2;
    return (static_cast<size_t>(s.sq.start + (rr >> lg)) * a.Hkv << lg) + (s.h << lg) + (rr & ((1 << lg) - 1));
  }

  static __device__ void softmax(const ChunkArgs& a, M& m, uint32_t tmem, int warp, int lane) {
    // after a wait that ran out the others are skipped: every thread still
    // reaches every named barrier (the results are not valid then)
    bool dead = false;
    const auto wait = [&](uint64_t* bar, uint32_t phase) {
      if (!dead && !Waiter{a.err}(bar, phase)) dead = true;
    };
    // stream, half of the step's tokens (and of the head's channels), row
    const int t = warp >> 3, h = (warp >> 2) & 1, tid = threadIdx.x;
    const int tile_row = (warp & 3) * 32 + lane;
    // the two warps of the same 32 rows
    const int pair = 4 + 4 * t + (warp & 3);
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    constexpr int kHalf = kTile / 2, kDh = D / 2;
    const uint32_t tS = lanes + t * 128 + h * kHalf, tO = lanes + 256 + t * 128 + h * kDh;
    uint32_t sc = 0, oc = 0, vc = 0;
    SegIter it(a.sh, m.plan);
    Seg s;
    while (it.next(s)) {
      const bool two = s.n_rows > kTile;
      const int r = two ? t * kTile + tile_row : tile_row;  // row of the item
      const int pos = s.sq.pos0 + ((s.row0 + r) >> a.sh.g_log2);
      const int pos_first = s.sq.pos0 + ((s.row0 + (two ? t * kTile : 0)) >> a.sh.g_log2);
      const int32_t* pt = a.page_table + static_cast<size_t>(s.b) * a.MP;
      // does the segment have a bad page at all?
      bool any_bad = false;
      {
        const int p1 = min(s.k1 * kTile - 1, s.last) >> a.s_log2;
#pragma unroll 4
        for (int lp = (s.k0 * kTile >> a.s_log2) + lane; lp <= p1; lp += 32) {
          const int page = pt[lp];
          any_bad |= page < 0 || page >= a.n_phys;
        }
        any_bad = __any_sync(0xffffffffu, any_bad);
        if (any_bad && warp == 0 && lane == 0) record_error(a.err, SPG_DEVERR_PAGE_ID);
      }
      Row row{-INFINITY, 0.f};
      const int step = two ? 1 : 2;
      for (int i = two ? 0 : t; i < s.k1 - s.k0; i += step) {
        const int k = s.at(i);
        uint32_t stage = 0;
        if constexpr (I8) {
          const uint32_t c = vc + i;
          stage = c % VST;
          wait(&m.v_full[stage], c / VST);
        }
        wait(&m.s_full[t], sc);
        ++sc;
        tc_fence_after();
        // 32 logits in registers at a time: the maximum of the upper ones,
        // then of the lower, which stay; the upper are read again when their
        // turn comes.  int8: logits times their key scales, and for the
        // maximum plus log2 of their value scales.
        const float* ks = m.ones;
        const float* lv = m.ones;
        if constexpr (I8) {
          ks = m.scales[stage][0] + h * kHalf;
          lv = m.scales[stage][2] + h * kHalf;
        }
        const int t0 = k * kTile + h * kHalf;
        const bool masked = k * kTile + kTile - 1 > pos_first || any_bad;
        uint32_t x[32];
        float top = -INFINITY;
#pragma unroll
        for (int q = 1; q >= 0; --q) {
          tmem_ld32(x, tS + 32 * q);
          tmem_wait_ld();
          const auto f = [&](int c) { return __uint_as_float(x[c]); };
          if (masked) {
            // the step's last tokens are hidden from some row, or a page is bad (per 16 tokens)
            unsigned bad16 = 0;
            if (any_bad)
              for (int c = 0; c < 32; c += 16) {
                const int tok = t0 + 32 * q + c;
                if (tok <= s.last) {
                  const int page = pt[tok >> a.s_log2];
                  if (page < 0 || page >= a.n_phys) bad16 |= 1u << (c / 16);
                }
              }
            const int lim = pos - t0 - 32 * q;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              if constexpr (I8) x[c] = __float_as_uint(f(c) * ks[32 * q + c]);
              if (c > lim || ((bad16 >> (c / 16)) & 1u)) x[c] = 0xff800000u;  // -inf
            }
            tmem_st32(tS + 32 * q, x);
          }
          float mx[4] = {top, top, top, top};  // chains that do not wait for one another
          if (I8 && !masked) {
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
              const float4 u = *reinterpret_cast<const float4*>(ks + 32 * q + c);
              const float4 w = *reinterpret_cast<const float4*>(ks + 32 * q + c + 4);
              const float4 ul = *reinterpret_cast<const float4*>(lv + 32 * q + c);
              const float4 wl = *reinterpret_cast<const float4*>(lv + 32 * q + c + 4);
              mx[0] = fmaxf(fmaxf(mx[0], fmaf(f(c), u.x, ul.x)), fmaf(f(c + 4), w.x, wl.x));
              mx[1] = fmaxf(fmaxf(mx[1], fmaf(f(c + 1), u.y, ul.y)), fmaf(f(c + 5), w.y, wl.y));
              mx[2] = fmaxf(fmaxf(mx[2], fmaf(f(c + 2), u.z, ul.z)), fmaf(f(c + 6), w.z, wl.z));
              mx[3] = fmaxf(fmaxf(mx[3], fmaf(f(c + 3), u.w, ul.w)), fmaf(f(c + 7), w.w, wl.w));
            }
          } else if (I8) {
#pragma unroll
            for (int c = 0; c < 32; c += 4)
#pragma unroll
              for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], f(c + i) + lv[32 * q + c + i]);
          } else {
#pragma unroll
            for (int c = 0; c < 32; c += 8)
#pragma unroll
              for (int i = 0; i < 4; ++i) mx[i] = fmaxf(fmaxf(mx[i], f(c + i)), f(c + 4 + i));
          }
          top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        }
        if (I8 && masked) ks = m.ones;  // the logits went back with their scales
        // the row's maximum over both halves (two buffers: the other warp may
        // be a step ahead)
        float* mine = &m.top[sc & 1][t][h][tile_row];
        *mine = top;
        bar_sync(pair, 64);
        top = fmaxf(top, m.top[sc & 1][t][h ^ 1][tile_row]);
        if constexpr (!I8) top *= a.scale_log2;
        const bool raise = top > row.m + kTop;  // -inf + kTop = -inf: the first finite logit
        if (__any_sync(0xffffffffu, raise)) {     // the same in both warps
          const float mn = raise ? top - kHead : row.m;
          const float factor = row.m == -INFINITY ? (raise ? 0.f : 1.f) : ex2(row.m - mn);
          row.m = mn;
          row.l *= factor;
          if (i >= step) {  // O holds earlier steps (all done: S of this step was issued after them)
            uint32_t o[16];
#pragma unroll 1
            for (int c = 0; c < kDh; c += 16) {
              tmem_ld16(o, tO + c);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
              tmem_st16(tO + c, o);
            }
            tmem_wait_st();
            tc_fence_before();
            bar_sync(pair, 64);  // the first half's products touch the other's channels too
          }
        }
        const float mm = row.m == -INFINITY ? 0.f : row.m;
        const uint64_t nm = f32x2(-mm, -mm), sc2 = f32x2(a.scale_log2, a.scale_log2);
        uint64_t l0 = f32x2(0.f, 0.f), l1 = l0;
        if (masked) tmem_wait_st();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          // 16 logits at a time: the parts of their P go over them, the upper
          // 32 are read again meanwhile
          uint32_t w[8 * PARTS];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e0 = 16 * (q & 1) + 2 * i;
            const uint64_t z = f32x2(__uint_as_float(x[e0]), __uint_as_float(x[e0 + 1]));
            uint64_t mul = sc2;
            if constexpr (I8) mul = *reinterpret_cast<const uint64_t*>(ks + 16 * q + 2 * i);
            const float2 e = unpack_f32x2(fma_f32x2(z, mul, nm));
            float2 p = make_float2(ex2(e.x), ex2(e.y));
            if (i & 1) l1 = add_f32x2(l1, f32x2(p.x, p.y)); else l0 = add_f32x2(l0, f32x2(p.x, p.y));
            if constexpr (I8) {
              const float2 vs = *reinterpret_cast<const float2*>(&m.scales[stage][1][h * kHalf + 16 * q + 2 * i]);
              p.x *= vs.x;
              p.y *= vs.y;
            }
            w[i] = pack2<TQ>(p.x, p.y);
            if constexpr (PARTS == 2) {  // what the rounding left
              const float2 hi = unpack2f<TQ>(w[i]);
              w[8 + i] = pack2<TQ>(p.x - hi.x, p.y - hi.y);
            }
          }
          if (q == 1 || q == 2) tmem_wait_ld();
          if constexpr (PARTS == 2) tmem_st16(tS + 16 * q, w); else tmem_st8(tS + 16 * q, w);
          if (q < 2) tmem_ld16(x + 16 * q, tS + 32 + 16 * q);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&m.p_full[t][h]);
        const float2 s0 = unpack_f32x2(l0), s1 = unpack_f32x2(l1);
        row.l += (s0.x + s0.y) + (s1.x + s1.y);
      }
      vc += s.k1 - s.k0;

      // ---- the segment's end ----
      const bool whole = s.whole();
      m.sum[t][h][tile_row] = row.l;
      if (h == 0) m.max[t][tile_row] = row.m;
      wait(&m.o_full[t], oc);
      float f0 = 1.f, f1 = 0.f;
      if (two) {
        bar_sync(pair, 64);
        row.l += m.sum[t][h ^ 1][tile_row];
        bar_sync(pair, 64);  // read before the next segment's are written
      } else {  // the rows' two streams
        if (t == 0) wait(&m.o_full[1], oc);
        bar_sync(1, kSoftmax);
        if (t == 0) {
          const float m1 = m.max[1][tile_row], l1 = m.sum[1][0][tile_row] + m.sum[1][1][tile_row];
          const float l0 = m.sum[0][0][tile_row] + m.sum[0][1][tile_row];
          const float mm = fmaxf(row.m, m1);
          f0 = row.m == -INFINITY ? 0.f : ex2(row.m - mm);
          f1 = m1 == -INFINITY ? 0.f : ex2(m1 - mm);
          row.l = l0 * f0 + l1 * f1;
          row.m = mm;
        }
      }
      ++oc;
      tc_fence_after();
      if (two || t == 0) {
        const bool live = r < s.n_rows;
        const bool both = !two && s.k1 - s.k0 > 1;  // stream 1 has had a step
        const float inv = reciprocal(row.l);
        if (whole) {
          f0 *= inv;
          f1 *= inv;
        }
        const size_t orow = live ? out_row(a, s, r) : 0;
        float* part = part_at(a, own_slot(s), live ? r : 0);
#pragma unroll 1
        for (int c = 0; c < kDh; c += 16) {
          uint32_t o[16];
          tmem_ld16(o, tO + c);
          tmem_wait_ld();
          // f0 = 0 stands for rows that saw nothing: their O may not be trusted to be finite
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(f0 == 0.f ? 0.f : __uint_as_float(o[i]) * f0);
          if (both) {
            uint32_t o1[16];
            tmem_ld16(o1, tO + 128 + c);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (f1 != 0.f) o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), f1, __uint_as_float(o[i])));
          }
          if (live && whole) {
            TQ* dst = static_cast<TQ*>(a.out) + orow * D + h * kDh + c;
#pragma unroll
            for (int i = 0; i < 16; i += 8)
              *reinterpret_cast<uint4*>(dst + i) = make_uint4(pack2<TQ>(__uint_as_float(o[i]), __uint_as_float(o[i + 1])),
                                                             pack2<TQ>(__uint_as_float(o[i + 2]), __uint_as_float(o[i + 3])),
                                                             pack2<TQ>(__uint_as_float(o[i + 4]), __uint_as_float(o[i + 5])),
                                                             pack2<TQ>(__uint_as_float(o[i + 6]), __uint_as_float(o[i + 7])));
          } else if (live) {
#pragma unroll
            for (int i = 0; i < 16; ++i) __stcg(part + (h * kDh + c + i) * a.part_rows, __uint_as_float(o[i]));
          }
        }
        if (live && h == 0) {
          if (whole) {
            if (a.lse) a.lse[orow] = log_sum(row.m, row.l);
          } else {
            __stcg(part + D * a.part_rows, row.m);
            __stcg(part + (D + 1) * a.part_rows, row.l);
          }
        }
      }
      tc_fence_before();  // the loads of O come before the next segment's first product
      if (!two) bar_sync(2, kSoftmax);
      if (!whole) join(a, m, s, tid);
    }
  }

  // Counts a part of an item in; the last to arrive joins them all.
  static __device__ void join(const ChunkArgs& a, M& m, const Seg& s, int tid) {
    const PartRange pr(m.plan, s);
    const int c0 = pr.c0, c1 = pr.c1;
    __threadfence();
    bar_sync(1, kSoftmax);
    if (tid == 0) m.last = atomicAdd(&a.counters[c0], 1) == c1 - c0;
    bar_sync(2, kSoftmax);
    if (!m.last) return;
    __threadfence();
    // two threads per row with half the channels each, or four with a quarter
    const bool two = s.n_rows > kTile;
    const int r = tid % (two ? kItemRows : kTile), share = two ? D / 2 : D / 4;
    const int d0 = tid / (two ? kItemRows : kTile) * share, d1 = d0 + share;
    if (r < s.n_rows) {
      const auto at = [&](int c) { return part_at(a, pr.slot(c), r); };
      float mm = -INFINITY, l = 0.f;
#pragma unroll 2
      for (int c = c0; c <= c1; ++c) mm = fmaxf(mm, __ldcg(at(c) + D * a.part_rows));
      if (mm == -INFINITY) mm = 0.f;  // every part's weight is 0
#pragma unroll 2
      for (int c = c0; c <= c1; ++c)
        l = fmaf(__ldcg(at(c) + (D + 1) * a.part_rows), ex2(__ldcg(at(c) + D * a.part_rows) - mm), l);
      const float inv = reciprocal(l);
      const size_t orow = out_row(a, s, r);
      TQ* dst = static_cast<TQ*>(a.out) + orow * D;
      for (int d = d0; d < d1; d += 16) {
        float o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = 0.f;
#pragma unroll 2
        for (int c = c0; c <= c1; ++c) {
          const float* p = at(c);
          const float f = ex2(__ldcg(p + D * a.part_rows) - mm);
          p += d * a.part_rows;
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = fmaf(__ldcg(p + i * a.part_rows), f, o[i]);
        }
#pragma unroll
        for (int i = 0; i < 16; i += 8)
          *reinterpret_cast<uint4*>(dst + d + i) =
              make_uint4(pack2<TQ>(o[i] * inv, o[i + 1] * inv), pack2<TQ>(o[i + 2] * inv, o[i + 3] * inv),
                         pack2<TQ>(o[i + 4] * inv, o[i + 5] * inv), pack2<TQ>(o[i + 6] * inv, o[i + 7] * inv));
      }
      if (d0 == 0 && a.lse) a.lse[orow] = log_sum(mm, l);
    }
    if (tid == 0) a.counters[c0] = 0;  // ready for the next call
  }
};

template <typename T, typename TQ, int D, int PARTS>
__global__ void __launch_bounds__(768, 1) k_chunk(const __grid_constant__ ChunkArgs a) {
  using K = Kernel<T, TQ, D, PARTS>;
  using Lay = typename K::Lay;
  using M = typename K::M;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  M& m = *reinterpret_cast<M*>(smem + Lay::misc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&m.q_full, 1);
    mbar_init(&m.q_empty, 2);
    for (int i = 0; i < K::KST; ++i) {
      mbar_init(&m.k_full[i], K::kLoadThreads);
      mbar_init(&m.k_empty[i], 2);
    }
    for (int i = 0; i < K::VST; ++i) {
      mbar_init(&m.v_full[i], K::kLoadThreads);
      mbar_init(&m.v_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m.s_full[i], 1);
      mbar_init(&m.p_full[i][0], 128);
      mbar_init(&m.p_full[i][1], 128);
      mbar_init(&m.o_full[i], 1);
      mbar_init(&m.turn[i], 1);
      mbar_init(&m.drain[i], 1);
    }
    mbar_fence_init();
  }
  if (K::I8 && threadIdx.x < kTile) m.ones[threadIdx.x] = 1.f;
  if (warp == K::kMmaWarp) tmem_alloc(&m.tmem, kTmemCols);
  pdl_wait();
  if (warp == 0) make_plan(a.sh, &m.plan, a.err, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem;

  if (warp < K::kLoadWarp) {
    regs_up<K::kRegsSoftmax>();
    K::softmax(a, m, tmem, warp, lane);
  } else {
    if (warp < K::kMmaWarp) {
      regs_down<K::kRegsLoad>();
      K::load(a, m, smem, threadIdx.x - K::kLoadWarp * 32, lane);
    } else {
      regs_down<K::kRegsIssue>();
      if (warp == K::kQWarp) {
        if (lane == 0) K::load_q(a, m, smem);
        __syncwarp();
      } else if (warp < K::kQWarp) {
        const int t = warp - K::kMmaWarp;
        if (!K::issue(a, m, smem_u32(smem), tmem, t)) {
          // products in flight end before TMEM goes back
          if (elect_one()) mma_commit(&m.drain[t]);
          __syncwarp();
          mbar_wait_bounded(&m.drain[t], 0);
        }
      }
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

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int part_rows(const spg_params& p, int total_q) {
  const long long rows = static_cast<long long>(total_q) * (p.num_q_heads / p.num_kv_heads);
  return static_cast<int>(std::min<long long>(kItemRows, rows));
}

template <typename T, typename TQ, int D, int PARTS>
cudaError_t chunk_typed(const spg_params& p, ChunkArgs& a, const void* q, cudaStream_t st) {
  using K = Kernel<T, TQ, D, PARTS>;
  if (!make_q_tmap(&a.tmq, q, p, a.sh.total_q, kTile)) return cudaErrorNotSupported;
  const auto kern = k_chunk<T, TQ, D, PARTS>;
  const size_t smem = 1024 + K::Lay::misc + sizeof(typename K::M);
  const cudaError_t e = ensure_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(std::min(device_sm_count(), kMaxCtas)), dim3(K::kThreads), smem, st, a);
}

}  // namespace

size_t chunk_workspace_bytes(const spg_params& p, int total_q) {
  return round256(workspace_bytes(p)) +
         round256(sizeof(float) * 2 * kMaxCtas * part_rows(p, total_q) * (p.head_dim + 2));
}

cudaError_t launch_chunk(const spg_params& p, const ChunkRows& r, const void* k_pool, const void* v_pool,
                         const void* k_scale, const void* v_scale, void* out, float* lse, int parts,
                         void* ws, cudaStream_t stream) {
  ChunkArgs a{};
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.k_scale = static_cast<const __half*>(k_scale);
  a.v_scale = static_cast<const __half*>(v_scale);
  a.sh.q_start = r.q_start;
  a.sh.seq_lens = r.seq_lens;
  a.sh.B = p.batch;
  a.sh.Hkv = p.num_kv_heads;
  a.sh.g_log2 = log2_of(p.num_q_heads / p.num_kv_heads);
  a.sh.total_q = r.total_q;
  a.sh.max_tokens = p.max_pages_per_seq * p.page_size;
  a.page_table = r.page_table;
  a.out = out;
  a.lse = lse;
  const Workspace w = carve_workspace(p, ws);
  a.err = w.err;
  a.counters = w.part_counters;
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + round256(workspace_bytes(p)));
  a.Hkv = p.num_kv_heads;
  a.S = p.page_size;
  a.s_log2 = log2_of(p.page_size);
  a.MP = p.max_pages_per_seq;
  a.n_phys = p.num_phys_pages;
  a.part_rows = part_rows(p, r.total_q);
  a.scale_log2 = (p.softmax_scale > 0.f ? p.softmax_scale : 1.0f / sqrtf(static_cast<float>(p.head_dim))) * kLog2e;
#define SPG_CHUNK(T, TQ)                                                     \
  do {                                                                       \
    if (parts == 1)                                                          \
      return p.head_dim == 128 ? chunk_typed<T, TQ, 128, 1>(p, a, r.q, stream) \
                               : chunk_typed<T, TQ, 64, 1>(p, a, r.q, stream); \
    return p.head_dim == 128 ? chunk_typed<T, TQ, 128, 2>(p, a, r.q, stream) \
                             : chunk_typed<T, TQ, 64, 2>(p, a, r.q, stream); \
  } while (0)
  if (p.kv_dtype == SPG_F16) SPG_CHUNK(__half, __half);
  if (p.kv_dtype == SPG_BF16) SPG_CHUNK(__nv_bfloat16, __nv_bfloat16);
  if (p.q_dtype == SPG_F16) SPG_CHUNK(int8_t, __half);
  SPG_CHUNK(int8_t, __nv_bfloat16);
#undef SPG_CHUNK
}

}  // namespace spg
