// Attention over a paged cache of latent vectors (paged_latent_attention), on
// the tcgen05 tensor cores.
//
// Keys and values of all heads are the cached rows themselves: row t of the
// pool is [c_t | k_t], a key in its whole length and a value in its first R
// channels.  So a row (new token, head) of the queries is one of up to 64 that
// share every cached row, and a step of 64 tokens is read once for both
// products, both transposed:
//   S^T = KV Q^T     64 tokens (M) x up to 64 rows (N), K = R + 64
//   P^T = exp2(scale S^T - m)   by the softmax warps
//   O^T += C^T P^T   R / 128 times 128 channels (M) x rows (N), K = 64 tokens
// N follows the rows there are (one token of 16 heads: 16), and 64 rows' O^T
// leaves half of TMEM for S^T.  With the rows as M, 128 of them would fill TMEM
// with their O alone.
//
// A step comes to shared memory as groups of 8 tokens, [group][64-channel
// block][8 rows of 128 bytes], by one TMA copy per page (of any size) and half
// of the channels.  The same bytes are the K-major operand of the first
// product and the MN-major one of the second.  The rotary block is no value:
// once S is done P^T takes its place.  P enters as two 16-bit values
// (spg_set_chunk_parts), the second what the first's rounding left: up to 32
// rows both lie side by side in that block as one operand of twice the columns
// (a product's time is mostly its A operand's, 4 KB of shared memory: 32 cycles
// with 32 columns, 41 with 64), beyond it the second stands in a buffer of its
// own and is a second operand.
//
// The running maximum m of a row is only raised when a (base 2) logit exceeds
// it by more than kTop, and then set kHead below that logit (as in the chunk
// attention): a step only asks whether any logit does, all tokens' threads
// together, and the sums l stay apart per thread until the end.  Logits come
// from TMEM as product fragments, so that all lanes of a warp have some
// although a product of 64 tokens fills only half of TMEM's lanes.
//
// Steps of all items (up to 64 rows of a sequence) are dealt out to the CTAs
// in equal contiguous shares.  Items that cross a border leave (m, l, O) of
// their parts in the workspace with a record of where the others are, and a
// second launch joins them, the work shared out to the CTAs that had the
// parts (joined by the last CTA to arrive, as in the chunk attention, 64 KB to
// 128 KB a part would pass through one SM).  With more than 64 rows per
// sequence neighbouring CTAs take the two halves of 128 rows over the same
// steps, so that the second reads them from L2.
//
// Measured (GB300, R = 512, bf16 or fp16, both launches, inputs from memory):
// one token of 32 heads of 8 sequences of 4K to 64K 60 us, 4.4 TB/s over all
// and 6.2 in the middle (copies alone 6.45); of one sequence at 32K 23 us; of
// 128 heads of 16 sequences at 10K 90 us; 500 tokens of 16 heads over 16K 407
// us, 690 TFLOP/s.  With 64 rows a CTA it is the chain of a step: copy 2200
// cycles, S 2000 (beside the other step's O), softmax 2000, O 1800, and only
// two steps find room in shared memory beside the queries, so that one ends
// every 3900 to 4000 cycles.  The products alone are 2200 of them (a product of
// 64 tokens by 64 rows 25, one of 128 channels 41).  With few rows it is the
// bytes, and about 7 us of start (lengths, plan, pages, first copy) and 5 of the
// second launch.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "spg_deal.cuh"
#include "spg_latent.h"
#include "spg_ring.cuh"
#include "spg_tcgen05.cuh"

namespace spg {
namespace {

constexpr int kRows = 64;   // rows of a CTA: columns of S^T and O^T
constexpr int kStep = 64;   // tokens of a step
constexpr int kRope = 64;
constexpr uint32_t kTmemCols = 512, kTmemS = 256;  // O^T: R / 128 times 64 columns, then two S^T of 64
// m of a row that has seen nothing, the least finite value: any other logit is
// above it by more than kTop (or overflows, which is above it too), and a token
// that is not seen, -inf, is not
constexpr float kUnset = -FLT_MAX;
constexpr float kHead = 7.f, kTop = 15.f;  // the weights of a row are at most 2^15, under fp16's 65504

// sum of floor((a i + b) / m) over 0 <= i < n, by the steps of Euclid's algorithm
__device__ __noinline__ unsigned long long floor_sum(unsigned long long n, unsigned long long m, unsigned long long a, unsigned long long b) {
  unsigned long long sum = 0;
  while (n > 0) {
    if (a >= m) {
      sum += n * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      sum += n * (b / m);
      b %= m;
    }
    const unsigned long long y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const unsigned long long t = m;
    m = a;
    a = t;
  }
  return sum;
}

// ---- the plan: items of 64 rows (128 for a pair of CTAs) -------------------------------
struct LatentItems : ChunkShape {
  static constexpr int kLeast = 2, kExtra = 3, kMostParts = kMaxCtas;
  int H, rows_log2;
  __device__ int items(const ChunkSeq& s) const {
    return static_cast<int>((static_cast<unsigned>(s.n) * H + (1u << rows_log2) - 1) >> rows_log2);
  }
  // one past the last token that item i sees
  __device__ int seen(const ChunkSeq& s, int i) const {
    const unsigned last = (static_cast<unsigned>(i + 1) << rows_log2) - 1;
    return s.pos0 + min(s.n, static_cast<int>(last / H) + 1);
  }
  __device__ int item_steps(const ChunkSeq& s, int i) const { return (seen(s, i) + kStep - 1) / kStep; }
  // Item i but the last sees pos0 + floor((rows (i + 1) - 1) / H) + 1 tokens,
  // floor((rows i + H (pos0 + 64) + rows - 1) / (64 H)) steps; the last ends with the sequence.
  __device__ long long steps(const ChunkSeq& s, int m) const {
    const int n = items(s);
    long long sum = static_cast<long long>(m) * kExtra;
    const int full = min(m, n - 1);
    const unsigned long long rows = 1u << rows_log2;
    if (full > 0)
      sum += floor_sum(full, static_cast<unsigned long long>(kStep) * H, rows,
                       static_cast<unsigned long long>(H) * (s.pos0 + kStep) + rows - 1);
    if (m == n && n > 0) sum += (s.L + kStep - 1) / kStep;
    return sum;
  }
};

// A CTA's part of an item: its rows and steps.  A pair of CTAs takes the two
// halves of the rows; an item of at most 64 rows is taken whole by one of them,
// or, when other pairs have parts of it too, in two halves of the steps.
struct Seg : Part {
  int row0, n_rows, half, k0_of_pair;
  bool split;  // the result is left as a part
};
struct SegIter : PartIter<LatentItems> {
  int pair, rank;
  __device__ SegIter(const LatentItems& shape, const Plan& p, int pair_, int rank_) : PartIter(shape, p, Planned{}), pair(pair_), rank(rank_) {}
  __device__ bool next(Seg& s) {
    while (PartIter::next(s)) {
      s.row0 = s.item << sh.rows_log2;
      s.n_rows = min(1 << sh.rows_log2, s.sq.n * sh.H - s.row0);
      s.split = !s.whole();
      s.half = rank;
      s.k0_of_pair = s.k0;
      if (pair && s.n_rows > kRows) {
        s.row0 += rank * kRows;
        s.n_rows = rank == 0 ? kRows : s.n_rows - kRows;
      } else if (pair && !s.split) {
        if (((s.b ^ s.item) & 1) != rank) continue;
      } else if (pair) {
        const int mid = (s.k0 + s.k1 + 1) / 2;
        if (rank == 0) s.k1 = mid; else s.k0 = mid;  // may leave rank 1 nothing: a part without weight
      }
      return true;
    }
    return false;
  }
};

// What the second launch has to know of a part: CTA c0 + i, i < n, has part i
// of the same rows (by_half: its two halves of the steps, parts 2 i and 2 i + 1).
struct PartRecord {
  int row, n_rows, c0, n, index, by_half, half, pad;  // first row of the chunk; this part's number
};
static_assert(sizeof(PartRecord) == 32, "two 16-byte loads");
constexpr int kSlots = 2 * kMaxCtas;

struct LatentArgs {
  LatentItems sh;
  CUtensorMap tmq, tmkv, tmkv2;  // query rows; the halves of the cached ones
  const uint8_t* pool;
  const int32_t* page_table;
  void* out;
  float* lse;
  int32_t* err;
  float* part;        // [2 * CTAs][part_rows][R]
  float2* part_ml;    // m and l, [64][2 * CTAs]: a row's parts are neighbours
  PartRecord* record;  // [2 * CTAs], n = 0 for a slot without a part
  int S, s_log2, MP, n_phys, part_rows, pair;
  float scale_log2;
};

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ int slot_of(const LatentArgs& a, int c, bool first, int half) {
  return ((2 * c + (first ? 1 : 0)) << a.pair) + half;
}

// A stage holds a step in two halves, the first R / 2 channels of its tokens
// and the others with the rotary block, that come and go by themselves: the
// first's products run while the second is on its way, and the next step's
// first half comes while the second's products run.
template <int R>
struct Layout {
  static constexpr int NA = R / 64 + 1;      // 64-channel blocks of a cached row
  static constexpr int kBlocksA = R / 128, kBlocksB = kBlocksA + 1;  // of its halves
  static constexpr uint32_t kGroupA = kBlocksA * 1024, kGroupB = kBlocksB * 1024, kGroupQ = NA * 1024;  // 8 tokens, 8 query rows
  static constexpr uint32_t kHalfB = kStep / 8 * kGroupA;  // where the second half begins
  static constexpr uint32_t kStage = kHalfB + kStep / 8 * kGroupB;
  static constexpr uint32_t kRopeBlock = kHalfB + kBlocksA * 1024;
  static constexpr int ST = R == 512 ? 2 : 4;
  static constexpr uint32_t q_off = 0, kv_off = kRows / 8 * kGroupQ, lo_off = kv_off + ST * kStage, misc = lo_off + kStep * 128;
};
template <int ST>
struct Misc {
  uint64_t q_full, q_empty, full[ST][2], empty[ST][2], s_full[2], p_full[2], drain[2];
  uint64_t live[ST];  // tokens of a step that are there
  Plan plan;
  uint32_t tmem;
  union {
    int lim[kRows];     // last token a row sees
    float inv[kRows];   // at the end
  };
  float top[4][kRows];  // largest logit of a step, per 16 tokens; at the end the sums
  float factor[kRows];  // what O is rescaled by; at the end the maxima
};

template <typename T, int R, int PARTS>
struct Kernel {
  using Lay = Layout<R>;
  static constexpr int ST = Lay::ST, NA = Lay::NA;
  using M = Misc<ST>;
  // two softmax warpgroups, then the warps that load the steps, issue S, issue O and load Q
  static constexpr int kThreads = 384, kSoftmax = 256, kLoadWarp = 8, kSWarp = 9, kQWarp = 11;

  static __device__ __forceinline__ int columns(const Seg& s) { return (s.n_rows + 15) & ~15; }
  // up to 32 rows: both values of P side by side in one operand, O in two parts
  static __device__ __forceinline__ bool side_by_side(const Seg& s) { return PARTS == 2 && s.n_rows <= kRows / 2; }
  static __device__ __forceinline__ uint32_t idesc(int m, int n, bool a_mn, bool b_mn) {
    return instr_desc<T>(0, 0, b_mn) | (a_mn ? 1u << 15 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
  }
  static __device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

  // ---- S^T, one warp (an elected lane issues) ----------------------------------------------
  static __device__ bool issue_s(const LatentArgs& a, M& m, uint8_t* smem, uint32_t tmem, int rank, int lane) {
    const auto wait = [&](uint64_t* bar, uint32_t phase) { return __all_sync(0xffffffffu, Waiter{a.err}(bar, phase)) != 0; };
    const uint32_t sm = smem_u32(smem), dq = desc_k_major(sm + Lay::q_off), dk = desc_k_major(sm + Lay::kv_off);
    uint32_t c = 0, qc = 0;
    SegIter it(a.sh, m.plan, a.pair, rank);
    Seg s;
    while (uniform(it.next(s))) {
      const int n = uniform(s.k1 - s.k0);
      if (n == 0) continue;
      const uint32_t id = uniform(idesc(64, columns(s), false, false));
      // While a step's products run and its chain goes on, the step that will
      // take its place comes to L2 (earlier it would hold up the copies on
      // their way).  Not for sequences of several items, whose steps others
      // bring there (a prompt piece: 400 us, with it 424).
      const bool bring = uniform(it.n_items == 1);
      const int per = min(a.S, kStep), copies = kStep / per;
      const int32_t* pt = a.page_table + static_cast<size_t>(s.b) * a.MP;
      const auto page_at = [&](int k) {
        const int t = k * kStep + lane * per;
        const bool there = k < s.k1 && lane < copies && t < s.sq.L;
        const int page = pt[there ? t >> a.s_log2 : s.k0 * kStep >> a.s_log2];
        return there && page >= 0 && page < a.n_phys ? page : -1;
      };
      int ahead = bring ? page_at(s.k0 + ST) : -1;
      if (!wait(&m.q_full, qc++)) return false;
      for (int i = 0; i < n; ++i, ++c) {
        const uint32_t stage = c % ST;
        const uint32_t d = tmem + kTmemS + (c & 1) * kRows;
        const auto products = [&](auto which) {
          constexpr int half = decltype(which)::value;
          constexpr int kBlocks = half == 0 ? Lay::kBlocksA : Lay::kBlocksB;
          constexpr uint32_t kGroup = kBlocks * 1024;
          if (!wait(&m.full[stage][half], c / ST)) return false;
          const uint64_t live = m.live[stage];
          if (~live != 0) {
            // tokens that are not there: as keys they are masked, as values they have to be finite
            uint8_t* base = smem + Lay::kv_off + stage * Lay::kStage + half * Lay::kHalfB;
            for (int t = 0; t < kStep; ++t) {
              if ((live >> t) & 1) continue;
              uint8_t* row = base + (t >> 3) * kGroup + (t & 7) * 128;
              for (int x = lane; x < kBlocks * 8; x += 32)
                *reinterpret_cast<uint4*>(row + (x >> 3) * 1024 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();
            __syncwarp();
          }
          // S of two steps ago has been read
          if (half == 0 && c >= 2 && !wait(&m.p_full[c & 1], (c >> 1) - 1)) return false;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t k = dk + ((stage * Lay::kStage + half * Lay::kHalfB) >> 4), q = dq + half * (Lay::kGroupA >> 4);
#pragma unroll
            for (int ks = 0; ks < kBlocks * 4; ++ks) {
              const uint32_t off = ((ks >> 2) * 1024 + (ks & 3) * 32) >> 4;
              mma_ss_groups<kGroup, Lay::kGroupQ>(d, k + off, q + off, id, half > 0 || ks > 0);
            }
            if (half == 1) {
              mma_commit(&m.s_full[c & 1]);
              if (i + 1 == n) mma_commit(&m.q_empty);
            }
          }
          __syncwarp();
          return true;
        };
        if (!products(std::integral_constant<int, 0>{}) || !products(std::integral_constant<int, 1>{})) return false;
        if (bring) {
          if (ahead >= 0) {
            const int t = (s.k0 + i + ST) * kStep + lane * per;
            bulk_prefetch_l2(a.pool + (static_cast<size_t>(ahead) * a.S + (t & (a.S - 1))) * ((R + kRope) * 2),
                             min(per, s.sq.L - t) * ((R + kRope) * 2));
          }
          ahead = page_at(s.k0 + i + 1 + ST);
        }
      }
    }
    return true;
  }

  // ---- O^T, another ----------------------------------------------------------------------------
  static __device__ bool issue_pv(const LatentArgs& a, M& m, uint8_t* smem, uint32_t tmem, int rank) {
    const auto wait = [&](uint64_t* bar, uint32_t phase) { return __all_sync(0xffffffffu, Waiter{a.err}(bar, phase)) != 0; };
    const uint32_t sm = smem_u32(smem), dv = desc_mn_major(sm + Lay::kv_off, 1024);
    const uint32_t dlo = desc_mn_major(sm + Lay::lo_off, 1024);
    uint32_t c = 0;
    SegIter it(a.sh, m.plan, a.pair, rank);
    Seg s;
    while (uniform(it.next(s))) {
      const int n = uniform(s.k1 - s.k0);
      const bool one = uniform(PARTS == 1 || side_by_side(s));  // one operand
      const uint32_t id = uniform(idesc(128, side_by_side(s) ? 2 * columns(s) : columns(s), true, true));
      for (int i = 0; i < n; ++i, ++c) {
        const uint32_t stage = c % ST;
        if (!wait(&m.p_full[c & 1], c >> 1)) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t v = dv + (stage * Lay::kStage >> 4), hi = v + (Lay::kRopeBlock >> 4);
#pragma unroll
          for (int mt = 0; mt < R / 128; ++mt) {
            constexpr int kMtA = R / 256;  // the first half's
#pragma unroll
            for (int ks = 0; ks < kStep / 16; ++ks) {
              const auto product = [&](auto b_groups, uint32_t b, bool acc) {
                constexpr uint32_t SB = decltype(b_groups)::value;
                if (mt < kMtA)
                  mma_ss_groups<Lay::kGroupA, SB>(tmem + mt * kRows, v + ((2 * ks * Lay::kGroupA + mt * 2048) >> 4), b, id, acc);
                else
                  mma_ss_groups<Lay::kGroupB, SB>(tmem + mt * kRows, v + ((Lay::kHalfB + 2 * ks * Lay::kGroupB + (mt - kMtA) * 2048) >> 4), b, id, acc);
              };
              product(std::integral_constant<uint32_t, Lay::kGroupB>{}, hi + (2 * ks * Lay::kGroupB >> 4), i > 0 || ks > 0);
              if (!one) product(std::integral_constant<uint32_t, 1024>{}, dlo + (ks * 2048 >> 4), true);
            }
            if (mt + 1 == kMtA) mma_commit(&m.empty[stage][0]);
          }
          mma_commit(&m.empty[stage][1]);
        }
        __syncwarp();
      }
    }
    return true;
  }

  // ---- query rows, 8 to a copy (one thread) ----------------------------------------------------
  static __device__ void load_q(const LatentArgs& a, M& m, uint8_t* smem, int rank) {
    const Waiter wait{a.err};
    uint32_t c = 0;
    SegIter it(a.sh, m.plan, a.pair, rank);
    Seg s;
    while (it.next(s)) {
      if (s.k0 == s.k1) continue;
      if (c > 0 && !wait(&m.q_empty, c - 1)) break;
      const int groups = columns(s) / 8, row = s.sq.start * a.sh.H + s.row0;
      mbar_arrive_expect_tx(&m.q_full, groups * Lay::kGroupQ);
      for (int g = 0; g < groups; ++g) tma_tile_3d(smem + Lay::q_off + g * Lay::kGroupQ, &a.tmq, 0, row + 8 * g, 0, &m.q_full);
      ++c;
    }
    if (c > 0) wait(&m.q_full, c - 1);  // nothing is in flight when the CTA leaves
  }

  // ---- steps (one warp) --------------------------------------------------------------------------
  static __device__ void load_kv(const LatentArgs& a, M& m, uint8_t* smem, int rank, int lane) {
    const Waiter wait{a.err};
    const int per = min(a.S, kStep), copies = kStep / per;  // tokens of a copy
    PartRing<ST, 2> ring;
    bool ok = true;
    SegIter it(a.sh, m.plan, a.pair, rank);
    Seg s;
    while (ok && it.next(s)) {
      if (s.k0 == s.k1) continue;
      const int32_t* pt = a.page_table + static_cast<size_t>(s.b) * a.MP;
      const auto page_at = [&](int k) {  // of this lane's copy: -1 none, -2 a bad one
        const int t = k * kStep + lane * per;
        const bool there = k < s.k1 && lane < copies && t < s.sq.L;
        const int page = pt[there ? t >> a.s_log2 : s.k0 * kStep >> a.s_log2];
        return there ? (page >= 0 && page < a.n_phys ? page : -2) : -1;
      };
      int next = page_at(s.k0);
      for (int k = s.k0; ok && k < s.k1; ++k) {
        const int page = next, t = k * kStep + lane * per;
        next = page_at(k + 1);
        if (page == -2) record_error(a.err, SPG_DEVERR_PAGE_ID);
        uint64_t live = 0;
        if (page >= 0) {
          const int cnt = min(per, s.sq.L - t);
          live = (cnt == 64 ? ~0ull : (1ull << cnt) - 1) << (lane * per);
        }
        const uint32_t lo = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(live));
        const uint32_t up = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(live >> 32));
        const int n = __popc(__ballot_sync(0xffffffffu, page >= 0));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t group = half == 0 ? Lay::kGroupA : Lay::kGroupB;
          ok = ok && ring.put(
              half,
              [&](uint32_t stage, uint32_t phase) { return __all_sync(0xffffffffu, wait(&m.empty[stage][half], phase)) != 0; },
              [&](uint32_t stage) {
                if (lane == 0) {
                  // nobody reads the last step's any more: the S warp did before that step's S, the softmax warps
                  // before its P, and the first half's products, waited for above, came after both
                  if (half == 0) m.live[stage] = static_cast<uint64_t>(up) << 32 | lo;
                  mbar_arrive_expect_tx(&m.full[stage][half], n * (per / 8) * group);
                }
                __syncwarp();
                if (page >= 0)
                  tma_tile_4d(smem + Lay::kv_off + stage * Lay::kStage + half * Lay::kHalfB + lane * (per / 8) * group,
                              half == 0 ? &a.tmkv : &a.tmkv2, 0, 0, half * Lay::kBlocksA, page * (a.S / 8) + (t & (a.S - 1)) / 8,
                              &m.full[stage][half]);
              });
        }
      }
    }
    // nothing is in flight when the CTA leaves
    ring.drain([&](uint32_t stage, int half, uint32_t phase) { wait(&m.full[stage][half], phase); });
  }

  // ---- softmax ---------------------------------------------------------------------------------------
  // Warp w of a warpgroup has tokens 16 w to 16 w + 15 of a step, the
  // warpgroup half of the rows (in eights): a thread two tokens (lane / 4 and
  // 8 more) over the rows 8 j + 2 (lane % 4) and the next.  The warpgroups
  // have nothing to tell one another before the end.
  static __device__ void softmax(const LatentArgs& a, M& m, uint8_t* smem, uint32_t tmem, int rank, int warp, int lane) {
    bool dead = false;  // after a wait that ran out the others are skipped, and every barrier is still reached
    const auto wait = [&](uint64_t* bar, uint32_t phase) {
      if (!dead && !Waiter{a.err}(bar, phase)) dead = true;
    };
    const int wg = warp >> 2, w4 = warp & 3, own_bar = 2 + wg;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(w4 * 32) << 16);
    const int tok = 16 * w4 + (lane >> 2);
    // this lane's row of the matrices it addresses (lanes 0 to 15): token half, row r
    const int st_r = lane & 7, st_g = 2 * w4 + ((lane >> 3) & 1);
    const uint32_t sm = smem_u32(smem);
    const uint32_t st_hi = sm + Lay::kv_off + Lay::kRopeBlock + st_g * Lay::kGroupB + st_r * 128;
    const uint32_t st_lo = sm + Lay::lo_off + st_g * 1024 + st_r * 128;
    const int cta = static_cast<int>(blockIdx.x) >> a.pair;
    uint32_t c = 0;
    if (threadIdx.x < 2) a.record[slot_of(a, cta, threadIdx.x, rank)].n = 0;
    SegIter it(a.sh, m.plan, a.pair, rank);
    Seg s;
    while (it.next(s)) {
      const int n = s.k1 - s.k0, nb = columns(s) / 16, j0 = wg * nb;  // the warpgroup's eights: j0 to j0 + nb
      const int cl = 8 * j0 + 2 * (lane & 3);
      const bool beside = side_by_side(s);
      const int pos_first = s.sq.pos0 + s.row0 / a.sh.H;
      if (threadIdx.x < kRows)
        m.lim[threadIdx.x] = threadIdx.x < s.n_rows ? s.sq.pos0 + (s.row0 + static_cast<int>(threadIdx.x)) / a.sh.H : -1;
      bar_sync(1, kSoftmax);
      float nm[8], l[8];  // -m and the thread's sums
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        nm[i] = -kUnset;
        l[i] = 0.f;
      }
      for (int i = 0; i < n; ++i, ++c) {
        const uint32_t stage = c % ST;
        wait(&m.s_full[c & 1], c >> 1);
        tc_fence_after();
        uint32_t v[16];
        tmem_ld_frag32(v, lanes + kTmemS + (c & 1) * kRows + 8 * j0);
        const int t0 = (s.k0 + i) * kStep;
        const uint64_t live = m.live[stage];
        tmem_wait_ld();
        if (~live != 0 || t0 + kStep - 1 > pos_first) {
          const bool la = (live >> tok) & 1, lb = (live >> (tok + 8)) & 1;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < nb) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int lim = m.lim[8 * j + cl + e] - t0;
                if (!la || tok > lim) v[4 * j + e] = 0xff800000u;  // -inf
                if (!lb || tok + 8 > lim) v[4 * j + 2 + e] = 0xff800000u;
              }
            }
        }
        // the scaled logits, rounded here once: m is one of them, and what it is
        // taken from has to be the same however large they are
#pragma unroll
        for (int x = 0; x < 16; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * a.scale_log2);
        const auto f = [&](int x) { return __uint_as_float(v[x]); };
        bool over = false;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < nb) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              over |= fmaxf(f(4 * j + e), f(4 * j + 2 + e)) + nm[2 * j + e] > kTop;
          }
        if (bar_any(own_bar, 128, over)) {
          // some row's maximum is raised: the maxima of the warpgroup's rows over the step
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < nb) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x = fmaxf(f(4 * j + e), f(4 * j + 2 + e));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                if (lane < 4) m.top[w4][8 * j + cl + e] = x;
              }
            }
          bar_sync(own_bar, 128);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < nb) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int col = 8 * j + cl + e, x = 2 * j + e;
                const float top = fmaxf(fmaxf(m.top[0][col], m.top[1][col]), fmaxf(m.top[2][col], m.top[3][col]));
                float fac = 1.f;
                if (top + nm[x] > kTop) {
                  fac = ex2(kHead - top - nm[x]);  // 0 for a row that has seen nothing
                  nm[x] = kHead - top;
                  l[x] *= fac;
                }
                if (w4 == 0 && lane < 4) m.factor[col] = fac;
              }
            }
          if (i > 0) {
            bar_sync(own_bar, 128);
            wait(&m.empty[(c - 1) % ST][1], (c - 1) / ST);  // O holds earlier steps, all done
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < R / 128 * nb; ++x) {
              const int col = 8 * (j0 + x % nb);
              const uint32_t at = lanes + x / nb * kRows + col;
#pragma unroll 1
              for (int side = 0; side <= (beside ? 16 * nb : 0); side += 16 * nb) {  // O's second part
                uint32_t o[8];
                tmem_ld8(o, at + side);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 8; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * m.factor[col + y]);
                tmem_st8(at + side, o);
              }
            }
            tmem_wait_st();
          }
        }
        uint32_t hi[8], lo[8];  // of eight j: the first token's pair of rows, the second's
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < nb) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float p0 = ex2(f(4 * j + 2 * r) + nm[2 * j]);
              const float p1 = ex2(f(4 * j + 2 * r + 1) + nm[2 * j + 1]);
              l[2 * j] += p0;
              l[2 * j + 1] += p1;
              hi[2 * j + r] = pack2<T>(p0, p1);
              if constexpr (PARTS == 2) {  // what the rounding left
                const float2 h = unpack2f<T>(hi[2 * j + r]);
                lo[2 * j + r] = pack2<T>(p0 - h.x, p1 - h.y);
              }
            }
          }
        const uint32_t to = st_hi + stage * Lay::kStage;
        if (PARTS == 2 && !beside && c > 0) wait(&m.empty[(c - 1) % ST][1], (c - 1) / ST);  // the second values' buffer is free
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < nb) {
            stmatrix_x2(to + (((j0 + j) ^ st_r) << 4), hi[2 * j], hi[2 * j + 1]);
            if constexpr (PARTS == 2)
              stmatrix_x2(beside ? to + (((2 * nb + j0 + j) ^ st_r) << 4) : st_lo + (((j0 + j) ^ st_r) << 4), lo[2 * j], lo[2 * j + 1]);
          }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.p_full[c & 1]);
      }

      // ---- the segment's end: sums over the tokens' threads, then O^T by channels ----
      bar_sync(own_bar, 128);  // the last raise's top and factor are read
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < nb) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = l[2 * j + e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (lane < 4) {
              m.top[w4][8 * j + cl + e] = x;
              if (w4 == 0) m.factor[8 * j + cl + e] = -nm[2 * j + e];
            }
          }
        }
      bar_sync(1, kSoftmax);
      const int col = threadIdx.x;
      const size_t grow = static_cast<size_t>(s.sq.start) * a.sh.H + s.row0;
      const int slot = slot_of(a, cta, s.k0_of_pair == 0, s.half);
      if (s.split && threadIdx.x == 128) {
        const PartRange pr(m.plan, s);
        const int parts = pr.c1 - pr.c0 + 1, x = cta - pr.c0;
        const bool by_half = a.pair && min(1 << a.sh.rows_log2, s.sq.n * a.sh.H - (s.item << a.sh.rows_log2)) <= kRows;
        a.record[slot] = {static_cast<int>(grow), s.n_rows, pr.c0, by_half ? 2 * parts : parts, by_half ? 2 * x + rank : x, by_half, rank, 0};
      }
      if (col < s.n_rows) {
        const float sum = (m.top[0][col] + m.top[1][col]) + (m.top[2][col] + m.top[3][col]), mx = m.factor[col];
        m.inv[col] = sum == 0.f ? 0.f : 1.f / sum;
        if (s.split) {
          __stcg(a.part_ml + col * kSlots + slot, make_float2(mx, sum));
        } else if (a.lse) {
          a.lse[grow + col] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
        }
      }
      if (n > 0) wait(&m.empty[(c - 1) % ST][1], (c - 1) / ST);
      bar_sync(1, kSoftmax);
      tc_fence_after();
      if (n > 0) {
        // a warpgroup takes every other 128 channels
#pragma unroll 1
        for (int mt = wg; mt < R / 128; mt += 2) {
          const int ch = mt * 128 + w4 * 32 + lane;
#pragma unroll 1
          for (int c0 = 0; c0 < s.n_rows; c0 += 16) {
            uint32_t o[16];
            tmem_ld16(o, lanes + mt * kRows + c0);
            if (beside) {
              uint32_t o2[16];
              tmem_ld16(o2, lanes + mt * kRows + 16 * nb + c0);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) + __uint_as_float(o2[x]));
            }
            tmem_wait_ld();
            if (s.split) {
              float* dst = a.part + (static_cast<size_t>(slot) * a.part_rows + c0) * R + ch;
#pragma unroll
              for (int x = 0; x < 16; ++x)
                if (c0 + x < s.n_rows) __stcg(dst + x * R, __uint_as_float(o[x]));
            } else {
              T* dst = static_cast<T*>(a.out) + (grow + c0) * R + ch;
#pragma unroll
              for (int x = 0; x < 16; ++x)
                if (c0 + x < s.n_rows) {
                  const float inv = m.inv[c0 + x];
                  // inv = 0: a row that saw nothing
                  dst[x * R] = static_cast<T>(inv == 0.f ? 0.f : __uint_as_float(o[x]) * inv);
                }
            }
          }
        }
      }
      tc_fence_before();      // the reads of O come before the next segment's first product
      bar_sync(1, kSoftmax);  // lim, top, factor and inv are read
    }
  }
};

template <typename T, int R, int PARTS>
__global__ void __launch_bounds__(384, 1) k_latent(const __grid_constant__ LatentArgs a) {
  using K = Kernel<T, R, PARTS>;
  using Lay = typename K::Lay;
  using M = typename K::M;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  M& m = *reinterpret_cast<M*>(smem + Lay::misc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = a.pair ? static_cast<int>(blockIdx.x) & 1 : 0;
  if (threadIdx.x == 0) {
    mbar_init(&m.q_full, 1);
    mbar_init(&m.q_empty, 1);
    for (int i = 0; i < K::ST; ++i) {
      for (int half = 0; half < 2; ++half) {
        mbar_init(&m.full[i][half], 1);
        mbar_init(&m.empty[i][half], 1);
      }
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m.s_full[i], 1);
      mbar_init(&m.p_full[i], K::kSoftmax / 32);
      mbar_init(&m.drain[i], 1);
    }
    mbar_fence_init();
  }
  if (warp == K::kSWarp) tmem_alloc(&m.tmem, kTmemCols);
  if (threadIdx.x == 32 * K::kLoadWarp) {
    tma_prefetch_desc(&a.tmkv);
    tma_prefetch_desc(&a.tmkv2);
  }
  if (threadIdx.x == 32 * K::kQWarp) tma_prefetch_desc(&a.tmq);
  {
    // the chain before the first copy is lengths, plan, pages: what they are
    // read from (whatever it will hold) comes to L2 meanwhile
    const long long at = (static_cast<long long>(blockIdx.x) * K::kThreads + threadIdx.x) * 128;
    if (at < static_cast<long long>(a.sh.B) * a.MP * 4) prefetch_l2(reinterpret_cast<const uint8_t*>(a.page_table) + at);
    if (threadIdx.x * 32 <= a.sh.B) prefetch_l2(a.sh.q_start + threadIdx.x * 32);
    if (threadIdx.x * 32 < a.sh.B) prefetch_l2(a.sh.seq_lens + threadIdx.x * 32);
  }
  pdl_wait();
  if (warp == 0) make_plan(a.sh, &m.plan, a.err, lane, static_cast<int>(blockIdx.x) >> a.pair, static_cast<int>(gridDim.x) >> a.pair);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem;

  if (warp < K::kLoadWarp) {
    K::softmax(a, m, smem, tmem, rank, warp, lane);
  } else if (warp == K::kLoadWarp) {
    K::load_kv(a, m, smem, rank, lane);
  } else if (warp == K::kQWarp) {
    if (lane == 0) K::load_q(a, m, smem, rank);
    __syncwarp();
  } else {
    const bool ok = warp == K::kSWarp ? K::issue_s(a, m, smem, tmem, rank, lane) : K::issue_pv(a, m, smem, tmem, rank);
    if (!ok) {  // products in flight end before TMEM goes back
      uint64_t* bar = &m.drain[warp - K::kSWarp];
      if (elect_one()) mma_commit(bar);
      __syncwarp();
      mbar_wait_bounded(bar, 0);
    }
  }
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  if (warp == K::kSWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- the parts of an item joined ------------------------------------------------------------
// CTA (x, y) takes, for each part that CTA x of the first launch left, its
// share of the (row, 128 channels) units of that part's rows; a unit's parts
// are shared out to 1 to 16 warps.
constexpr int kJoinWarps = 16, kJoinY = 4;

template <typename T, int R>
__device__ __forceinline__ void join_part(const LatentArgs& a, const PartRecord& rec, float4 (*acc_s)[32], int warp, int lane) {
  constexpr int kPieces = R / 128, kWeights = kMaxCtas / 32;
  // warps to a unit: at most ten parts a warp with 16, four with fewer
  const int wlog = rec.n > 32 ? 4 : rec.n > 16 ? 3 : rec.n > 8 ? 2 : rec.n > 4 ? 1 : 0;
  const int sub = warp & ((1 << wlog) - 1), per_round = kJoinWarps >> wlog, units = rec.n_rows * kPieces;
  const auto slot = [&](int i) {
    const int c = rec.by_half ? i >> 1 : i;
    return slot_of(a, rec.c0 + c, c == 0, rec.by_half ? i & 1 : rec.half);
  };
  for (int u0 = (rec.index * kJoinY + static_cast<int>(blockIdx.y)) * per_round; u0 < units; u0 += rec.n * kJoinY * per_round) {
    const int u = u0 + (warp >> wlog);
    const bool live = u < units;
    const int row = live ? u / kPieces : 0, ch = (u % kPieces) * 128 + lane * 4;
    // a lane has the weights of every 32nd part
    float w[kWeights], l[kWeights], mm = kUnset, sum = 0.f;
#pragma unroll
    for (int k = 0; k < kWeights; ++k) {
      const float2 ml = 32 * k < rec.n ? __ldcg(a.part_ml + row * kSlots + slot(min(32 * k + lane, rec.n - 1))) : make_float2(0.f, 0.f);
      w[k] = ml.x;
      l[k] = 32 * k + lane < rec.n ? ml.y : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kWeights; ++k)
      if (l[k] != 0.f) mm = fmaxf(mm, w[k]);  // else the part saw nothing, and may not have written its O
    mm = warp_max(mm);
#pragma unroll
    for (int k = 0; k < kWeights; ++k) {
      w[k] = l[k] != 0.f ? ex2(w[k] - mm) : 0.f;
      sum = fmaf(w[k], l[k], sum);
    }
    sum = warp_sum(sum);
    // this warp's parts sub + (q << wlog): all of them on their way at once
    float4 o[2 * kWeights];
#pragma unroll
    for (int q = 0; q < 2 * kWeights; ++q) {
      const int i = sub + (q << wlog);
      o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
      if ((q < 4 || wlog == 4) && i < rec.n)
        o[q] = __ldcg(reinterpret_cast<const float4*>(a.part + (static_cast<size_t>(slot(i)) * a.part_rows + row) * R + ch));
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < 2 * kWeights; ++q) {
      if (q >= 4 && wlog != 4) break;
      const float wq = __shfl_sync(0xffffffffu, q < 2 || wlog == 4 ? w[q >> 1] : w[0], (sub + (q << wlog)) & 31);
      if (wq != 0.f) {
        acc.x = fmaf(wq, o[q].x, acc.x);
        acc.y = fmaf(wq, o[q].y, acc.y);
        acc.z = fmaf(wq, o[q].z, acc.z);
        acc.w = fmaf(wq, o[q].w, acc.w);
      }
    }
    if (wlog > 0) {  // the same in the whole CTA
      acc_s[warp][lane] = acc;
      __syncthreads();
      if (sub == 0)
        for (int q = 1; q < 1 << wlog; ++q) {
          const float4 o = acc_s[warp + q][lane];
          acc.x += o.x;
          acc.y += o.y;
          acc.z += o.z;
          acc.w += o.w;
        }
      __syncthreads();
    }
    if (live && sub == 0) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const size_t grow = static_cast<size_t>(rec.row) + row;
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + grow * R + ch) =
          make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
      if (a.lse && ch == 0) a.lse[grow] = sum == 0.f ? -INFINITY : (mm + log2f(sum)) * kLn2;
    }
  }
}

template <typename T, int R>
__global__ void __launch_bounds__(32 * kJoinWarps, 2) k_latent_join(const __grid_constant__ LatentArgs a) {
  __shared__ float4 acc_s[kJoinWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  // the two slots of a CTA of the first launch
  const PartRecord* rec = a.record + slot_of(a, static_cast<int>(blockIdx.x) >> a.pair, false, blockIdx.x & a.pair);
  const int4 r0[2] = {__ldcg(reinterpret_cast<const int4*>(rec)), __ldcg(reinterpret_cast<const int4*>(rec + (1 << a.pair)))};
  const int4 r1[2] = {__ldcg(reinterpret_cast<const int4*>(rec) + 1), __ldcg(reinterpret_cast<const int4*>(rec + (1 << a.pair)) + 1)};
  pdl_trigger();
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int4 ra = which == 0 ? r0[0] : r0[1], rb = which == 0 ? r1[0] : r1[1];
    if (ra.w > 0) join_part<T, R>(a, {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, 0}, acc_s, warp, lane);
  }
}

// ---- host ------------------------------------------------------------------------------------

int part_rows(const spg_latent_params& p, int total_q) {
  return static_cast<int>(std::max<long long>(1, std::min<long long>(kRows, static_cast<long long>(total_q) * p.num_heads)));
}

template <typename T, int R, int PARTS>
cudaError_t latent_typed(const spg_latent_params& p, LatentArgs& a, const void* q_lat, const void* pool, cudaStream_t st) {
  using K = Kernel<T, R, PARTS>;
  const uint64_t row = 2 * (R + kRope);
  const uint64_t qd[3] = {64, static_cast<uint64_t>(a.sh.total_q) * p.num_heads, K::NA}, qs[2] = {row, 128};
  const uint32_t qb[3] = {64, 8, K::NA};
  const uint64_t kd[4] = {64, 8, K::NA, static_cast<uint64_t>(p.num_phys_pages) * (p.page_size / 8)}, ks[3] = {row, 128, 8 * row};
  uint32_t kb[4] = {64, 8, Layout<R>::kBlocksA, static_cast<uint32_t>(std::min(p.page_size, kStep) / 8)};
  if (!make_tmap16(&a.tmq, p.dtype, q_lat, 3, qd, qs, qb) || !make_tmap16(&a.tmkv, p.dtype, pool, 4, kd, ks, kb))
    return cudaErrorNotSupported;
  kb[2] = Layout<R>::kBlocksB;
  if (!make_tmap16(&a.tmkv2, p.dtype, pool, 4, kd, ks, kb)) return cudaErrorNotSupported;
  const auto kern = k_latent<T, R, PARTS>;
  const size_t smem = 1024 + K::Lay::misc + sizeof(typename K::M);
  static_assert(1024 + K::Lay::misc + sizeof(typename K::M) <= 232448, "shared memory of a CTA");
  cudaError_t e = ensure_smem(kern, smem);
  if (e != cudaSuccess) return e;
  const int ctas = std::min(device_sm_count(), kMaxCtas) >> a.pair;
  e = launch_pdl(kern, dim3(ctas << a.pair), dim3(K::kThreads), smem, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_latent_join<T, R>, dim3(ctas << a.pair, kJoinY), dim3(32 * kJoinWarps), 0, st, a);
}

}  // namespace

namespace {
size_t scratch_bytes(const spg_latent_params& p, int total_q) {
  return sizeof(PartRecord) * kSlots + sizeof(float2) * kSlots * kRows + sizeof(float) * kSlots * part_rows(p, total_q) * p.latent_dim;
}
}  // namespace

size_t latent_workspace_bytes(const spg_latent_params& p, int total_q) { return 256 + scratch_bytes(p, total_q); }

cudaError_t launch_latent_attention(const spg_latent_params& p, const LatentRows& r, const void* q_lat, const void* pool,
                                    void* o_lat, float* lse, int parts, void* ws, size_t ws_bytes, cudaStream_t stream) {
  LatentArgs a{};
  a.sh.q_start = r.q_start;
  a.sh.seq_lens = r.seq_lens;
  a.sh.B = p.batch;
  a.sh.Hkv = 1;
  a.sh.total_q = r.total_q;
  a.sh.max_tokens = p.max_pages_per_seq * p.page_size;
  a.sh.H = p.num_heads;
  // two CTAs over the same steps where sequences have more than 64 rows (on average)
  a.pair = static_cast<long long>(r.total_q) * p.num_heads > static_cast<long long>(kRows) * p.batch || p.num_heads > kRows ? 1 : 0;
  a.sh.rows_log2 = 6 + a.pair;
  a.page_table = r.page_table;
  a.pool = static_cast<const uint8_t*>(pool);
  a.out = o_lat;
  a.lse = lse;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.err = reinterpret_cast<int32_t*>(base);
  // What is left here is not zero, and other entry points keep counters that
  // have to be, where their sizes put them from the workspace's start on: so
  // this stands at its end, behind them where there is room for both.
  a.record = reinterpret_cast<PartRecord*>(base + ((ws_bytes - scratch_bytes(p, r.total_q)) & ~static_cast<size_t>(255)));
  a.part_ml = reinterpret_cast<float2*>(a.record + kSlots);
  a.part = reinterpret_cast<float*>(a.part_ml + kSlots * kRows);
  a.S = p.page_size;
  a.s_log2 = log2_of(p.page_size);
  a.MP = p.max_pages_per_seq;
  a.n_phys = p.num_phys_pages;
  a.part_rows = part_rows(p, r.total_q);
  a.scale_log2 = (p.softmax_scale > 0.f ? p.softmax_scale : 1.0f / sqrtf(static_cast<float>(p.nope_dim + p.rope_dim))) * kLog2e;
#define SPG_LATENT(T)                                                                                             \
  do {                                                                                                            \
    if (parts == 1)                                                                                               \
      return p.latent_dim == 512 ? latent_typed<T, 512, 1>(p, a, q_lat, pool, stream)                             \
                                 : latent_typed<T, 256, 1>(p, a, q_lat, pool, stream);                            \
    return p.latent_dim == 512 ? latent_typed<T, 512, 2>(p, a, q_lat, pool, stream)                               \
                               : latent_typed<T, 256, 2>(p, a, q_lat, pool, stream);                              \
  } while (0)
  if (p.dtype == SPG_F16) SPG_LATENT(__half);
  SPG_LATENT(__nv_bfloat16);
#undef SPG_LATENT
}

}  // namespace spg
