// Attention mass when there are few rows per sequence (decode steps): the
// keys' bytes are all there is to it.
//
// The pages of all (sequence, kv-head) units are dealt out to the CTAs in
// contiguous shares, equal in pages times groups of 8 rows; a page is the
// share's that its first step falls into.  A producer warp streams the K pages by TMA into a
// ring of slots, one lane per slot; four warps take the pages in turn and
// compute S^T = K Q^T for 16 tokens and 8 rows at a time on mma.sync
// m16n8k16 (a tcgen05 tile would be 128 x 128 for 8 rows), int8 codes widened
// in registers.  exp2(scale s - lse) is summed over a token's rows by the
// lanes that hold them and written with the old mass in one pass: a token
// belongs to one page, so nothing is joined.
//
// Measured (GB300): one token of each of 16 sequences over int8 keys of 9K to
// 10K, GQA 32/8: 44 to 49 us for 170 MB, 3.8 TB/s (the tile kernel 94 us; the int8
// decode attention reads its cache at 4.4 TB/s).
#include <algorithm>
#include <cmath>

#include "spg_attn_core.cuh"
#include "spg_deal.cuh"
#include "spg_internal.h"

namespace spg {
namespace {

constexpr int kWarps = 4;            // that sum; one more fills the ring
// four CTAs per SM (eight sequences of bf16 keys to 32K: 76.8 us, with three
// rings of 64 KB 80.9)
constexpr int kCtas = 4;
constexpr int kRingBytes = 48 * 1024;
constexpr size_t kSmBytes = 228 * 1024;  // shared memory of an SM
constexpr int kMaxSlots = 32;        // one per lane of the filling warp

struct PageItems : ChunkShape {
  static constexpr int kLeast = 4;
  int s_log2;
  __device__ int items(const ChunkSeq& s) const { return (s.L + (1 << s_log2) - 1) >> s_log2; }
  // of one page: groups of 8 rows that it meets (without rows, its decay)
  __device__ int page_steps(const ChunkSeq& s) const { return max(1, ((s.n << g_log2) + 7) >> 3); }
  __device__ long long steps(const ChunkSeq& s, int m) const { return static_cast<long long>(m) * page_steps(s); }
};

struct FewArgs {
  PageItems sh;
  CUtensorMap tmk;
  int whole_page;
  const void* q;
  const __half* k_scale;
  const int32_t* page_table;
  const float *lse, *mass_in;
  float* mass_out;
  int32_t* err;
  int Hkv, g_log2, S, MP, n_phys, slots;
  float scale_log2, decay;
};

// A page of the CTA's share: page p of the P of (b, h), its first step `pos`.
struct Cursor {
  const FewArgs& a;
  long long pos, hi;
  int b, h, p, P, each;
  ChunkSeq sq;
  __device__ Cursor(const FewArgs& args, const Plan& plan)
      : a(args), pos(plan.item_first), hi(plan.hi), b(plan.b), h(plan.h), p(plan.item) {
    load();
    if (pos < plan.lo) advance(1);  // the share begins within a page
  }
  __device__ bool live() const { return pos < hi; }
  __device__ void load() {
    int32_t bad = 0;
    sq = a.sh.seq(b, bad);
    P = a.sh.items(sq);
    each = a.sh.page_steps(sq);
  }
  // k pages on, or to the end of all pages (which is the end of the share)
  __device__ void advance(int k) {
    while (k >= P - p) {
      k -= P - p;
      pos += static_cast<long long>(P - p) * each;
      p = 0;
      if (++h == a.Hkv) {
        h = 0;
        if (b + 1 >= a.sh.B) {
          pos = hi;
          return;
        }
        ++b;
        load();
      }
    }
    p += k;
    pos += static_cast<long long>(k) * each;
  }
};

// S^T of 16 tokens and 8 rows; the rows' fragments stay in registers.
template <typename T, typename TQ, int D>
struct Rows8 {
  static constexpr bool I8 = sizeof(T) == 1;
  static constexpr int KS = D / 16;
  uint32_t qb[KS][2];

  // row n = lane / 4 of the eight (null: zeros).  int8: the k index of the
  // product is mapped to four consecutive channels per lane, as the codes lie
  __device__ void load(const TQ* row, int lane) {
    const int t = lane & 3;
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int c = I8 ? 16 * j + 4 * t + 2 * hf : 16 * j + 2 * t + 8 * hf;
        qb[j][hf] = row ? *reinterpret_cast<const uint32_t*>(row + c) : 0u;
      }
  }
  // tokens t0 + g and t0 + g + 8 (g = lane / 4) of a staged page against rows 2t, 2t + 1
  __device__ void qk16(uint32_t kb, int S, int t0, int lane, float (&c)[4]) const {
    const int mi = lane >> 3, r8 = lane & 7, tok = t0 + (mi & 1) * 8 + r8;
    const uint32_t row = kb + tok * 128u;
    float c0[4] = {}, c1[4] = {};
    if constexpr (I8) {
#pragma unroll
      for (int j = 0; j < KS; j += 2) {
        uint32_t r[4];  // tokens 0-7 and 8-15 of 16-channel pieces j and j + 1
        ldmatrix_x4(r, row + (((j + (mi >> 1)) ^ (tok & 7)) << 4));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t f[4];
          AttnMmaI8<1>::i8x4_to_h2(r[2 * i], f[0], f[2]);
          AttnMmaI8<1>::i8x4_to_h2(r[2 * i + 1], f[1], f[3]);
          mma_16816<__half>(i ? c1 : c0, f, qb[j + i][0], qb[j + i][1]);
        }
      }
    } else {
      const uint32_t half = static_cast<uint32_t>(S) * 128u;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const int piece = 2 * j + (mi >> 1);
        uint32_t f[4];
        ldmatrix_x4(f, row + (piece >> 3) * half + (((piece & 7) ^ (tok & 7)) << 4));
        mma_16816<T>(j & 1 ? c1 : c0, f, qb[j][0], qb[j][1]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = c0[e] + c1[e];
  }
};

template <typename T, typename TQ, int D>
__global__ void __launch_bounds__((kWarps + 1) * 32, kCtas) k_mass_few(const __grid_constant__ FewArgs a) {
  constexpr bool I8 = sizeof(T) == 1;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[kMaxSlots], empty[kMaxSlots];
  __shared__ Plan plan;
  const int S = a.S, slots = a.slots, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t page_bytes = static_cast<uint32_t>(S) * D * sizeof(T);
  __half* s_scale = reinterpret_cast<__half*>(smem + slots * page_bytes);  // int8: [slots][S]
  if (threadIdx.x < slots) {
    mbar_init(&full[threadIdx.x], 1);
    mbar_init(&empty[threadIdx.x], 1);
    mbar_fence_init();
  }
  if (threadIdx.x == kWarps * 32) tma_prefetch_desc(&a.tmk);
  pdl_wait();
  if (warp == 0) make_plan(a.sh, &plan, a.err, lane);
  __syncthreads();
  pdl_trigger();
  if (plan.lo == plan.hi) return;

  if (warp == kWarps) {
    // ---- one lane per slot: slot l takes pages l, l + slots, ... of the share
    if (lane < slots) {
      const uint64_t pol = policy_evict_first();
      Cursor c(a, plan);
      c.advance(lane);
      int round = 0;
      for (; c.live(); c.advance(slots), ++round) {
        int page = -1;
        if (c.sq.n > 0) {
          page = a.page_table[static_cast<size_t>(c.b) * a.MP + c.p];
          if (page < 0 || page >= a.n_phys) page = -1;
        }
        if (round > 0 && !mbar_wait_bounded(&empty[lane], (round - 1) & 1)) {
          record_error(a.err, SPG_DEVERR_TIMEOUT);
          break;
        }
        if (page >= 0) {
          const int row = (page * a.Hkv + c.h) * S;
          uint8_t* dst = smem + lane * page_bytes;
          mbar_arrive_expect_tx(&full[lane], page_bytes + (I8 ? 2 * S : 0));
          if (a.whole_page) {
            tma_load_3d(dst, &a.tmk, 0, row, 0, &full[lane], pol);
          } else {
            constexpr int NT = D * static_cast<int>(sizeof(T)) / 128, EPT = 128 / static_cast<int>(sizeof(T));
#pragma unroll
            for (int x = 0; x < NT; ++x) tma_load_2d(dst + x * S * 128, &a.tmk, x * EPT, row, &full[lane], pol);
          }
          if constexpr (I8) bulk_g2s(s_scale + lane * S, a.k_scale + row, 2 * S, &full[lane]);
        } else {
          mbar_arrive(&full[lane]);
        }
      }
      // the last copy of the slot has landed before the CTA leaves
      if (round > 0) mbar_wait_bounded(&full[lane], (round - 1) & 1);
    }
    return;
  }

  // ---- warp w takes pages w, w + 4, ...
  Rows8<T, TQ, D> rows;
  int have_b = -1, have_h = -1, have_g = -1;  // whose rows are in registers
  float l0 = 0.f, l1 = 0.f;                   // lse of rows 2t, 2t + 1 in the log2 domain
  const int g = lane >> 2, t = lane & 3;
  Cursor c(a, plan);
  c.advance(warp);
  for (int j = warp; c.live(); j += kWarps, c.advance(kWarps)) {
    const int slot = j % slots;
    const int n_rows = c.sq.n << a.g_log2, groups = (n_rows + 7) / 8;
    const int tok0 = c.p * S, nv = min(S, c.sq.L - tok0);
    const size_t at = (static_cast<size_t>(c.b) * a.Hkv + c.h) * a.MP * S + tok0;
    bool ok = false;
    if (c.sq.n > 0) {
      const int page = a.page_table[static_cast<size_t>(c.b) * a.MP + c.p];
      ok = page >= 0 && page < a.n_phys;
      if (!ok && lane == 0) record_error(a.err, SPG_DEVERR_PAGE_ID);
    }
    const auto take_rows = [&](int grp) {
      if (c.b == have_b && c.h == have_h && grp == have_g) return;
      have_b = c.b, have_h = c.h, have_g = grp;
      const auto row_of = [&](int r) {
        return ((static_cast<size_t>(c.sq.start) + (r >> a.g_log2)) * a.Hkv << a.g_log2) + (c.h << a.g_log2) +
               (r & ((1 << a.g_log2) - 1));
      };
      const int r = grp * 8 + g;
      rows.load(r < n_rows ? static_cast<const TQ*>(a.q) + row_of(r) * D : nullptr, lane);
      const int r0 = grp * 8 + 2 * t;
      l0 = r0 < n_rows ? a.lse[row_of(r0)] : -INFINITY;
      l1 = r0 + 1 < n_rows ? a.lse[row_of(r0 + 1)] : -INFINITY;
      l0 = l0 == -INFINITY ? INFINITY : l0 * kLog2e;
      l1 = l1 == -INFINITY ? INFINITY : l1 * kLog2e;
    };
    if (ok) take_rows(0);
    if (!mbar_wait_bounded(&full[slot], (j / slots) & 1)) {
      if (lane == 0) record_error(a.err, SPG_DEVERR_TIMEOUT);
      break;
    }
    const uint32_t kb = smem_u32(smem + slot * page_bytes);
    for (int t0 = 0; t0 < nv; t0 += 16) {
      const int mine = t0 + g + 8 * (t & 1);  // lanes t = 0, 1 write this token
      float old = 0.f;
      if (t < 2 && mine < nv && a.mass_in && a.decay > 0.f && tok0 + mine < c.sq.pos0) old = a.mass_in[at + mine] * a.decay;
      float sum[2] = {0.f, 0.f};
      if (ok)
        for (int grp = 0; grp < groups; ++grp) {
          if (groups > 1) take_rows(grp);
          float s[4];
          rows.qk16(kb, S, t0, lane, s);
          float k[2] = {a.scale_log2, a.scale_log2};
          if constexpr (I8) {
            k[0] *= __half2float(s_scale[slot * S + t0 + g]);
            k[1] *= __half2float(s_scale[slot * S + t0 + g + 8]);
          }
          // the first row that sees the token, of those at or past pos0; rows
          // without a log-sum-exp are left out, whatever their products are
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int from = ((tok0 + t0 + g + 8 * e - c.sq.pos0) << a.g_log2) - grp * 8 - 2 * t;
            if (from <= 0 && l0 != INFINITY) sum[e] += exp2f(fmaf(s[2 * e], k[e], -l0));
            if (from <= 1 && l1 != INFINITY) sum[e] += exp2f(fmaf(s[2 * e + 1], k[e], -l1));
          }
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
      }
      if (t < 2 && mine < nv) a.mass_out[at + mine] = old + sum[t];
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
  }
}

template <typename T, typename TQ, int D>
cudaError_t few_typed(const spg_params& p, FewArgs& a, const void* k_pool, cudaStream_t st) {
  const long long rows = static_cast<long long>(p.num_phys_pages) * p.num_kv_heads * p.page_size;
  bool whole = false;
  if (!make_kv_tmap(&a.tmk, k_pool, p.kv_dtype, rows, D, p.page_size, &whole)) return cudaErrorNotSupported;
  a.whole_page = whole ? 1 : 0;
  const size_t page = static_cast<size_t>(p.page_size) * D * sizeof(T);
  // a multiple of the summing warps: each slot has one owner (pages of 8 KB and
  // more leave it one slot, whose next page is on its way only after the sums)
  a.slots = std::max(kWarps, std::min<int>(kMaxSlots, static_cast<int>(kRingBytes / page)) / kWarps * kWarps);
  const size_t smem = 1024 + a.slots * (page + (sizeof(T) == 1 ? 2 * p.page_size : 0));
  const auto kern = k_mass_few<T, TQ, D>;
  const cudaError_t e = ensure_smem(kern, smem);
  if (e != cudaSuccess) return e;
  // CTAs that an SM holds at once (each with 1 KB of the system's and up to 2
  // KB of barriers and plan): the shares are equal, a CTA more would run alone
  const int ctas = std::min<int>(kCtas, static_cast<int>(kSmBytes / (smem + 3 * 1024)));
  return launch_pdl(kern, dim3(ctas * device_sm_count()), dim3((kWarps + 1) * 32), smem, st, a);
}

}  // namespace

cudaError_t launch_mass_few(const spg_params& p, const ChunkRows& r, const void* k_pool, const void* k_scale,
                            const float* lse, const float* mass_in, float* mass_out, float decay, int32_t* err,
                            cudaStream_t stream) {
  const bool i8 = p.kv_dtype == SPG_I8;
  if (i8 && (p.head_dim != 128 || p.q_dtype != SPG_F16)) return cudaErrorNotSupported;
  FewArgs a{};
  a.sh.q_start = r.q_start;
  a.sh.seq_lens = r.seq_lens;
  a.sh.B = p.batch;
  a.sh.Hkv = p.num_kv_heads;
  a.sh.g_log2 = log2_of(p.num_q_heads / p.num_kv_heads);
  a.sh.total_q = r.total_q;
  a.sh.max_tokens = p.max_pages_per_seq * p.page_size;
  a.sh.s_log2 = log2_of(p.page_size);
  a.q = r.q;
  a.k_scale = static_cast<const __half*>(k_scale);
  a.page_table = r.page_table;
  a.lse = lse;
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  a.err = err;
  a.Hkv = p.num_kv_heads;
  a.g_log2 = a.sh.g_log2;
  a.S = p.page_size;
  a.MP = p.max_pages_per_seq;
  a.n_phys = p.num_phys_pages;
  a.scale_log2 = (p.softmax_scale > 0.f ? p.softmax_scale : 1.0f / sqrtf(static_cast<float>(p.head_dim))) * kLog2e;
  a.decay = decay;
  if (i8) return few_typed<int8_t, __half, 128>(p, a, k_pool, stream);
  if (p.kv_dtype == SPG_F16)
    return p.head_dim == 128 ? few_typed<__half, __half, 128>(p, a, k_pool, stream) : few_typed<__half, __half, 64>(p, a, k_pool, stream);
  return p.head_dim == 128 ? few_typed<__nv_bfloat16, __nv_bfloat16, 128>(p, a, k_pool, stream)
                           : few_typed<__nv_bfloat16, __nv_bfloat16, 64>(p, a, k_pool, stream);
}

}  // namespace spg
