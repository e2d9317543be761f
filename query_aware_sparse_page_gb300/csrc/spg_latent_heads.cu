// The per-head products around latent attention, on the tcgen05 tensor cores:
//   latent_absorb   q_lat[t][h][0:r] = W_uk[h]^T q[t][h][0:dn]
//   latent_project  out[t][h]        = W_uv[h] o_lat[t][h]
//
// Per head a product of [T][K] rows with a [K][N] matrix: K = dn and N = r, or
// K = r and N = dv.  A CTA has 128 rows and one or more tiles of NT columns of
// one head; both operands come by TMA in chunks of 64 of the contraction (rows
// past T as zeros, for which nothing is read), the accumulator stays in TMEM,
// and a tile of many rows leaves by TMA as well, through shared memory.  W_uk's
// rows are the contraction (MN-major), W_uv's are the columns (K-major): the
// matrices stay as the caller has them.
//
// For few rows it is bound by the matrices' bytes (H K N 2), for many by the
// rows': each head's products are too few (2 K flops per element written) to
// bound it.  So with few rows every tile of columns has a CTA of its own, and
// with many one CTA walks all columns of its rows, which it reads once; while
// the tensor cores work on a tile the one before is converted and stored.
//
// Measured (GB300, r = 512, dn = dv = 128, launches back to back, inputs from
// memory): absorbing 16 rows of
// 128 heads 5.1 us, projecting them 6.0 (19 MB each); absorbing 2048 rows of 32
// heads 22.3 us, 3.9 TB/s (every tile of columns by itself, stored from the
// registers: 38).
#include "spg_latent.h"
#include "spg_tcgen05.cuh"

namespace spg {
namespace {

constexpr int kRowsTile = 128, kThreads = 192;
constexpr uint32_t kABytes = kRowsTile * 128;

struct HeadsArgs {
  CUtensorMap tmx, tmw, tmy;
  void* y;
  long long y_row;           // elements from one row of y to the next, and from head to head
  int y_head;
  int n_tiles, walk, w_row;  // tiles of columns, those of one CTA; first row of the head's matrix used
  int few;                   // rows, when they fit one tile: stored from the registers; else 0
  int rows;                  // of a tile, as copied
};

// the tile a copy will bring, into L2
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
               : "memory");
}

// KC: chunks of 64 of the contraction.  ABSORB: the rows' chunks stay for all
// tiles of columns, the matrix's pass through ST buffers; else one tile of
// columns, and both pass through them.  A single tile leaves through the place
// of its operands.  With few rows their chunks have only these (in eights): the
// product's other rows are whatever lies behind, in rows that nobody stores.
template <int KC, int NT, int ST, bool ABSORB>
struct HeadsLayout {
  static constexpr uint32_t kBBytes = NT * 128, kAStages = ABSORB ? KC : ST, kOutBytes = kRowsTile * 128;
  __host__ __device__ static constexpr uint32_t b_off(uint32_t a_bytes) { return kAStages * a_bytes; }
  __host__ __device__ static constexpr uint32_t end(uint32_t a_bytes) { return b_off(a_bytes) + ST * kBBytes; }
  static constexpr uint32_t bytes(uint32_t a_bytes, int walk) { return end(a_bytes) + (walk > 1 ? kOutBytes : 0); }
  static_assert(end(kABytes) >= kOutBytes, "room for 64 columns");
  static_assert(end(1024) >= (kAStages - 1) * 1024 + kABytes, "what a product reads of few rows' chunks");
};

template <typename T, int KC, int NT, int ST, bool ABSORB>
__global__ void __launch_bounds__(kThreads) k_latent_heads(const __grid_constant__ HeadsArgs a) {
  using Lay = HeadsLayout<KC, NT, ST, ABSORB>;
  const uint32_t a_bytes = a.rows * 128, b_off = Lay::b_off(a_bytes), tmem_cols = a.walk > 1 ? 2 * NT : NT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  // (full: the matrix's chunk, with it the rows' while they come; done, free: a tile's accumulator)
  __shared__ uint64_t full[ST], empty[ST], done[2], free_[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_failed;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_row = a.n_tiles / a.walk;
  const int n_first = static_cast<int>(blockIdx.x % per_row) * a.walk, t0 = static_cast<int>(blockIdx.x / per_row) * kRowsTile;
  const int h = blockIdx.y, chunks = a.walk * KC;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&done[i], 1);
      mbar_init(&free_[i], 4);
    }
    s_failed = 0;
    mbar_fence_init();
  }
  if (warp == 5) tmem_alloc(&s_tmem, tmem_cols);
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&a.tmx);
    tma_prefetch_desc(&a.tmw);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_trigger();
  // (every role waits for the launch before ahead of its first bounded wait:
  // however long that launch takes, none of them runs out over it)

  if (warp == 4) {
    if (lane == 0) {
      // The matrices are the caller's weights, but nothing says that the launch
      // before did not write them: until it is done they only come to L2.
      if (a.walk == 1) {
#pragma unroll
        for (int k = 0; k < KC; ++k) {
          if (ABSORB) {
#pragma unroll
            for (int i = 0; i < NT / 64; ++i) tma_prefetch_3d(&a.tmw, n_first * NT + 64 * i, a.w_row + 64 * k, h);
          } else {
            tma_prefetch_3d(&a.tmw, 64 * k, a.w_row + n_first * NT, h);
          }
        }
      }
      pdl_wait();
      for (int c = 0; c < chunks; ++c) {
        const int st = c % ST, k = c % KC, n0 = (n_first + c / KC) * NT;
        if (c >= ST && !mbar_wait_bounded(&empty[st], (c / ST - 1) & 1)) break;
        const bool rows = !ABSORB || c < KC;
        uint8_t* b = smem + b_off + st * Lay::kBBytes;
        mbar_arrive_expect_tx(&full[st], Lay::kBBytes + (rows ? a_bytes : 0));
        if (ABSORB) {
#pragma unroll
          for (int i = 0; i < NT / 64; ++i) tma_tile_3d(b + i * 8192, &a.tmw, n0 + 64 * i, a.w_row + 64 * k, h, &full[st]);
        } else {
          tma_tile_3d(b, &a.tmw, 64 * k, a.w_row + n0, h, &full[st]);
        }
        if (rows) tma_tile_3d(smem + (ABSORB ? k : st) * a_bytes, &a.tmx, 64 * k, h, t0, &full[st]);
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    constexpr uint32_t id = instr_desc<T>(kRowsTile, NT, ABSORB);
    const uint32_t base = smem_u32(smem);
    const auto wait = [&](uint64_t* bar, uint32_t phase) { return __all_sync(0xffffffffu, mbar_wait_bounded(bar, phase & 1)) != 0; };
    pdl_wait();
    for (int c = 0; c < chunks; ++c) {
      const int st = c % ST, k = c % KC, n = c / KC, acc = n & 1;
      // (a tile's accumulator has been read)
      if ((k == 0 && n >= 2 && !wait(&free_[acc], n / 2 - 1)) || !wait(&full[st], c / ST)) {
        // the copies on their way end before the CTA does
        for (int i = c; i < chunks && i < c + ST; ++i) mbar_wait_bounded(&full[i % ST], (i / ST) & 1);
        *static_cast<volatile int*>(&s_failed) = 1;
        if (elect_one()) {  // nobody is left waiting
          mma_commit(&done[0]);
          mma_commit(&done[1]);
        }
        __syncwarp();
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        const uint32_t at = base + (ABSORB ? k : st) * a_bytes, bt = base + b_off + st * Lay::kBBytes;
        const uint32_t da = desc_k_major(at), db = ABSORB ? desc_mn_major(bt, 8192) : desc_k_major(bt);
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_ss(tmem + acc * NT, da + 2 * i, db + i * (ABSORB ? 128 : 2), id, k > 0 || i > 0);
        mma_commit(&empty[st]);
        if (k == KC - 1) mma_commit(&done[acc]);
      }
      __syncwarp();
    }
  } else {
    // ---- a tile's rows, one a thread, to 16 bits and out ----
    uint8_t* out = smem + (a.walk > 1 ? Lay::end(a_bytes) : 0);
    const int r = threadIdx.x;
    pdl_wait();
    for (int n = 0; n < a.walk; ++n) {
      const int acc = n & 1;
      const bool ok = mbar_wait_bounded(&done[acc], (n >> 1) & 1) && *static_cast<volatile int*>(&s_failed) == 0;
      tc_fence_after();
      if (a.few && warp * 32 >= a.few) break;
#pragma unroll
      for (int c = 0; c < NT; c += 32) {
        uint32_t x[32];
        tmem_ld32(x, tmem + (static_cast<uint32_t>(warp * 32) << 16) + acc * NT + c);
        tmem_wait_ld();
        if (!ok) {  // a wait ran out: not a result
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0x7fc00000u;
        }
        if (a.few) {
          if (r >= a.few) continue;
          T* dst = static_cast<T*>(a.y) + r * a.y_row + static_cast<size_t>(h) * a.y_head + n_first * NT + c;
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            const auto f = [&](int e) { return __uint_as_float(x[i + e]); };
            *reinterpret_cast<uint4*>(dst + i) =
                make_uint4(pack2<T>(f(0), f(1)), pack2<T>(f(2), f(3)), pack2<T>(f(4), f(5)), pack2<T>(f(6), f(7)));
          }
          continue;
        }
        // 64 columns at a time through one buffer
        if (c % 64 == 0 && n + c > 0) {
          if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last ones have left
          bar_sync(1, kRowsTile);
        }
        uint8_t* row = out + r * 128;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          const auto f = [&](int e) { return __uint_as_float(x[i + e]); };
          *reinterpret_cast<uint4*>(row + (((((c & 63) + i) >> 3) ^ (r & 7)) << 4)) =
              make_uint4(pack2<T>(f(0), f(1)), pack2<T>(f(2), f(3)), pack2<T>(f(4), f(5)), pack2<T>(f(6), f(7)));
        }
        if (c + 32 == NT) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&free_[acc]);
        }
        if (c % 64 == 32) {
          fence_proxy_async();
          bar_sync(1, kRowsTile);
          if (threadIdx.x == 0) {
            tma_store_3d(&a.tmy, out, (n_first + n) * NT + c - 32, h, t0);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      }
      if (a.few) break;  // a single tile
    }
    if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

template <typename T, int KC, int NT, int ST, bool ABSORB>
cudaError_t heads_typed(const spg_latent_params& p, int total_q, const void* x, int64_t x_stride, const void* w, void* y,
                        cudaStream_t st) {
  using Lay = HeadsLayout<KC, NT, ST, ABSORB>;
  HeadsArgs a{};
  const uint64_t H = p.num_heads, K = 64 * KC, N = ABSORB ? p.latent_dim : p.v_dim, rows = total_q;
  const uint64_t xh = ABSORB ? p.nope_dim + p.rope_dim : p.latent_dim, wr = p.nope_dim + p.v_dim;
  const uint64_t yh = ABSORB ? p.latent_dim + p.rope_dim : p.v_dim;
  a.w_row = ABSORB ? 0 : p.nope_dim;
  a.n_tiles = static_cast<int>(N / NT);
  const long long row_tiles = (static_cast<long long>(total_q) + kRowsTile - 1) / kRowsTile;
  // One CTA for all columns of its rows where every SM has one so, and there
  // are rows enough for reading them once to pay: up to 16 rows the columns stay
  // apart (r 512, 1 and 16 rows; apart against walked: 152 heads 5.0 and 5.4
  // against 7.0 and 7.5 us, 192 heads 7.7 and 8.2 against 7.9 and 8.4, 256 heads
  // 9.0 and 9.5 against 8.6 and 9.2, 1024 heads 26.4 and 28.8 against 30.4 and
  // 32.8; 32 rows of 256 heads 11.9 against 10.0, 128 rows of 192 heads 18.9
  // against 13.3, 640 rows of 32 heads 12.9 against 12.0).
  constexpr int kApart = 16;
  a.walk = ABSORB && total_q > kApart && row_tiles * p.num_heads >= device_sm_count() ? a.n_tiles : 1;
  // rows of one tile straight from the registers, and no more of them copied than there are (16 rows absorbed: 128 heads 5.1
  // against 8.3 us by way of shared memory with a whole tile, 16 heads 3.0 against 3.4; 33 to 128 rows projected: 16 heads
  // 4.4 to 5.7 against 4.7 to 5.5, 128 heads 7.8 to 10.2 against 6.7 to 9.5)
  a.few = a.walk == 1 && total_q <= kRowsTile ? total_q : 0;
  a.rows = a.few ? (a.few + 7) & ~7 : kRowsTile;
  a.y = y;
  a.y_head = static_cast<int>(yh);
  a.y_row = static_cast<long long>(yh * H);
  const uint64_t xd[3] = {K, H, rows}, xs[2] = {2 * xh, 2 * static_cast<uint64_t>(x_stride)};
  const uint64_t wd[3] = {static_cast<uint64_t>(p.latent_dim), wr, H}, ws[2] = {2 * wd[0], 2 * wd[0] * wr};
  const uint64_t yd[3] = {N, H, rows}, ys[2] = {2 * yh, 2 * yh * H};
  const uint32_t xb[3] = {64, 1, static_cast<uint32_t>(a.rows)}, wb[3] = {64, ABSORB ? 64u : static_cast<uint32_t>(NT), 1};
  const uint32_t yb[3] = {64, 1, kRowsTile};
  if (!make_tmap16(&a.tmx, p.dtype, x, 3, xd, xs, xb) || !make_tmap16(&a.tmw, p.dtype, w, 3, wd, ws, wb) ||
      (!a.few && !make_tmap16(&a.tmy, p.dtype, y, 3, yd, ys, yb)))
    return cudaErrorNotSupported;
  const auto kern = k_latent_heads<T, KC, NT, ST, ABSORB>;
  const size_t smem = 1024 + Lay::bytes(a.rows * 128, a.walk);
  const cudaError_t e = ensure_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(static_cast<unsigned>(row_tiles * (a.n_tiles / a.walk)), p.num_heads), dim3(kThreads), smem, st, a);
}

template <typename T, int KC>
cudaError_t project_typed(const spg_latent_params& p, int total_q, const void* x, int64_t x_stride, const void* w, void* y,
                          cudaStream_t st) {
  // few rows: all chunks on their way at once, 32 columns a CTA; else three in flight, 64 columns.  Measured both ways (r 512,
  // dv 128; first this one): 16 heads 1 row 3.7 / 4.0 us, 32 rows 4.1 / 4.4, 33 rows 4.1 / 4.4, 128 rows 4.5 / 5.7; 32 heads
  // 4.3 / 4.8, 4.7 / 5.0, 4.7 / 5.1, 4.9 / 6.3; 128 heads (more CTAs than fit at once) 6.4 / 7.8, 16 rows 6.0 / 8.2, 32 rows
  // 9.0 / 7.6, 33 rows 9.1 / 7.8, 128 rows 18.9 / 10.2: the border is between the two.
  if (total_q <= 32) return heads_typed<T, KC, 32, KC, false>(p, total_q, x, x_stride, w, y, st);
  // 64 columns a CTA while one tile has all rows (twice the CTAs for the matrices' bytes)
  if (p.v_dim == 64 || total_q <= kRowsTile) return heads_typed<T, KC, 64, 3, false>(p, total_q, x, x_stride, w, y, st);
  return heads_typed<T, KC, 128, 3, false>(p, total_q, x, x_stride, w, y, st);
}

template <typename T>
cudaError_t heads(const spg_latent_params& p, bool project, int total_q, const void* x, int64_t x_stride, const void* w, void* y,
                  cudaStream_t st) {
  if (!project)
    return p.nope_dim == 128 ? heads_typed<T, 2, 128, 3, true>(p, total_q, x, x_stride, w, y, st)
                             : heads_typed<T, 1, 128, 3, true>(p, total_q, x, x_stride, w, y, st);
  return p.latent_dim == 512 ? project_typed<T, 8>(p, total_q, x, x_stride, w, y, st)
                             : project_typed<T, 4>(p, total_q, x, x_stride, w, y, st);
}

}  // namespace

cudaError_t launch_latent_heads(const spg_latent_params& p, bool project, int total_q, const void* x, int64_t x_stride,
                                const void* w_kv, void* y, cudaStream_t stream) {
  return p.dtype == SPG_F16 ? heads<__half>(p, project, total_q, x, x_stride, w_kv, y, stream)
                            : heads<__nv_bfloat16>(p, project, total_q, x, x_stride, w_kv, y, stream);
}

}  // namespace spg
