// The per-head products around latent attention, on the tcgen05 tensor cores:
//   latent_absorb   q_lat[t][h][0:r] = W_uk[h]^T q[t][h][0:dn]
//   latent_project  out[t][h]        = W_uv[h] o_lat[t][h]
//
// Per head a product of [T][K] rows with a [K][N] matrix: K = dn and N = r, or
// K = r and N = dv.  A CTA has 128 rows and NT columns of one head; both
// operands come by TMA in chunks of 64 of the contraction (rows past T as
// zeros, for which nothing is read), the accumulator stays in TMEM.  W_uk's
// rows are the contraction (MN-major), W_uv's are the columns (K-major): the
// matrices stay as the caller has them.
//
// For few rows it is bound by the matrices' bytes (H K N 2), for many by the
// rows': each head's products are too few (2 K flops per element read) to
// bound it.
#include "spg_latent.h"
#include "spg_tcgen05.cuh"

namespace spg {
namespace {

constexpr int kRowsTile = 128, kThreads = 192;
constexpr uint32_t kABytes = kRowsTile * 128;

struct HeadsArgs {
  CUtensorMap tmx, tmw;
  void* y;
  long long y_row;  // elements from one row of y to the next
  int total_q, n_tiles, w_row, y_head;  // first row of the head's matrix used; elements from head to head of y
};

__device__ __forceinline__ void tma_tile_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// KC: chunks of 64 of the contraction; ST: how many of them are in flight
template <typename T, int KC, int NT, int ST, bool ABSORB>
__global__ void __launch_bounds__(kThreads) k_latent_heads(const __grid_constant__ HeadsArgs a) {
  constexpr uint32_t kBBytes = NT * 128, kStage = kABytes + kBBytes;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[ST], empty[ST], done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_failed;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = static_cast<int>(blockIdx.x % a.n_tiles) * NT, t0 = static_cast<int>(blockIdx.x / a.n_tiles) * kRowsTile;
  const int h = blockIdx.y;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    s_failed = 0;
    mbar_fence_init();
  }
  if (warp == 5) tmem_alloc(&s_tmem, NT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_trigger();

  if (warp == 4) {
    if (lane == 0) {
      const auto load_w = [&](int k) {
        uint8_t* b = smem + (k % ST) * kStage + kABytes;
        if (ABSORB) {
#pragma unroll
          for (int i = 0; i < NT / 64; ++i)
            tma_tile_3d(b + i * 8192, &a.tmw, n0 + 64 * i, a.w_row + 64 * k, h, &full[k % ST]);
        } else {
          tma_tile_3d(b, &a.tmw, 64 * k, a.w_row + n0, h, &full[k % ST]);
        }
      };
      // the matrices are the caller's weights, but nothing says that the launch before did not write them
      pdl_wait();
      for (int k = 0; k < KC; ++k) {
        if (k >= ST && !mbar_wait_bounded(&empty[k % ST], (k / ST - 1) & 1)) break;
        mbar_arrive_expect_tx(&full[k % ST], kStage);
        load_w(k);
        tma_tile_3d(smem + (k % ST) * kStage, &a.tmx, 64 * k, h, t0, &full[k % ST]);
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    constexpr uint32_t id = instr_desc<T>(kRowsTile, NT, ABSORB);
    const uint32_t base = smem_u32(smem);
    for (int k = 0; k < KC; ++k) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[k % ST], (k / ST) & 1))) {
        // the copies on their way end before the CTA does
        for (int i = k; i < KC && i < k + ST; ++i) mbar_wait_bounded(&full[i % ST], (i / ST) & 1);
        *static_cast<volatile int*>(&s_failed) = 1;
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        const uint32_t at = base + (k % ST) * kStage, bt = at + kABytes;
        const uint32_t da = desc_k_major(at), db = ABSORB ? desc_mn_major(bt, 8192) : desc_k_major(bt);
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_ss(tmem, da + 2 * i, db + i * (ABSORB ? 128 : 2), id, k > 0 || i > 0);
        if (KC > ST) mma_commit(&empty[k % ST]);
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit(&done);
    __syncwarp();
  }
  const bool ok = mbar_wait_bounded(&done, 0) && *static_cast<volatile int*>(&s_failed) == 0;
  tc_fence_after();
  const int t = t0 + threadIdx.x;
  if (warp < 4 && t0 + warp * 32 < a.total_q) {
    T* dst = static_cast<T*>(a.y) + static_cast<size_t>(t) * a.y_row + static_cast<size_t>(h) * a.y_head + n0;
#pragma unroll
    for (int c = 0; c < NT; c += 32) {
      uint32_t x[32];
      tmem_ld32(x, tmem + (static_cast<uint32_t>(warp * 32) << 16) + c);
      tmem_wait_ld();
      if (!ok) {  // a wait ran out: not a result
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = 0x7fc00000u;
      }
      if (t < a.total_q) {
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          const auto f = [&](int e) { return __uint_as_float(x[i + e]); };
          *reinterpret_cast<uint4*>(dst + c + i) =
              make_uint4(pack2<T>(f(0), f(1)), pack2<T>(f(2), f(3)), pack2<T>(f(4), f(5)), pack2<T>(f(6), f(7)));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, NT);
  }
}

template <typename T, int KC, int NT, bool ABSORB>
cudaError_t heads_typed(const spg_latent_params& p, HeadsArgs& a, const void* x, int64_t x_stride, const void* w,
                        cudaStream_t st) {
  constexpr int ST = KC < 3 ? KC : 3;
  const uint64_t H = p.num_heads, K = 64 * KC, N = ABSORB ? p.latent_dim : p.v_dim;
  const uint64_t xh = ABSORB ? p.nope_dim + p.rope_dim : p.latent_dim, wr = p.nope_dim + p.v_dim;
  const uint64_t xd[3] = {K, H, static_cast<uint64_t>(a.total_q)}, xs[2] = {2 * xh, 2 * static_cast<uint64_t>(x_stride)};
  const uint32_t xb[3] = {64, 1, kRowsTile};
  const uint64_t wd[3] = {static_cast<uint64_t>(p.latent_dim), wr, H}, ws[2] = {2 * wd[0], 2 * wd[0] * wr};
  const uint32_t wb[3] = {64, ABSORB ? 64u : static_cast<uint32_t>(NT), 1};
  if (!make_tmap16(&a.tmx, p.dtype, x, 3, xd, xs, xb) || !make_tmap16(&a.tmw, p.dtype, w, 3, wd, ws, wb))
    return cudaErrorNotSupported;
  a.n_tiles = static_cast<int>(N / NT);
  const auto kern = k_latent_heads<T, KC, NT, ST, ABSORB>;
  const size_t smem = 1024 + ST * (kABytes + NT * 128);
  const cudaError_t e = ensure_smem(kern, smem);
  if (e != cudaSuccess) return e;
  const long long tiles = (static_cast<long long>(a.total_q) + kRowsTile - 1) / kRowsTile * a.n_tiles;
  return launch_pdl(kern, dim3(static_cast<unsigned>(tiles), p.num_heads), dim3(kThreads), smem, st, a);
}

template <typename T>
cudaError_t heads(const spg_latent_params& p, bool project, HeadsArgs& a, const void* x, int64_t x_stride, const void* w,
                  cudaStream_t st) {
  if (!project)
    return p.nope_dim == 128 ? heads_typed<T, 2, 128, true>(p, a, x, x_stride, w, st)
                             : heads_typed<T, 1, 128, true>(p, a, x, x_stride, w, st);
  // 64 columns a CTA while one tile has all rows (twice the CTAs for the matrices' bytes)
  if (p.v_dim == 64 || a.total_q <= kRowsTile)
    return p.latent_dim == 512 ? heads_typed<T, 8, 64, false>(p, a, x, x_stride, w, st)
                               : heads_typed<T, 4, 64, false>(p, a, x, x_stride, w, st);
  return p.latent_dim == 512 ? heads_typed<T, 8, 128, false>(p, a, x, x_stride, w, st)
                             : heads_typed<T, 4, 128, false>(p, a, x, x_stride, w, st);
}

}  // namespace

cudaError_t launch_latent_heads(const spg_latent_params& p, bool project, int total_q, const void* x, int64_t x_stride,
                                const void* w_kv, void* y, cudaStream_t stream) {
  HeadsArgs a{};
  a.y = y;
  a.total_q = total_q;
  a.w_row = project ? p.nope_dim : 0;
  a.y_head = project ? p.v_dim : p.latent_dim + p.rope_dim;
  a.y_row = static_cast<long long>(p.num_heads) * a.y_head;
  return p.dtype == SPG_F16 ? heads<__half>(p, project, a, x, x_stride, w_kv, stream)
                            : heads<__nv_bfloat16>(p, project, a, x, x_stride, w_kv, stream);
}

}  // namespace spg
