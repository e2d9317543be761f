// Tiles of 128 tokens of a paged pool in shared memory, as tensor-core
// operands: 128 threads copy 16 bytes at a time from the pages straight into
// the swizzled tile (halves of 64 channels, 128-byte rows).  Tokens that are
// not there become zeros on the way.  int8 codes land in the upper half of
// their tile's own space and are widened in place to exact 16-bit values.
#pragma once

#include "spg_tcgen05.cuh"

namespace spg {

constexpr int kTile = 128;

template <typename T, typename TQ, int D>
struct TileLoader {
  static constexpr bool I8 = sizeof(T) == 1;
  static constexpr int kThreads = 128;
  static constexpr uint32_t kHalf = kTile * 128, kTileBytes = D / 64 * kHalf;
  // A thread's pieces of a tile are one 16-byte column of every kPieces-th row.
  static constexpr int kCpr = D * static_cast<int>(sizeof(T)) / 16;  // pieces of a row
  static constexpr int kRowsPer = kThreads / kCpr;              // rows of the threads together
  static constexpr int kPieces = kTile / kRowsPer;

  // the pages of the tile of 128 tokens at t0, one per lane (-1: none before `end`, or a bad one)
  static __device__ __forceinline__ int page_of(const int32_t* pt, int t0, int end, int s_log2, int n_phys, int lane) {
    const int t = t0 + (lane << s_log2);
    if (lane >= kTile >> s_log2 || t >= end) return -1;
    const int page = pt[t >> s_log2];
    return page >= 0 && page < n_phys ? page : -1;
  }
  // copies the tile at t0 of kv-head h; tokens at or past L become zeros
  static __device__ __forceinline__ void copy(const void* pool, int Hkv, int h, int s_log2, int t0, int L, int page, int tid,
                                              uint32_t dst) {
    const int c = tid % kCpr, r0 = tid / kCpr, in_page = (1 << s_log2) - 1;
    const uint8_t* base = static_cast<const uint8_t*>(pool) + c * 16;
    if constexpr (I8) dst += kTileBytes / 2;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int r = r0 + i * kRowsPer;
      const int pg = __shfl_sync(0xffffffffu, page, r >> s_log2);
      const bool live = pg >= 0 && t0 + r < L;
      const size_t row = (((static_cast<size_t>(live ? pg : 0) * Hkv + h) << s_log2) + (r & in_page));
      uint32_t to;
      if constexpr (I8)
        to = r * D + c * 16;
      else
        to = (c >> 3) * kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4);
      copy16(dst + to, base + row * (D * sizeof(T)), live);
    }
  }

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
  // int8: the codes in the tile's upper half become the tile
  static __device__ __forceinline__ void widen(uint8_t* tile, int tid, int bar) {
    uint4 w[kPieces];
    const uint8_t* raw = tile + kTileBytes / 2;
    const int x = tid % kCpr, r0 = tid / kCpr, c = 2 * x;  // two 16-byte pieces of 16-bit values
#pragma unroll
    for (int i = 0; i < kPieces; ++i) w[i] = *reinterpret_cast<const uint4*>(raw + (r0 + i * kRowsPer) * D + x * 16);
    bar_sync(bar, kThreads);  // every code is in a register
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int r = r0 + i * kRowsPer;
      uint4 lo, hi;
      widen4(w[i].x, lo.x, lo.y);
      widen4(w[i].y, lo.z, lo.w);
      widen4(w[i].z, hi.x, hi.y);
      widen4(w[i].w, hi.z, hi.w);
      uint8_t* row = tile + (c >> 3) * kHalf + r * 128;
      *reinterpret_cast<uint4*>(row + (((c & 7) ^ (r & 7)) << 4)) = lo;
      *reinterpret_cast<uint4*>(row + ((((c & 7) + 1) ^ (r & 7)) << 4)) = hi;
    }
  }
};

}  // namespace spg
