// What the kernels over a ragged chunk of new tokens share: which sequence
// and which rows a tile of the launch stands for.
//
// The host knows total_q but not q_start, so a launch has room for as many
// tiles as a batch of B sequences can need (floor(total / rows) + B) and
// every CTA finds its own on the device.
#pragma once

#include "spg_common.cuh"

namespace spg {

// One sequence of a chunk: rows [start, start + n), the first at cache
// position pos0 = L - n.  n = 0 when an entry is out of range.
struct ChunkSeq {
  int start, n, L, pos0;
};

__device__ __forceinline__ ChunkSeq chunk_seq(const int32_t* q_start, const int32_t* seq_lens, int b,
                                              int total_q, int max_tokens, int32_t& bad) {
  ChunkSeq s;
  s.start = q_start[b];
  const int end = q_start[b + 1];
  s.L = seq_lens[b];
  s.n = end - s.start;
  if (s.L < 0 || s.L > max_tokens) {
    bad |= SPG_DEVERR_SEQ_LEN;
    s.L = 0;
    s.n = 0;
  } else if (s.start < 0 || end > total_q || end < s.start || s.n > s.L) {
    bad |= SPG_DEVERR_Q_START;
    s.n = 0;
  }
  s.pos0 = s.L - s.n;
  return s;
}

// Tile `idx` of the launch when sequence b has ceil(n_b * G / rows) of them:
// the sequence and the tile within it.  One whole warp; false past the last.
__device__ __forceinline__ bool find_tile(const int32_t* q_start, const int32_t* seq_lens, int B, int total_q,
                                          int max_tokens, int G, int rows, int idx, int lane, int& b, int& tile,
                                          int32_t& bad) {
  int base = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    int tiles = 0;
    if (b0 + lane < B) {
      const ChunkSeq s = chunk_seq(q_start, seq_lens, b0 + lane, total_q, max_tokens, bad);
      tiles = static_cast<int>((static_cast<long long>(s.n) * G + rows - 1) / rows);
    }
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int lo = base + incl - tiles;
    const unsigned hit = __ballot_sync(0xffffffffu, idx >= lo && idx < lo + tiles);
    if (hit) {
      const int l = __ffs(hit) - 1;
      b = b0 + l;
      tile = idx - __shfl_sync(0xffffffffu, lo, l);
      return true;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

}  // namespace spg
