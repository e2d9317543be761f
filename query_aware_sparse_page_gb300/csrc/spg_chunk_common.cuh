// What the kernels over a ragged chunk of new tokens share: a sequence's rows
// and where they stand, checked before anything is read by them.
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
    s.L = 0;
    s.n = 0;
  }
  s.pos0 = s.L - s.n;
  return s;
}

// 8 values of a 16-byte piece
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2f<T>(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}

}  // namespace spg
