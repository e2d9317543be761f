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

}  // namespace spg
