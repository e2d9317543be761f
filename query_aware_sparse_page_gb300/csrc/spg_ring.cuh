// What a copying warp has put into a ring of ST stages whose PARTS parts are
// filled and given back by themselves.  Counted part by part: when a wait for
// room runs out between the parts of a step, those already issued are waited
// for like the others.
#pragma once

#include <stdint.h>

namespace spg {

template <int ST, int PARTS>
struct PartRing {
  uint32_t n[PARTS] = {};  // copies issued
  // The next copy of a part.  room(stage, phase): waits until the one before it
  // in its place has been read; issue(stage).  False when the wait ran out.
  template <typename Room, typename Issue>
  __host__ __device__ __forceinline__ bool put(int part, const Room& room, const Issue& issue) {
    const uint32_t stage = n[part] % ST;
    if (n[part] >= ST && !room(stage, n[part] / ST - 1)) return false;
    issue(stage);
    ++n[part];
    return true;
  }
  // landed(stage, part, phase) for every copy that nobody is known to have waited for
  template <typename Landed>
  __host__ __device__ __forceinline__ void drain(const Landed& landed) const {
    for (int part = 0; part < PARTS; ++part)
      for (uint32_t i = n[part] > ST ? n[part] - ST : 0; i < n[part]; ++i) landed(i % ST, part, i / ST);
  }
};

}  // namespace spg
