// Work over a ragged chunk dealt out to the CTAs of one launch.
//
// An item is a tile of one (sequence, kv-head); it takes a number of steps
// that only the device knows.  The steps of all items, in the order
// (sequence, kv-head, item), are cut into equal contiguous shares, one per
// CTA, whatever the lengths.  Every CTA finds its share by itself, from
// prefix sums that the kernel's shape gives in closed form:
//   Shape::items(s)      items of one kv-head of sequence s
//   Shape::steps(s, m)   steps of the first m of them
//   Shape::item_steps(s, i)  steps of item i alone (every role asks at every
//                        item's start: kept to a few instructions)
//   Shape::kLeast        fewest steps worth a CTA of their own
//   Shape::kMostParts   most parts an average item is split into
//   Shape::kExtra        what an item costs beside its steps, in steps: it
//                        follows them in the count (steps() holds it)
// An item that crosses a border is worked on in parts; the CTAs of the parts
// are consecutive and each can tell who the others are.  No CTA waits for
// another: the part that arrives last joins them.
#pragma once

#include "spg_chunk_common.cuh"

namespace spg {

constexpr int kMaxCtas = 160;   // shares of a plan (one per SM)

struct ChunkShape {
  static constexpr int kMostParts = 32;
  const int32_t *q_start, *seq_lens;
  int B, Hkv, g_log2, total_q, max_tokens;  // 2^g_log2 query heads per kv-head
  __device__ ChunkSeq seq(int b, int32_t& bad) const { return chunk_seq(q_start, seq_lens, b, total_q, max_tokens, bad); }
};

// a / b, b > 0, a >= 0: in 32 bits where both fit, a sixth of the time
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  if ((static_cast<unsigned long long>(a) | static_cast<unsigned long long>(b)) >> 32)
    return a / b;
  return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

struct Plan {
  long long total, lo, hi;  // steps in all, and this CTA's
  long long item_first;     // first step of the item that lo lies in
  int ctas, b, h, item, n_items;
  ChunkSeq sq;              // sequence b
};

// one whole warp; the share of CTA c of n_ctas
template <typename Shape>
__device__ void make_plan(const Shape& sh, Plan* out, int32_t* err, int lane, int c = static_cast<int>(blockIdx.x),
                          int n_ctas = static_cast<int>(gridDim.x)) {
  // steps up to and with each lane's first sequence, then those of the others
  long long items = 0;
  int32_t bad = 0;
  ChunkSeq first_sq{};
  int first_items = 0;
  long long first_w = 0;
  if (lane < sh.B) {
    first_sq = sh.seq(lane, bad);
    first_items = sh.items(first_sq);
    first_w = sh.Hkv * sh.steps(first_sq, first_items);
  }
  long long incl = first_w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  const long long first_incl = incl, first_total = __shfl_sync(0xffffffffu, incl, 31);
  long long total = first_total;
  items = static_cast<long long>(sh.Hkv) * first_items;
  if (sh.B > 32) {
    long long rest = 0;
    for (int b = lane + 32; b < sh.B; b += 32) {
      const ChunkSeq s = sh.seq(b, bad);
      const int ni = sh.items(s);
      rest += sh.Hkv * sh.steps(s, ni);
      items += static_cast<long long>(sh.Hkv) * ni;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
    total += rest;
  }
  if constexpr (Shape::kMostParts < kMaxCtas) {  // else no item can have more parts
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) items += __shfl_xor_sync(0xffffffffu, items, o);
  }
  if (bad && blockIdx.x == 0) record_error(err, bad);
  Plan p{};
  p.total = total;
  long long n = min(static_cast<long long>(n_ctas), (total + Shape::kLeast - 1) / Shape::kLeast);
  if constexpr (Shape::kMostParts < kMaxCtas) n = min(n, items * Shape::kMostParts);
  p.ctas = static_cast<int>(n);
  if (c >= n) {
    if (lane == 0) *out = p;  // lo = hi = 0: nothing to do
    return;
  }
  p.lo = div_pos(c * total, n);
  p.hi = div_pos((c + 1) * total, n);
  long long base = 0;
  for (int b0 = 0; b0 < sh.B; b0 += 32) {
    const int b = b0 + lane;
    long long w = first_w, upto = first_incl;
    ChunkSeq s = first_sq;
    int ni = first_items;
    if (b0 > 0) {
      w = 0;
      if (b < sh.B) {
        s = sh.seq(b, bad);
        ni = sh.items(s);
        w = sh.Hkv * sh.steps(s, ni);
      }
      upto = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
    }
    const long long first = base + upto - w;
    if (p.lo >= first && p.lo < first + w) {  // one lane
      const long long per_head = div_pos(w, sh.Hkv);
      p.b = b;
      p.h = static_cast<int>(div_pos(p.lo - first, per_head));
      const long long rest = p.lo - first - p.h * per_head;
      int x = 0, y = ni - 1;  // the last item that starts at or before rest
      while (x < y) {
        const int mid = (x + y + 1) >> 1;
        if (sh.steps(s, mid) <= rest) x = mid; else y = mid - 1;
      }
      p.item = x;
      p.n_items = ni;
      p.sq = s;
      p.item_first = first + p.h * per_head + sh.steps(s, x);
      *out = p;
    }
    base += b0 == 0 ? first_total : __shfl_sync(0xffffffffu, upto, 31);
    if (base > p.lo) break;
  }
}

// A CTA's part of one item: steps [k0, k1) of its nk.
struct Part {
  ChunkSeq sq;
  int b, h, item, k0, k1, nk;
  long long item_first;
  __device__ bool whole() const { return k0 == 0 && k1 == nk; }
};

// The parts of a CTA's share in order; every role walks them by itself.
template <typename Shape>
struct PartIter {
  const Shape& sh;
  long long pos, hi, item_first;
  int b, h, item, n_items;
  ChunkSeq sq;
  __device__ PartIter(const Shape& shape, const Plan& p)
      : sh(shape), pos(p.lo), hi(p.hi), item_first(p.item_first), b(p.b), h(p.h), item(p.item) {
    if (pos < hi) load();
  }
  // the first sequence from the plan (the reads of load() are 700 cycles on the way to the first copy)
  struct Planned {};
  __device__ PartIter(const Shape& shape, const Plan& p, Planned)
      : sh(shape), pos(p.lo), hi(p.hi), item_first(p.item_first), b(p.b), h(p.h), item(p.item), n_items(p.n_items), sq(p.sq) {}
  __device__ void load() {
    int32_t bad = 0;
    sq = sh.seq(b, bad);
    n_items = sh.items(sq);
  }
  __device__ bool next(Part& s) {
    while (pos < hi) {
      s.sq = sq;
      s.b = b;
      s.h = h;
      s.item = item;
      s.nk = sh.item_steps(sq, item);
      s.item_first = item_first;
      s.k0 = static_cast<int>(pos - item_first);
      s.k1 = static_cast<int>(min(static_cast<long long>(s.nk), hi - item_first));
      const long long end = item_first + s.nk + Shape::kExtra;
      pos = min(end, hi);
      if (pos == end) {
        item_first = end;
        if (++item == n_items) {
          item = 0;
          if (++h == sh.Hkv) {
            h = 0;
            if (pos < hi) do { ++b; load(); } while (n_items == 0);
          }
        }
      }
      if (s.k0 < s.k1) return true;  // else the share began behind the item's last step
    }
    return false;
  }
};

// Where the parts of an item are: CTAs c0 .. c1.  A CTA has two slots for
// parts, one for an item it enters in the middle and one for an item it
// begins and does not end.
struct PartRange {
  int c0, c1;
  __device__ PartRange(const Plan& p, const Part& s)
      : c0(static_cast<int>(((s.item_first + 1) * p.ctas - 1) / p.total)),
        c1(static_cast<int>(((s.item_first + s.nk) * p.ctas - 1) / p.total)) {}
  __device__ int slot(int c) const { return c == c0 ? 2 * c + 1 : 2 * c; }
};
__device__ __forceinline__ int own_slot(const Part& s) { return 2 * static_cast<int>(blockIdx.x) + (s.k0 > 0 ? 0 : 1); }

}  // namespace spg
