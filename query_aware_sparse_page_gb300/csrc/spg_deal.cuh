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
//   Shape::kExtra        what an item costs beside its steps, in steps: it
//                        follows them in the count (steps() holds it)
// An item that crosses a border is worked on in parts; the CTAs of the parts
// are consecutive and each can tell who the others are.  No CTA waits for
// another: the part that arrives last joins them.
#pragma once

#include "spg_chunk_common.cuh"

namespace spg {

constexpr int kMaxCtas = 160;   // shares of a plan (one per SM)
constexpr int kMaxParts = 32;   // most parts an average item is split into

struct ChunkShape {
  const int32_t *q_start, *seq_lens;
  int B, Hkv, g_log2, total_q, max_tokens;  // 2^g_log2 query heads per kv-head
  __device__ ChunkSeq seq(int b, int32_t& bad) const { return chunk_seq(q_start, seq_lens, b, total_q, max_tokens, bad); }
};

struct Plan {
  long long total, lo, hi;  // steps in all, and this CTA's
  long long item_first;     // first step of the item that lo lies in
  int ctas, b, h, item;
};

// one whole warp
template <typename Shape>
__device__ void make_plan(const Shape& sh, Plan* out, int32_t* err, int lane) {
  long long total = 0, items = 0;
  int32_t bad = 0;
  for (int b = lane; b < sh.B; b += 32) {
    const ChunkSeq s = sh.seq(b, bad);
    const int ni = sh.items(s);
    total += sh.Hkv * sh.steps(s, ni);
    items += static_cast<long long>(sh.Hkv) * ni;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    items += __shfl_xor_sync(0xffffffffu, items, o);
  }
  if (bad && blockIdx.x == 0) record_error(err, bad);
  Plan p{};
  p.total = total;
  long long n = min(static_cast<long long>(gridDim.x), (total + Shape::kLeast - 1) / Shape::kLeast);
  n = min(n, items * kMaxParts);
  p.ctas = static_cast<int>(n);
  const int c = blockIdx.x;
  if (c >= n) {
    if (lane == 0) *out = p;  // lo = hi = 0: nothing to do
    return;
  }
  p.lo = c * total / n;
  p.hi = (c + 1) * total / n;
  long long base = 0;
  for (int b0 = 0; b0 < sh.B; b0 += 32) {
    const int b = b0 + lane;
    long long w = 0;
    ChunkSeq s{};
    if (b < sh.B) {
      s = sh.seq(b, bad);
      w = sh.Hkv * sh.steps(s, sh.items(s));
    }
    long long incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const long long first = base + incl - w;
    if (p.lo >= first && p.lo < first + w) {  // one lane
      const long long per_head = w / sh.Hkv;
      p.b = b;
      p.h = static_cast<int>((p.lo - first) / per_head);
      const long long rest = (p.lo - first) % per_head;
      int x = 0, y = sh.items(s) - 1;  // the last item that starts at or before rest
      while (x < y) {
        const int mid = (x + y + 1) >> 1;
        if (sh.steps(s, mid) <= rest) x = mid; else y = mid - 1;
      }
      p.item = x;
      p.item_first = first + p.h * per_head + sh.steps(s, x);
      *out = p;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
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
