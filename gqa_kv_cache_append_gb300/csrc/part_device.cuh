// part_device.cuh - where the rows lie that a unit reads of a part of the cache:
// the first `head` positions and those from `lo` on.
//
// A unit's tiles are cut from its span, in which the two places follow one
// another.  Copies move boxes of G positions (a power of two, at most a block
// of the table), so the head takes sb = head rounded up to G indices, and the
// body begins at the box that holds lo:
//
//   index v < sb   position v                  (seen: v < head)
//   index v >= sb  position v + shift          (seen: from lo on)
//
// With the body close behind the head nothing is left out (shift = 0, sb = 0: an
// index is a position).  Indices [head, z) and those of positions >= L are
// rows that no token of the call sees: they may hold anything, so their V rows
// are zeroed in shared memory (a weight of zero times NaN would be NaN).
#pragma once

#include "gqa_device.cuh"

namespace gqa {

struct PartSpan {
  int shift, sb, z;
};

// lo: first position of the unit's body; lo_all: that of all of the sequence's
// new tokens (at or below lo).  aligned: boxes start at multiples of G (else
// anywhere).  apart: the head is not the sequence's own rows.
__host__ __device__ __forceinline__ PartSpan part_span(int lo, int lo_all, int head, int G,
                                                       bool aligned, bool apart) {
  const int sb = (head + G - 1) & ~(G - 1);
  const int start = aligned ? lo & ~(G - 1) : lo;
  if (!apart && start <= sb) return {0, 0, lo_all};
  const int shift = start - sb;
  const int unseen = lo_all - shift;
  return {shift, sb, unseen > sb ? unseen : sb};
}

// the lowest n of 32 bits
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
}

// What a query row sees of a span: [0, head) and [lo, hi).
struct PartVisible {
  int head, lo, hi;
  __device__ bool all(int x0, int n) const {
    return x0 + n <= head || (x0 >= lo && x0 + n <= hi);
  }
  __device__ uint32_t bits(int x0) const {  // of the 32 indices from x0 on
    return low_bits(head - x0) | (low_bits(hi - x0) & ~low_bits(lo - x0));
  }
};

// The tiles of a sequence whose n = lmin new tokens see their last `window`
// positions and the first `sinks` (one unit to a KV head).
struct WindowSpan {
  int window, sinks, gran;
  __device__ __forceinline__ PartSpan at(int L, int n) const {
    const int lo = max(L - n - window + 1, 0);
    return part_span(lo, lo, sinks, gran, true, false);
  }
  __device__ __forceinline__ int tiles(int L, int lmin, int cap, int T) const {
    if (L < lmin || L < 1 || L > cap) return 0;
    return (L - at(L, lmin).shift + T - 1) / T;
  }
};

}  // namespace gqa
