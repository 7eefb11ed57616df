// Index arithmetic of the attention over the paged cache, for host and device
// (the CPU tests compile this header by itself).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define DSV_HD __host__ __device__ __forceinline__
#else
#define DSV_HD inline
#endif

namespace dsvit {

// The blocks of 2^shift keys that rows at positions p0 .. p1 see: the blocks
// of the first `sinks` keys that lie before the window of p0, then the
// blocks from that window's first key to p1.  Rows before position 0 see none.
struct KeyBlocks {
  int sink;    // blocks 0 .. sink - 1
  int first;   // then blocks first, first + 1, ...
  int count;   // both together
  DSV_HD int at(int i) const { return i < sink ? i : first + (i - sink); }
};

DSV_HD KeyBlocks key_blocks(int p0, int p1, int window, int sinks, int shift) {
  if (p1 < 0) return KeyBlocks{0, 0, 0};
  const int lo = window != 0 && p0 >= window ? p0 - window + 1 : 0;   // first key of p0's window
  const int first = lo >> shift;
  const int kept = sinks < lo ? sinks : lo;
  int sink = (kept >> shift) + ((kept & ((1 << shift) - 1)) != 0);
  if (sink > first) sink = first;
  return KeyBlocks{sink, first, sink + (p1 >> shift) - first + 1};
}

// U units of work dealt to W <= U workers in order: worker w takes units
// share_begin(w) .. share_begin(w + 1) - 1, at least one.
DSV_HD int64_t share_begin(int64_t w, int64_t W, int64_t U) { return w * U / W; }

// The worker that takes unit x: the largest w with floor(w U / W) <= x.
DSV_HD int64_t share_of(int64_t x, int64_t W, int64_t U) { return ((x + 1) * W - 1) / U; }

}  // namespace dsvit
