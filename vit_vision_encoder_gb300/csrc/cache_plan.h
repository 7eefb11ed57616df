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

// Why a sequence is refused: 1 for rows out of order, outside the packed ones
// or more than max_rows, 2 for a length that the table row has no places for, 0
// if it is not.
DSV_HD int seq_refused(int row0, int row1, int kv, int rows, int max_rows, int64_t places) {
  if (row0 < 0 || row1 < row0 || row1 > rows || row1 - row0 > max_rows) return 1;
  return kv < 0 || kv > places ? 2 : 0;
}
DSV_HD bool page_there(int page, int64_t n_pages) { return page >= 0 && page < n_pages; }

// The sequences whose entries a thread of a grid checks: check_first, + check_step,
// ... below n.  Grids of up to 2^28 blocks (rows are fewer than 2^30): 64 bits.
DSV_HD int64_t check_first(uint32_t block, int threads, int thread) {
  return static_cast<int64_t>(block) * threads + thread;
}
DSV_HD int64_t check_step(uint32_t blocks, int threads) { return static_cast<int64_t>(blocks) * threads; }

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

// U units of work dealt in order to W workers, W <= U (or both 0): the first
// `more` take each + 1 units, the others `each`.
struct Shares {
  int64_t each, more;
  DSV_HD int64_t begin(int64_t w) const { return w * each + (w < more ? w : more); }
  // The worker that takes unit x.
  DSV_HD int64_t owner(int64_t x) const {
    const int64_t head = more * (each + 1);
    return x < head ? x / (each + 1) : more + (x - head) / each;
  }
};
DSV_HD Shares deal(int64_t U, int64_t W) {
  const int64_t each = W > 0 ? U / W : 0;
  return Shares{each, U - each * W};
}

// Division of 0 <= n < 2^31 by a fixed d >= 1 without a divide: with
// 2^s >= d and m = ceil(2^(32 + s) / d) - 2^32, n / d = (mulhi(n, m) + n) >> s.
struct FastDiv {
  uint32_t m;
  int s, d;
  DSV_HD int operator()(int n) const {
    const uint32_t u = static_cast<uint32_t>(n);
    return static_cast<int>((static_cast<uint32_t>((static_cast<uint64_t>(u) * m) >> 32) + u) >> s);
  }
};
inline FastDiv fast_div(int d) {
  int s = 0;
  while ((int64_t{1} << s) < d) ++s;
  const uint64_t m = ((((uint64_t{1} << s) - static_cast<uint64_t>(d)) << 32) + static_cast<uint64_t>(d) - 1) /
                     static_cast<uint64_t>(d);
  return FastDiv{static_cast<uint32_t>(m), s, d};
}

// A share's border inside an item of units i0 .. i1 - 1, the first `cost` of
// which stand for what an item takes besides its tiles.  It moves to the item's
// nearer end when that is at most `snap` units away (a split item costs a second
// load of its rows, a record of each part and their sum), and never lies within
// the first `cost`.
DSV_HD int64_t snap_border(int64_t x, int64_t i0, int64_t i1, int64_t snap, int64_t cost) {
  const int64_t a = x - i0, b = i1 - x;
  if (a > b) return b <= snap ? i1 : a <= cost ? i0 : x;
  return a <= snap || a <= cost ? i0 : x;
}

}  // namespace dsvit
