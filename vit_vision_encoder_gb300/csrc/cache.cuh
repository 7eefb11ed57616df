// The paged K/V cache: argument blocks and device helpers shared by the
// kernels that write it, read it back and attend over it.
#pragma once

#include "cache_plan.h"
#include "internal.h"
#include "ptx.cuh"

namespace dsvit {

// Device view of a ds_vit_cache: pages [n_pages, kv_heads, page, D].
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_exp;   // e4m3 pages: exponent byte of each (page, head, slot)
  uint8_t* v_exp;
  int64_t n_pages;
  int kv_heads;
  int page_shift;   // page = 1 << page_shift tokens
};

// Device view of a ds_vit_chunks plus the rows of the packed tensors.
struct ChunkView {
  const int32_t* row_off;
  const int32_t* kv_len;
  const int32_t* table;
  int n, table_cols, max_rows;
  int rows;
};

// One sequence's part of the packed rows.
struct Seq {
  int row0;   // its first packed row
  int c;      // its rows (new tokens)
  int kv;     // its cached tokens, the new ones included
};

// Sequence s after the checks of its entries: rows ordered and inside the
// packed tensors, at most max_rows of them, no more tokens than the table
// row has places for.  On an error the code goes to *status and the sequence
// is taken as empty.
__device__ __forceinline__ Seq load_seq(const ChunkView& b, int page_shift, int s, int* status) {
  const int a = __ldg(b.row_off + s), e = __ldg(b.row_off + s + 1), kv = __ldg(b.kv_len + s);
  Seq q{a, e - a, kv};
  const int why = seq_refused(a, e, kv, b.rows, b.max_rows, static_cast<int64_t>(b.table_cols) << page_shift);
  if (why) {
    report_error(status, why == 1 ? DS_VIT_EINVAL : DS_VIT_ERANGE);
    q = Seq{0, 0, 0};
  }
  return q;
}

// The sequence that packed row r belongs to: the last s with row_off[s] <= r,
// found by a warp 32 ways at a time (two rounds of loads up to 1024
// sequences); -1 when r lies before the first or behind the last row.  Offsets
// out of order give some sequence, whose own checks then refuse it.
__device__ __forceinline__ int find_seq(const ChunkView& b, int r, int lane) {
  int lo = 0, n = b.n + 1;            // the answer's index is in [lo - 1, lo + n - 1]
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int at = lo + (lane + 1) * step - 1;
    const bool below = at < lo + n && at <= b.n && __ldg(b.row_off + at) <= r;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, below));
    const int end = lo + n;
    lo += k * step;
    n = min(step - 1, end - lo);
    if (k == 32) n = end - lo;
  }
  const int s = lo - 1;
  return s >= 0 && s < b.n ? s : -1;
}

// Page that holds position pos of sequence s, or -1 with *status set when the
// table's entry names no page.
__device__ __forceinline__ int64_t page_of(const ChunkView& b, const CacheView& c, int s, int pos, int* status) {
  const int p = __ldg(b.table + static_cast<int64_t>(s) * b.table_cols + (pos >> c.page_shift));
  if (!page_there(p, c.n_pages)) {
    report_error(status, DS_VIT_ERANGE);
    return -1;
  }
  return p;
}

// Row number of (page, head, slot) in the pages seen as rows of D values.
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int64_t page, int head, int pos) {
  return ((page * c.kv_heads + head) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// The factor 2^e of an exponent byte e + 127 (10 .. 247; 255 marks a row with
// an infinity or NaN, which reads as NaN).
__device__ __forceinline__ float exp_factor(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : byte << 23);
}

// Two e4m3 values -> two floats (exact).
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  float lo, hi;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return make_float2(lo, hi);
}

struct AttentionArgs {
  CacheView c;
  ChunkView b;
  const bf16* q;
  int64_t q_stride;     // elements between rows
  bf16* out;
  int64_t out_stride;
  int heads, group;     // group = heads / kv_heads
  FastDiv by_group;
  int window, sinks;
  float scale_log2;     // scale * log2(e)
  int* status;
};

// Whether the row at position p sees key j (j < kv always holds).
__device__ __forceinline__ bool sees(const AttentionArgs& a, int p, int j) {
  return j <= p && (a.window == 0 || j > p - a.window || j < a.sinks);
}

// The first key of the window of the row at position p.
__device__ __forceinline__ int window_start(const AttentionArgs& a, int p) {
  return a.window != 0 && p >= a.window ? p - a.window + 1 : 0;
}

}  // namespace dsvit
