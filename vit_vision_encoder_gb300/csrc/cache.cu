// The paged K/V cache of the prompt's language model: writing the rows of new
// tokens, reading rows back, and the entry points (include/dsvit.h).
//
// Both kernels move each byte once and are bound by memory at prompt lengths,
// by their chain of dependent loads (row -> sequence -> page -> slot) at one
// token a sequence.  One warp takes one token: its keys and values of all
// heads are two contiguous runs of the packed rows, read as 16-byte pieces (few
// heads and many rows: several tokens, cache_read_tokens_kernel).
// Measured at 8 heads of 128, inputs not in L2: 6900 rows quantised as they are written
// 12.9 us (49% of the rate of a plain copy, pieces of 128 bytes scattered over the pages;
// 8.4 with everything in L2), 92 thousand tokens read back out of e4m3 pages 86 us (98%),
// 48 single tokens 2.7 us.
#include "cache.cuh"

namespace dsvit {

namespace {

constexpr int kWarps = 4;     // tokens per block
constexpr int kPieces = 4;    // 16-byte pieces of the keys, and as many of the values, in flight per lane

// Quantisation of one row (a token's key or value of one head) to e4m3 with
// a power-of-two factor: a = max |x|, e the least integer with a <= 448 2^e
// (448 is the largest e4m3 value), at least -117 so that every value read
// back is a normal bf16 number; q = e4m3(x 2^-e), rounded to nearest even.  In
// the bits of a (exponent field E, mantissa M): 448 = 1.75 2^8, so
// e + 127 = E - 8, plus 1 when M > 96.  A power of two costs no accuracy (the
// elements are floating point) and makes the value read back exact in bf16;
// at e = 120, where 256 2^e would be past bf16's largest number, elements end
// at 240.
__device__ __forceinline__ uint32_t exponent_byte(uint32_t amax_bits) {
  const uint32_t E = amax_bits >> 7, M = amax_bits & 127u;
  if (E == 255u) return 255u;
  const int byte = static_cast<int>(E) - 8 + (M > 96u ? 1 : 0);
  return static_cast<uint32_t>(byte < 10 ? 10 : byte);
}

__device__ __forceinline__ uint32_t max_abs_bits(uint4 u) {
  // bf16 magnitudes order like their bits; NaN and infinity come out on top.
  const uint32_t a = __vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu);
  const uint32_t b = __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu);
  const uint32_t m = __vmaxu2(a, b);
  return max(m & 0xFFFFu, m >> 16);
}

// Two bf16 values times f as e4m3.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t two, float f) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(bf16hi(two) * f), "f"(bf16lo(two) * f));
  return r;
}

// One 16-byte piece w of a row of keys (x 0) or values into its place; the lanes of
// the row's other pieces are beside this one, and all lanes of the warp take part.
template <int D, bool E4M3>
__device__ __forceinline__ void write_piece(const CacheView& c, int x, int64_t row, int piece, bool on, uint4 w) {
  constexpr int kLanes = D / 8;
  uint8_t* to = x == 0 ? c.k : c.v;
  if constexpr (!E4M3) {
    if (on) reinterpret_cast<uint4*>(to)[row * kLanes + piece] = w;
  } else {
    uint32_t a = max_abs_bits(w);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    const uint32_t byte = exponent_byte(a);
    const float f = __uint_as_float((254u - byte) << 23);    // 2^-e
    uint2 y = make_uint2(e4m3x2(w.x, f) | e4m3x2(w.y, f) << 16, e4m3x2(w.z, f) | e4m3x2(w.w, f) << 16);
    if (byte >= 247u) {
      if (byte == 255u) {
        y = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
      } else {                                               // magnitudes 256 (0x78) end at 240 (0x77)
        y.x -= __vcmpgtu4(y.x & 0x7F7F7F7Fu, 0x77777777u) & 0x01010101u;
        y.y -= __vcmpgtu4(y.y & 0x7F7F7F7Fu, 0x77777777u) & 0x01010101u;
      }
    }
    if (on) {
      reinterpret_cast<uint2*>(to)[row * kLanes + piece] = y;
      if (piece == 0) (x == 0 ? c.k_exp : c.v_exp)[row] = static_cast<uint8_t>(byte);
    }
  }
}

// Every sequence's entries are checked, also those of sequences without rows.
__device__ __forceinline__ void check_seqs(const ChunkView& b, int page_shift, int* status) {
  const int64_t step = check_step(gridDim.x, 32 * kWarps);
  for (int64_t s = check_first(blockIdx.x, 32 * kWarps, threadIdx.x); s < b.n; s += step)
    load_seq(b, page_shift, static_cast<int>(s), status);
}

__device__ __forceinline__ bool has_row(const Seq& q, int r) {
  return static_cast<unsigned>(r - q.row0) < static_cast<unsigned>(q.c);
}

// kLanes lanes hold one row (a head's key or value) in 16-byte pieces, a warp
// kHeads heads at a time; a lane keeps its piece of the row throughout.
template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps)
    cache_write_kernel(const __grid_constant__ CacheView c, const __grid_constant__ ChunkView b,
                       const bf16* __restrict__ k, int64_t k_stride, const bf16* __restrict__ v,
                       int64_t v_stride, int* status) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int r = static_cast<int>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  check_seqs(b, c.page_shift, status);
  if (r >= b.rows) return;
  const int piece = lane % kLanes, h0 = lane / kLanes;
  const uint4* from[2] = {reinterpret_cast<const uint4*>(k + r * k_stride) + lane,
                          reinterpret_cast<const uint4*>(v + r * v_stride) + lane};
  // The token's first pieces are on their way while its place is looked up.
  uint4 u[2][kPieces];
  auto load = [&](int hb) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int t = 0; t < kPieces; ++t)
        u[x][t] = hb + h0 + t * kHeads < c.kv_heads ? __ldg(from[x] + hb * kLanes + 32 * t) : make_uint4(0, 0, 0, 0);
  };
  load(0);
  const int s = find_seq(b, r, lane);
  if (s < 0) return;
  const Seq q = load_seq(b, c.page_shift, s, status);
  const int pos = q.kv - q.c + (r - q.row0);
  if (!has_row(q, r) || pos < 0) return;        // refused sequence, or padding in front of position 0
  const int64_t page = page_of(b, c, s, pos, status);
  if (page < 0) return;
  const int64_t row0 = cache_row(c, page, h0, pos);
  for (int hb = 0; hb < c.kv_heads; hb += kHeads * kPieces) {
    if (hb > 0) load(hb);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int t = 0; t < kPieces; ++t) {
        const int h = hb + t * kHeads;                             // head of the warp's first lanes
        const int64_t row = row0 + (static_cast<int64_t>(h) << c.page_shift);
        const bool on = h + h0 < c.kv_heads;
        const uint4 w = u[x][t];
        if (E4M3 && h >= c.kv_heads) break;
        write_piece<D, E4M3>(c, x, row, piece, on, w);
      }
    }
  }
}

__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two, float f) {
  const float2 x = e4m3x2_to_float2(static_cast<uint16_t>(two));
  return pack_bf16x2(x.x * f, x.y * f);   // exact: 4 significant bits, a normal exponent
}

// What a piece of a row of keys or values holds, and the row's exponent byte.
template <int D, bool E4M3>
__device__ __forceinline__ void read_piece(const CacheView& c, int x, int64_t row, int piece, uint4& u, uint32_t& byte) {
  constexpr int kLanes = D / 8;
  const uint8_t* from = x == 0 ? c.k : c.v;
  if constexpr (!E4M3) {
    u = reinterpret_cast<const uint4*>(from)[row * kLanes + piece];
  } else {
    const uint2 w = reinterpret_cast<const uint2*>(from)[row * kLanes + piece];
    u.x = w.x;
    u.y = w.y;
    byte = (x == 0 ? c.k_exp : c.v_exp)[row];
  }
}
template <bool E4M3>
__device__ __forceinline__ uint4 as_bf16(uint4 w, uint32_t byte) {
  if constexpr (!E4M3) return w;
  const float f = exp_factor(byte);
  return make_uint4(e4m3x2_to_bf16x2(w.x & 0xFFFFu, f), e4m3x2_to_bf16x2(w.x >> 16, f),
                    e4m3x2_to_bf16x2(w.y & 0xFFFFu, f), e4m3x2_to_bf16x2(w.y >> 16, f));
}

// The inverse: rows of the packed outputs from the pages.  Rows in front of
// position 0 are zeros; rows behind the last sequence stay as they were.
template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps)
    cache_read_kernel(const __grid_constant__ CacheView c, const __grid_constant__ ChunkView b,
                      bf16* __restrict__ k, int64_t k_stride, bf16* __restrict__ v, int64_t v_stride, int* status) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int r = static_cast<int>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  check_seqs(b, c.page_shift, status);
  if (r >= b.rows) return;
  const int piece = lane % kLanes, h0 = lane / kLanes;
  const int s = find_seq(b, r, lane);
  if (s < 0) return;
  const Seq q = load_seq(b, c.page_shift, s, status);
  if (!has_row(q, r)) return;
  const int pos = q.kv - q.c + (r - q.row0);
  const int64_t page = pos < 0 ? -1 : page_of(b, c, s, pos, status);
  if (page < 0 && pos >= 0) return;
  const int64_t row0 = page < 0 ? 0 : cache_row(c, page, h0, pos);
  for (int hb = 0; hb < c.kv_heads; hb += kHeads * kPieces) {
    uint4 u[2][kPieces];
    uint32_t byte[2][kPieces];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int t = 0; t < kPieces; ++t) {
        const int h = hb + t * kHeads;
        const int64_t row = row0 + (static_cast<int64_t>(h) << c.page_shift);
        u[x][t] = make_uint4(0, 0, 0, 0);
        byte[x][t] = 127;
        if (h + h0 < c.kv_heads && page >= 0) {
          read_piece<D, E4M3>(c, x, row, piece, u[x][t], byte[x][t]);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint4* to = reinterpret_cast<uint4*>(x == 0 ? k + r * k_stride : v + r * v_stride) + hb * kLanes + lane;
#pragma unroll
      for (int t = 0; t < kPieces; ++t) {
        if (hb + t * kHeads + h0 >= c.kv_heads) continue;
        to[32 * t] = as_bf16<E4M3>(u[x][t], byte[x][t]);
      }
    }
  }
}

// Few K/V heads leave most of a warp's places for pieces empty; where the rows are
// more than run at once, a warp then takes several tokens in a row: place y holds
// head y % kv_heads of token y / kv_heads.  92 thousand tokens, one token a warp / several,
// us, e4m3: one head of 128 read 36.6 / 12.9, written 35.3 / 16.6, four heads of 64 (four
// tokens) 41.1 / 26.8 and 36.7 / 32.4; two tokens at a time gain nothing (51 / 49, 53 / 60).
struct Place {
  int r, head;     // packed row; r < 0: nothing here
  int64_t row;     // in the pages; < 0: in front of position 0
};

__device__ __forceinline__ Place place_of(const CacheView& c, const ChunkView& b, int first, int tokens, int y, int s,
                                          int* status) {
  const Place none{-1, 0, -1};
  const int i = y / c.kv_heads, r = first + i;
  if (i >= tokens || r >= b.rows) return none;
  while (s + 1 < b.n && r >= __ldg(b.row_off + s + 1)) ++s;
  const Seq q = load_seq(b, c.page_shift, s, status);
  if (!has_row(q, r)) return none;
  const int pos = q.kv - q.c + (r - q.row0), head = y - i * c.kv_heads;
  if (pos < 0) return Place{r, head, -1};
  const int64_t page = page_of(b, c, s, pos, status);
  return page < 0 ? none : Place{r, head, cache_row(c, page, head, pos)};
}

// The sequence to look from for rows first, first + 1, ...; -1 if all of them lie behind the last.
__device__ __forceinline__ int seq_from(const ChunkView& b, int first, int lane) {
  const int s = find_seq(b, first, lane);
  return s >= 0 || first >= __ldg(b.row_off) ? s : 0;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps)
    cache_write_tokens_kernel(const __grid_constant__ CacheView c, const __grid_constant__ ChunkView b,
                              const bf16* __restrict__ k, int64_t k_stride, const bf16* __restrict__ v,
                              int64_t v_stride, int tokens, int* status) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, piece = lane % kLanes, h0 = lane / kLanes;
  const int first = (static_cast<int>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * tokens;
  check_seqs(b, c.page_shift, status);
  if (first >= b.rows) return;
  uint4 u[2][kPieces];
#pragma unroll
  for (int t = 0; t < kPieces; ++t) {
    const int y = t * kHeads + h0, i = y / c.kv_heads, r = first + i;
    const int at = (y - i * c.kv_heads) * D + piece * 8;
    const bool on = i < tokens && r < b.rows;
    u[0][t] = on ? __ldg(reinterpret_cast<const uint4*>(k + r * k_stride + at)) : make_uint4(0, 0, 0, 0);
    u[1][t] = on ? __ldg(reinterpret_cast<const uint4*>(v + r * v_stride + at)) : make_uint4(0, 0, 0, 0);
  }
  const int s = seq_from(b, first, lane);
  if (s < 0) return;
  Place to[kPieces];
#pragma unroll
  for (int t = 0; t < kPieces; ++t) to[t] = place_of(c, b, first, tokens, t * kHeads + h0, s, status);
  __syncwarp();
#pragma unroll
  for (int t = 0; t < kPieces; ++t)
#pragma unroll
    for (int x = 0; x < 2; ++x) write_piece<D, E4M3>(c, x, to[t].row, piece, to[t].r >= 0 && to[t].row >= 0, u[x][t]);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps)
    cache_read_tokens_kernel(const __grid_constant__ CacheView c, const __grid_constant__ ChunkView b,
                             bf16* __restrict__ k, int64_t k_stride, bf16* __restrict__ v, int64_t v_stride, int tokens,
                             int* status) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, piece = lane % kLanes, h0 = lane / kLanes;
  const int first = (static_cast<int>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * tokens;
  check_seqs(b, c.page_shift, status);
  if (first >= b.rows) return;
  const int s = seq_from(b, first, lane);
  if (s < 0) return;
  Place from[kPieces];
#pragma unroll
  for (int t = 0; t < kPieces; ++t) from[t] = place_of(c, b, first, tokens, t * kHeads + h0, s, status);
  uint4 u[2][kPieces];
  uint32_t byte[2][kPieces];
#pragma unroll
  for (int t = 0; t < kPieces; ++t)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      u[x][t] = make_uint4(0, 0, 0, 0);
      byte[x][t] = 127;
      if (from[t].row >= 0) read_piece<D, E4M3>(c, x, from[t].row, piece, u[x][t], byte[x][t]);
    }
#pragma unroll
  for (int t = 0; t < kPieces; ++t) {
    if (from[t].r < 0) continue;
    const int at = from[t].head * D + piece * 8;
    *reinterpret_cast<uint4*>(k + from[t].r * k_stride + at) = as_bf16<E4M3>(u[0][t], byte[0][t]);
    *reinterpret_cast<uint4*>(v + from[t].r * v_stride + at) = as_bf16<E4M3>(u[1][t], byte[1][t]);
  }
}

// Tokens a warp takes: one, or as many as its places hold (four at least) where the
// rows are more warps than the device runs at once.
int tokens_per_warp(int head_dim, int kv_heads, int64_t rows) {
  const int places = kPieces * 32 / (head_dim / 8);
  return rows > 64 * static_cast<int64_t>(num_sms()) && places >= 4 * kv_heads ? places / kv_heads : 1;
}

}  // namespace

int check_pages_of(const ds_vit_cache* c, CacheView* cv) {
  if (!c || !c->k || !c->v) return DS_VIT_EINVAL;
  if ((c->kind != DS_VIT_CACHE_BF16 && c->kind != DS_VIT_CACHE_E4M3) || (c->head_dim != 64 && c->head_dim != 128) ||
      c->kv_heads < 1 || c->kv_heads > DS_VIT_CACHE_MAX_HEADS || c->n_pages < 1)
    return DS_VIT_EINVAL;
  int shift = 4;
  while (shift < 7 && (1 << shift) != c->page) ++shift;
  if ((1 << shift) != c->page) return DS_VIT_EINVAL;
  if (c->kind == DS_VIT_CACHE_E4M3 && (!c->k_exp || !c->v_exp || !aligned(c->k_exp, 16) || !aligned(c->v_exp, 16)))
    return DS_VIT_EINVAL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return DS_VIT_EINVAL;
  // Rows of the pages are TMA coordinates.
  if (c->n_pages > INT32_MAX / (c->page * c->kv_heads)) return DS_VIT_ERANGE;
  *cv = CacheView{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->k_exp, c->v_exp,
                  c->n_pages, c->kv_heads, shift};
  return DS_VIT_OK;
}

int check_cache(const ds_vit_cache* c, const ds_vit_chunks* b, int64_t rows, CacheView* cv, ChunkView* bv) {
  if (!b || !b->row_off || !b->kv_len || !b->table) return DS_VIT_EINVAL;
  const int rc = check_pages_of(c, cv);
  if (rc == DS_VIT_EINVAL) return rc;
  if (!aligned(b->row_off, 4) || !aligned(b->kv_len, 4) || !aligned(b->table, 4)) return DS_VIT_EINVAL;
  if (b->n < 1 || b->n > DS_VIT_MAX_SEQS || b->table_cols < 1 || b->max_rows < 1 || rows < 0) return DS_VIT_EINVAL;
  if (rc) return rc;
  // Positions are int32.
  if (b->table_cols > (INT32_MAX - 255) / c->page || rows > INT32_MAX / 2) return DS_VIT_ERANGE;
  *bv = ChunkView{b->row_off, b->kv_len, b->table, b->n, b->table_cols, b->max_rows, static_cast<int>(rows)};
  return DS_VIT_OK;
}

namespace {

// Rows that share a K/V head in one sequence: few of them leave the call bound
// by the cache's bytes, and the kernel that streams those through warp MMAs is
// taken; with more rows the tcgen05 one.
bool few_rows(const ChunkView& b, int head_dim, int group, bool e4m3) {
  return static_cast<int64_t>(b.max_rows) * group <= decode_rows(head_dim, e4m3);
}

size_t attention_workspace(const ChunkView& b, int head_dim, int group, bool e4m3) {
  return few_rows(b, head_dim, group, e4m3) ? cache_decode_workspace(head_dim, b.max_rows * group)
                                  : cache_prefill_workspace(head_dim);
}

}  // namespace

}  // namespace dsvit

using namespace dsvit;

extern "C" {

int ds_vit_cache_write(const ds_vit_cache* cache, const ds_vit_chunks* chunks, const void* k, int64_t k_stride,
                       const void* v, int64_t v_stride, int64_t rows, int32_t* status, void* stream) {
  CacheView c;
  ChunkView b;
  if (const int rc = check_cache(cache, chunks, rows, &c, &b)) return rc;
  const int64_t width = static_cast<int64_t>(c.kv_heads) * cache->head_dim;
  if (!status || !aligned(status, 4) || bad_rows(k, k_stride, width) || bad_rows(v, v_stride, width))
    return DS_VIT_EINVAL;
  if (rows == 0) return DS_VIT_OK;
  const bool e4m3 = cache->kind == DS_VIT_CACHE_E4M3;
  const int tokens = tokens_per_warp(cache->head_dim, c.kv_heads, rows);
  const dim3 grid(static_cast<unsigned>((rows + kWarps * tokens - 1) / (kWarps * tokens))), block(32 * kWarps);
  auto* s = static_cast<cudaStream_t>(stream);
  auto* kp = static_cast<const bf16*>(k);
  auto* vp = static_cast<const bf16*>(v);
  auto* st = reinterpret_cast<int*>(status);
  if (tokens > 1) {
    auto* fn = cache->head_dim == 128 ? (e4m3 ? cache_write_tokens_kernel<128, true> : cache_write_tokens_kernel<128, false>)
                                      : (e4m3 ? cache_write_tokens_kernel<64, true> : cache_write_tokens_kernel<64, false>);
    return launched(launch_pdl(fn, grid, block, 0, s, c, b, kp, k_stride, vp, v_stride, tokens, st));
  }
  auto* fn = cache->head_dim == 128 ? (e4m3 ? cache_write_kernel<128, true> : cache_write_kernel<128, false>)
                                    : (e4m3 ? cache_write_kernel<64, true> : cache_write_kernel<64, false>);
  return launched(launch_pdl(fn, grid, block, 0, s, c, b, kp, k_stride, vp, v_stride, st));
}

int ds_vit_cache_read(const ds_vit_cache* cache, const ds_vit_chunks* chunks, void* k, int64_t k_stride, void* v,
                      int64_t v_stride, int64_t rows, int32_t* status, void* stream) {
  CacheView c;
  ChunkView b;
  if (const int rc = check_cache(cache, chunks, rows, &c, &b)) return rc;
  const int64_t width = static_cast<int64_t>(c.kv_heads) * cache->head_dim;
  if (!status || !aligned(status, 4) || bad_rows(k, k_stride, width) || bad_rows(v, v_stride, width))
    return DS_VIT_EINVAL;
  if (rows == 0) return DS_VIT_OK;
  const bool e4m3 = cache->kind == DS_VIT_CACHE_E4M3;
  const int tokens = tokens_per_warp(cache->head_dim, c.kv_heads, rows);
  const dim3 grid(static_cast<unsigned>((rows + kWarps * tokens - 1) / (kWarps * tokens))), block(32 * kWarps);
  auto* s = static_cast<cudaStream_t>(stream);
  auto* kp = static_cast<bf16*>(k);
  auto* vp = static_cast<bf16*>(v);
  auto* st = reinterpret_cast<int*>(status);
  if (tokens > 1) {
    auto* fn = cache->head_dim == 128 ? (e4m3 ? cache_read_tokens_kernel<128, true> : cache_read_tokens_kernel<128, false>)
                                      : (e4m3 ? cache_read_tokens_kernel<64, true> : cache_read_tokens_kernel<64, false>);
    return launched(launch_pdl(fn, grid, block, 0, s, c, b, kp, k_stride, vp, v_stride, tokens, st));
  }
  auto* fn = cache->head_dim == 128 ? (e4m3 ? cache_read_kernel<128, true> : cache_read_kernel<128, false>)
                                    : (e4m3 ? cache_read_kernel<64, true> : cache_read_kernel<64, false>);
  return launched(launch_pdl(fn, grid, block, 0, s, c, b, kp, k_stride, vp, v_stride, st));
}

int ds_vit_cache_attention_workspace_bytes(const ds_vit_cache* cache, const ds_vit_chunks* chunks, int32_t heads,
                                           size_t* bytes) {
  CacheView c;
  ChunkView b;
  if (!bytes) return DS_VIT_EINVAL;
  if (const int rc = check_cache(cache, chunks, 0, &c, &b)) return rc;
  if (heads < 1 || heads % c.kv_heads != 0 || heads / c.kv_heads > DS_VIT_CACHE_MAX_GROUP) return DS_VIT_EINVAL;
  *bytes = attention_workspace(b, cache->head_dim, heads / c.kv_heads, cache->kind == DS_VIT_CACHE_E4M3);
  return DS_VIT_OK;
}

int ds_vit_cache_attention(const ds_vit_cache* cache, const ds_vit_chunks* chunks, const void* q, int64_t q_stride,
                           int64_t rows, int32_t heads, float scale, int32_t window, int32_t sinks, void* out,
                           int64_t out_stride, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  AttentionArgs a{};
  if (const int rc = check_cache(cache, chunks, rows, &a.c, &a.b)) return rc;
  if (heads < 1 || heads % a.c.kv_heads != 0 || heads / a.c.kv_heads > DS_VIT_CACHE_MAX_GROUP || !(scale > 0.f) ||
      !(scale <= 1e30f) || window < 0 || sinks < 0)
    return DS_VIT_EINVAL;
  const int64_t width = static_cast<int64_t>(heads) * cache->head_dim;
  if (!status || !aligned(status, 4) || bad_rows(q, q_stride, width) || bad_rows(out, out_stride, width) || !ws ||
      !aligned(ws, 16))
    return DS_VIT_EINVAL;
  const bool e4m3 = cache->kind == DS_VIT_CACHE_E4M3;
  if (ws_bytes < attention_workspace(a.b, cache->head_dim, heads / a.c.kv_heads, e4m3)) return DS_VIT_ECAP;
  // Rows that share a K/V head are counted in 32 bits.
  if (rows > INT32_MAX / 2 / (heads / a.c.kv_heads)) return DS_VIT_ERANGE;
  if (rows == 0) return DS_VIT_OK;
  a.q = static_cast<const bf16*>(q);
  a.q_stride = q_stride;
  a.out = static_cast<bf16*>(out);
  a.out_stride = out_stride;
  a.heads = heads;
  a.group = heads / a.c.kv_heads;
  a.by_group = fast_div(a.group);
  a.window = window;
  a.sinks = sinks;
  a.scale_log2 = 1.4426950408889634f * scale;
  a.status = reinterpret_cast<int*>(status);
  auto* launch = few_rows(a.b, cache->head_dim, a.group, e4m3) ? launch_cache_decode : launch_cache_prefill;
  return launch(a, cache->head_dim, e4m3, ws, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
