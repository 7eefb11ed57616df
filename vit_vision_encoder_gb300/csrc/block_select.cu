// Bounds of the keys of a cache's pages and the choice of the blocks that each row
// attends to (include/dsvit.h, ds_vit_cache_bounds and ds_vit_cache_select).
//
// Bounds: each completed page is read once, by one warp a K/V head, 32 keys in flight; bound by memory and, at the
// sizes of a chunk, by the chain sequence -> table -> keys (13.9 MB of e4m3 pages: 7.4 to 8.2 us).  The grid has the blocks
// of the longest chunk for every sequence: one of 8192 rows in pages of 16 takes 6.3 us, beside 63 single tokens 41.  (At head
// dim 64 over bf16 pages the compiler spills 12 bytes.)
//
// Selection: scores are a product of the blocks' bounds [blocks, 2 D] with the rows' shared
// queries [2 D, rows].  Both operands are small whole numbers (|n| <= 1024, |H| <= 127) and so is every
// partial sum (2^24 at most): exact in fp16 products and fp32 sums, in any order, so equal inputs give equal lists.  Many
// rows (up to sixteen of one sequence and K/V head a CTA) go through warp MMAs, blocks in the place of M; the order of the
// 2 D terms is free, so a lane uses the 16 bytes that it loads where they lie.  A single row goes
// through 16-bit dot products, by a CTA or by the CTAs of a cluster, which put their scores into the
// first one's shared memory.  Scores stay in shared memory as whole numbers that order like them
// ("keys"); the threshold is searched among the few keys over a bound that follows from the largest keys of
// each lane, and among all keys where those are too many.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "cache.cuh"

namespace dsvit {

namespace {

// ------------------------------------------------------------------ bounds

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The least e >= -100 with a <= (1 + 126/128) 2^(e + shift), a the bf16 value of bits `bits` << 16.
__device__ __forceinline__ int least_exponent(uint32_t bits, int shift) {
  const int e = static_cast<int>(bits >> 7) - 127 - shift + ((bits & 127u) > 126u ? 1 : 0);
  return max(e, -100);
}
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }

struct BoundsArgs {
  CacheView c;
  ChunkView b;
  int8_t* hi_lo;
  uint8_t* exp;
  int* status;
};

constexpr int kBoundWarps = 8;

template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kBoundWarps) cache_bounds_kernel(const __grid_constant__ BoundsArgs a) {
  constexpr int kPer = E4M3 ? 16 : 8;                       // values in 16 bytes
  constexpr int kLanes = D / kPer, kKeys = 32 / kLanes;     // lanes of a key, keys of a load
  constexpr int kLoads = 32 / kKeys;                        // of 32 keys, in flight together
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, s = blockIdx.y;
  const Seq q = load_seq(a.b, a.c.page_shift, s, a.status);
  const int end = q.kv >> a.c.page_shift, page = 1 << a.c.page_shift;
  for (int j = (max(q.kv - q.c, 0) >> a.c.page_shift) + blockIdx.x; j < end; j += gridDim.x) {
    const int64_t at = page_of(a.b, a.c, s, j << a.c.page_shift, a.status);
    if (at < 0) continue;
    for (int head = threadIdx.x >> 5; head < a.c.kv_heads; head += kBoundWarps) {
      const int64_t row0 = cache_row(a.c, at, head, 0) + lane / kLanes;
      const uint4* from = reinterpret_cast<const uint4*>(a.c.k) + row0 * kLanes + lane % kLanes;
      float hi[kPer], lo[kPer];
#pragma unroll
      for (int x = 0; x < kPer; ++x) hi[x] = -INFINITY, lo[x] = INFINITY;
      for (int k0 = 0; k0 < page; k0 += 32) {
        uint4 u[kLoads];
        uint32_t byte[kLoads];
#pragma unroll
        for (int y = 0; y < kLoads; ++y) {
          if (y * kKeys >= 16 && page == 16) break;
          u[y] = from[(k0 + y * kKeys) * kLanes];
          byte[y] = E4M3 ? a.c.k_exp[row0 + k0 + y * kKeys] : 0u;
        }
#pragma unroll
        for (int y = 0; y < kLoads; ++y) {
          if (y * kKeys >= 16 && page == 16) break;
          const uint32_t w[4] = {u[y].x, u[y].y, u[y].z, u[y].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if constexpr (E4M3) {
              const float f = exp_factor(byte[y]);
              const float2 p = e4m3x2_to_float2(static_cast<uint16_t>(w[x])),
                           r = e4m3x2_to_float2(static_cast<uint16_t>(w[x] >> 16));
              const float v[4] = {p.x * f, p.y * f, r.x * f, r.y * f};
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                hi[4 * x + z] = max_nan(hi[4 * x + z], v[z]);
                lo[4 * x + z] = min_nan(lo[4 * x + z], v[z]);
              }
            } else {
              hi[2 * x] = max_nan(hi[2 * x], bf16lo(w[x]));
              lo[2 * x] = min_nan(lo[2 * x], bf16lo(w[x]));
              hi[2 * x + 1] = max_nan(hi[2 * x + 1], bf16hi(w[x]));
              lo[2 * x + 1] = min_nan(lo[2 * x + 1], bf16hi(w[x]));
            }
          }
        }
      }
      uint32_t top = 0;      // magnitudes order like their bits, infinities and NaN on top
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1) {
          hi[x] = max_nan(hi[x], __shfl_xor_sync(0xFFFFFFFFu, hi[x], o));
          lo[x] = min_nan(lo[x], __shfl_xor_sync(0xFFFFFFFFu, lo[x], o));
        }
        top = max(top, max(__float_as_uint(hi[x]) & 0x7FFFFFFFu, __float_as_uint(lo[x]) & 0x7FFFFFFFu));
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      const bool fine = top < 0x7F800000u;
      const int e = least_exponent(top >> 16, 6);
      const float f = power_of_two(-e);
      if (lane < kLanes) {
        int8_t* to = a.hi_lo + (at * a.c.kv_heads + head) * 2 * D + lane * kPer;
        uint32_t h[kPer / 4] = {}, l[kPer / 4] = {};
        // The products, too, are rounded outwards: one that lies under every float is not 0, or the bound would not
        // hold its key.
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
          if (!fine) continue;
          h[x / 4] |= (static_cast<uint32_t>(__float2int_ru(__fmul_ru(hi[x], f))) & 255u) << 8 * (x & 3);
          l[x / 4] |= (static_cast<uint32_t>(__float2int_rd(__fmul_rd(lo[x], f))) & 255u) << 8 * (x & 3);
        }
        if constexpr (E4M3) {
          *reinterpret_cast<uint4*>(to) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(to + D) = make_uint4(l[0], l[1], l[2], l[3]);
        } else {
          *reinterpret_cast<uint2*>(to) = make_uint2(h[0], h[1]);
          *reinterpret_cast<uint2*>(to + D) = make_uint2(l[0], l[1]);
        }
        if (lane == 0) a.exp[at * a.c.kv_heads + head] = static_cast<uint8_t>(fine ? e + 127 : 255);
      }
    }
  }
}

// ------------------------------------------------------------------ selection

struct SelectArgs {
  ChunkView b;
  int64_t n_pages;
  int kv_heads, page_shift;
  const int8_t* hi_lo;
  const uint8_t* exp;
  const bf16* q;
  int64_t q_stride;
  int group, log2_group;     // G of the header: 2^log2_group >= group
  int top, first, last;
  int32_t* blocks;
  int64_t row_stride, head_stride;
  int* status;
  int tile_rows;             // rows of a CTA
  int places;                // scores of a row in shared memory
};

constexpr int kSelectWarps = 8, kSelectThreads = 32 * kSelectWarps, kTileRows = 16;
constexpr uint32_t kForced = 0xFFFFFFFFu, kNotFinite = 0xFFFFFFFEu;   // above every score's number; 0: not a candidate

// A whole number that orders like the float x * by (finite: under kNotFinite, over 0; -0 like 0).
__device__ __forceinline__ uint32_t ordered(float x, float by) {
  const uint32_t u = __float_as_uint(fmaf(x, by, 0.f));
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// Two of four bytes (0 .. 255) as an fp16 pair in units of 2^-24, the least that fp16 has: the bytes themselves.
constexpr int kByteUnit = 24;
__device__ __forceinline__ uint32_t f16_of_bytes(uint32_t bytes, uint32_t which) { return __byte_perm(bytes, 0u, which); }

// Heads of one row and K/V head, D / 32 values of each in a lane: read whenever they are looked at, kAtOnce on their way
// together, or held.
template <int D, int kAtOnce>
struct RowHeads {
  const bf16* q;
  int group, lane;
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
#pragma unroll kAtOnce
    for (int h = 0; h < group; ++h) {
      uint32_t u[D / 64];
#pragma unroll
      for (int y = 0; y < D / 64; ++y) u[y] = __ldg(reinterpret_cast<const uint32_t*>(q + h * D) + lane * (D / 64) + y);
      f(u);
    }
  }
};
constexpr int kHeldHeads = 8;
template <int D>
struct HeldHeads {
  uint32_t u[kHeldHeads][D / 64];
  __device__ __forceinline__ void load(const bf16* q, int group, int lane) {
#pragma unroll
    for (int h = 0; h < kHeldHeads; ++h)
#pragma unroll
      for (int y = 0; y < D / 64; ++y)
        u[h][y] = h < group ? __ldg(reinterpret_cast<const uint32_t*>(q + h * D) + lane * (D / 64) + y) : 0u;
  }
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
#pragma unroll
    for (int h = 0; h < kHeldHeads; ++h) f(u[h]);
  }
};

// The shared query of one row: w[0 .. D - 1] sums of positive, w[D .. 2 D - 1] of negative parts, as
// fp16 or 16-bit whole numbers.  By one warp; returns the sum of them all.
template <int D, typename T, typename Heads>
__device__ __forceinline__ int shared_query(const SelectArgs& a, const Heads& heads, T* w, int lane) {
  constexpr int kPer = D / 32;
  uint32_t top = 0;
  heads.each([&](const uint32_t(&u)[D / 64]) {
#pragma unroll
    for (int y = 0; y < D / 64; ++y) top = max(top, max(u[y] << 16 & 0x7FFFFFFFu, u[y] & 0x7FFF0000u));
  });
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  // 1016 = (1 + 126/128) 2^9
  const int f = least_exponent(top >> 16, 9 - a.log2_group);
  const float by = power_of_two(-f / 2), rest = power_of_two(-f - -f / 2);     // 2^-f may be no float
  int up[kPer] = {}, down[kPer] = {};
  if (top < 0x7F800000u) {
    heads.each([&](const uint32_t(&u)[D / 64]) {
#pragma unroll
      for (int y = 0; y < kPer; ++y) {
        const int n = __float2int_rn((y & 1 ? bf16hi(u[y / 2]) : bf16lo(u[y / 2])) * by * rest);
        up[y] += max(n, 0);
        down[y] += min(n, 0);
      }
    });
  }
#pragma unroll
  for (int y = 0; y < kPer; ++y) {
    w[lane * kPer + y] = static_cast<T>(up[y]);
    w[D + lane * kPer + y] = static_cast<T>(down[y]);
  }
  int sum = 0;
#pragma unroll
  for (int y = 0; y < kPer; ++y) sum += up[y] + down[y];
  return __reduce_add_sync(0xFFFFFFFFu, sum);
}

// The list of one row from its n keys, by `kThreads` threads (a warp or the CTA); up to the next multiple
// of four the places behind them hold 0.  The threshold is known to be in [lo, hi]: at least `top` keys >= lo, fewer > hi,
// unless there are no more candidates than that.
template <int kThreads>
__device__ __forceinline__ void pick(const uint32_t* keys, int n, int top, int32_t* out, int (*sums)[kSelectWarps],
                                     uint32_t lo, uint32_t hi) {
  const int tid = threadIdx.x & (kThreads - 1), lane = threadIdx.x & 31, warp = tid >> 5;
  int turn = 0;
  auto count = [&](uint32_t from) {     // keys >= from
    int x = 0;
#pragma unroll 2
    for (int i = 4 * tid; i < n; i += 4 * kThreads) {
      const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
      x += (k.x >= from) + (k.y >= from) + (k.z >= from) + (k.w >= from);
    }
    x = __reduce_add_sync(0xFFFFFFFFu, x);
    if constexpr (kThreads > 32) {
      if (lane == 0) sums[turn][warp] = x;
      __syncthreads();
      x = 0;
#pragma unroll
      for (int y = 0; y < kSelectWarps; ++y) x += sums[turn][y];
      turn ^= 1;
    }
    return x;
  };
  // All keys over the threshold are taken, and the first `ties` of those equal to it.
  uint32_t over = 0;
  int ties = 0;
  if (count(1) > top) {
    bool fits = false;
    while (!fits && lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      const int x = count(mid);
      if (x >= top)
        lo = mid;
      else
        hi = mid - 1;
      fits = x == top;
    }
    over = fits ? lo - 1 : lo;
    ties = fits ? 0 : top - (lo == kForced ? 0 : count(lo + 1));
  }
  const auto lower = (1u << lane) - 1;
  // Each warp of the group has a run of blocks; what the warps before it take comes first.
  const int each = (n + kThreads - 1) / kThreads * 32, begin = min(n, warp * each), end = min(n, begin + each);
  int taken = 0, equal = 0;
  if constexpr (kThreads > 32) {
    int x = 0, e = 0;
    for (int i = begin + lane; i < end; i += 32) {
      x += keys[i] > over;
      e += keys[i] == over;
    }
    x = __reduce_add_sync(0xFFFFFFFFu, x);
    e = __reduce_add_sync(0xFFFFFFFFu, e);
    __syncthreads();                    // the counts' sums have been read
    if (lane == 0) sums[0][warp] = x, sums[1][warp] = e;
    __syncthreads();
    for (int y = 0; y < warp; ++y) {
      taken += sums[0][y];
      equal += sums[1][y];
    }
    taken += min(equal, ties);
  }
  for (int i0 = begin; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < end ? keys[i] : 0u;
    const uint32_t same = __ballot_sync(0xFFFFFFFFu, i < end && k == over);
    const bool on = i < end && (k > over || (k == over && equal + __popc(same & lower) < ties));
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, on);
    if (on) out[taken + __popc(all & lower)] = i;
    taken += __popc(all);
    equal += __popc(same);
  }
  if constexpr (kThreads > 32) {
    __syncthreads();
    if (warp == kSelectWarps - 1 && lane == 0) sums[0][0] = taken;
    __syncthreads();
    taken = sums[0][0];
  }
  for (int i = taken + tid; i < top; i += kThreads) out[i] = -1;
}

// Sorted over the lanes of a warp, the largest first.
__device__ __forceinline__ uint32_t sorted_down(uint32_t x, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size *= 2)
#pragma unroll
    for (int o = size / 2; o > 0; o /= 2) {
      const uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, x, o);
      const bool keep_max = ((lane & o) == 0) == ((lane & size) == 0);
      x = keep_max ? max(x, y) : min(x, y);
    }
  return x;
}

// The same by one warp where few blocks of many are looked for.  Each lane finds its own kTop-th largest key; the
// (need / kTop)-th largest of those is a bound that at least `need` keys reach and not many more do.  Those are listed,
// and held by the lanes, a few each, while the threshold is searched.  False, with nothing written, where too many
// reach it, with what is known of the threshold.  keys + n up to the next multiple of four are 0.  (8 thousand lists
// of 3750 blocks: 20 of them 255 us, 128 302; 129, which go to the search through all keys, 483, 1024 505.)
constexpr int kHeldMost = 8;
__host__ __device__ constexpr int held_by_lane(int top) { return top <= 32 ? 2 : kHeldMost; }
template <int kTop>
__device__ __forceinline__ bool pick_few(const uint32_t* keys, int n, const SelectArgs& a, int32_t* out, uint2* kept,
                                         uint32_t& lo, uint32_t& hi) {
  constexpr int kHeld = held_by_lane(32 * kTop), kKept = 32 * kHeld;
  const int lane = threadIdx.x & 31, top = a.top;
  uint32_t most[kTop] = {};             // the lane's largest keys, largest first, plus 1: forced ones are 0
#pragma unroll 2
  for (int i = 4 * lane; i < n; i += 128) {
    const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
    uint32_t x[4] = {k.x + 1, k.y + 1, k.z + 1, k.w + 1};
#pragma unroll
    for (int z = 0; z < 4; ++z)
#pragma unroll
      for (int y = 0; y < kTop; ++y) {
        const uint32_t up = max(most[y], x[z]);
        x[z] = min(most[y], x[z]);
        most[y] = up;
      }
  }
  // The forced ones are among the first and the last.
  const int firsts = min(a.first, n), lasts = min(a.last, n - firsts);
  int forced = 0;
  for (int i = lane; i < firsts + lasts; i += 32) forced += keys[i < firsts ? i : n - lasts + i - firsts] == kForced;
  forced = __reduce_add_sync(0xFFFFFFFFu, forced);
  const int need = top - forced;        // at most 32 kTop: the lists this is called for
  lo = hi = kForced;
  if (need > 0) {
    lo = max(__shfl_sync(0xFFFFFFFFu, sorted_down(most[kTop - 1], lane), (need + kTop - 1) / kTop - 1), 2u) - 1;
    hi = max(__reduce_max_sync(0xFFFFFFFFu, most[0]), 2u) - 1;
  }
  const auto lower = (1u << lane) - 1;
  int n_kept = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const uint32_t k = i0 + lane < n ? keys[i0 + lane] : 0u;
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, k >= lo);
    if (all == 0) continue;
    const int to = n_kept + __popc(all & lower);
    n_kept += __popc(all);
    if (n_kept > kKept) return false;
    if (k >= lo) kept[to] = make_uint2(k, static_cast<uint32_t>(i0 + lane));
  }
  __syncwarp();
  uint32_t held[kHeld];
#pragma unroll
  for (int y = 0; y < kHeld; ++y) held[y] = 32 * y + lane < n_kept ? kept[32 * y + lane].x : 0u;
  auto count = [&](uint32_t from) {
    int x = 0;
#pragma unroll
    for (int y = 0; y < kHeld; ++y)
      if (32 * y < n_kept) x += held[y] >= from;
    return static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, x));
  };
  // The threshold is in [lo, hi]: at least `top` keys >= lo, fewer > hi (or all are taken).
  bool fits = n_kept <= top;
  while (!fits && lo < hi) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    const int x = count(mid);
    if (x >= top)
      lo = mid;
    else
      hi = mid - 1;
    fits = x == top;
  }
  const int ties = fits || lo == kForced ? top : top - count(lo + 1);       // of the keys equal to lo, in order
  int taken = 0, same = 0;
#pragma unroll
  for (int y = 0; y < kHeld; ++y) {
    if (32 * y >= n_kept) break;
    const uint32_t equal = __ballot_sync(0xFFFFFFFFu, held[y] == lo);
    const bool on = held[y] > lo || (held[y] == lo && same + __popc(equal & lower) < ties);
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, on);
    if (on) out[taken + __popc(all & lower)] = static_cast<int32_t>(kept[32 * y + lane].y);
    taken += __popc(all);
    same += __popc(equal);
  }
  for (int i = taken + lane; i < top; i += 32) out[i] = -1;
  return true;
}

// The same by the CTA.  The least of the warps' (top / 8)-th largest lane maxima (keys dealt to all lanes in
// turn) is a bound that at least `top` keys reach.  Those are listed and held, up to kEach a thread.
constexpr int kEach = 4, kListed = kEach * kSelectThreads;
__device__ __forceinline__ bool pick_some(const uint32_t* keys, int n, int top, int32_t* out, int (*sums)[kSelectWarps],
                                          uint4* of_warps, uint2* listed, uint32_t& lo, uint32_t& hi) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const auto lower = (1u << lane) - 1;
  const int rank = (top + kSelectWarps - 1) / kSelectWarps;
  lo = 1;
  hi = kForced;
  if (rank > 32) return false;
  uint32_t most = 0;                    // largest key of the lane's that is not forced
  int forced = 0, some = 0;
#pragma unroll 4
  for (int i = tid; i < n; i += kSelectThreads) {
    const uint32_t k = keys[i];
    forced += k == kForced;
    some += k != 0;
    most = max(most, k == kForced ? 0u : k);
  }
  forced = __reduce_add_sync(0xFFFFFFFFu, forced);
  some = __reduce_add_sync(0xFFFFFFFFu, some);
  const uint32_t largest = __reduce_max_sync(0xFFFFFFFFu, most);
  const uint32_t at_rank = __shfl_sync(0xFFFFFFFFu, sorted_down(most, lane), rank - 1);
  if (lane == 0) of_warps[warp] = make_uint4(forced, some, largest, at_rank);
  __syncthreads();
  uint32_t least = kForced, largest_of_all = 0;
  forced = some = 0;
#pragma unroll
  for (int y = 0; y < kSelectWarps; ++y) {
    const uint4 v = of_warps[y];
    forced += v.x;
    some += v.y;
    largest_of_all = max(largest_of_all, v.z);
    least = min(least, v.w);
  }
  if (some <= top) return false;
  lo = forced == top ? kForced : max(least, 1u);
  hi = forced == top ? kForced : largest_of_all;
  // Listed in order: each warp has a run of blocks.
  const int each = (n + kSelectThreads - 1) / kSelectThreads * 32, begin = min(n, warp * each), end = min(n, begin + each);
  int mine = 0;
  for (int i0 = begin; i0 < end; i0 += 32)
    mine += __popc(__ballot_sync(0xFFFFFFFFu, i0 + lane < end && keys[i0 + lane] >= lo));
  if (lane == 0) sums[0][warp] = mine;
  __syncthreads();
  int total = 0, to = 0;
#pragma unroll
  for (int y = 0; y < kSelectWarps; ++y) {
    to += y < warp ? sums[0][y] : 0;
    total += sums[0][y];
  }
  __syncthreads();                      // the sums have been read
  if (total > kListed) return false;
  for (int i0 = begin; i0 < end; i0 += 32) {
    const uint32_t k = i0 + lane < end ? keys[i0 + lane] : 0u;
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, k >= lo);
    if (k >= lo) listed[to + __popc(all & lower)] = make_uint2(k, static_cast<uint32_t>(i0 + lane));
    to += __popc(all);
  }
  __syncthreads();
  // Thread i holds listed key i, which a barrier counts, or keys 4i .. 4i + 3.
  const int per = total <= kSelectThreads ? 1 : kEach;
  uint32_t held[kEach], block[kEach];
#pragma unroll
  for (int y = 0; y < kEach; ++y) {
    const uint2 v = y < per && per * tid + y < total ? listed[per * tid + y] : make_uint2(0, 0);
    held[y] = v.x;
    block[y] = v.y;
  }
  int turn = 0;
  auto count = [&](uint32_t from) {
    if (per == 1) return __syncthreads_count(held[0] >= from);
    int x = 0;
#pragma unroll
    for (int y = 0; y < kEach; ++y) x += held[y] >= from;
    x = __reduce_add_sync(0xFFFFFFFFu, x);
    if (lane == 0) sums[turn][warp] = x;
    __syncthreads();
    const int4 a = *reinterpret_cast<const int4*>(sums[turn]), b = *reinterpret_cast<const int4*>(sums[turn] + 4);
    turn ^= 1;
    return a.x + a.y + a.z + a.w + b.x + b.y + b.z + b.w;
  };
  // The threshold is in [lo, hi]: at least `top` keys >= lo, fewer > hi.
  bool fits = total == top;
  while (!fits && lo < hi) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    const int x = count(mid);
    if (x >= top)
      lo = mid;
    else
      hi = mid - 1;
    fits = x == top;
  }
  const int ties = fits || lo == kForced ? top : top - count(lo + 1);       // of the keys equal to lo, in order
  // What comes before this thread's keys: over the threshold in the upper half, equal to it in the lower one.
  uint32_t here = 0;
#pragma unroll
  for (int y = 0; y < kEach; ++y) here += (held[y] > lo ? 0x10000u : 0u) + (held[y] == lo && held[y] != 0 ? 1u : 0u);
  uint32_t upto = here;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) sums[turn][warp] = static_cast<int>(upto);
  __syncthreads();
  uint32_t before = upto - here;
  for (int y = 0; y < warp; ++y) before += static_cast<uint32_t>(sums[turn][y]);
  int over = static_cast<int>(before >> 16), same = static_cast<int>(before & 0xFFFFu);
#pragma unroll
  for (int y = 0; y < kEach; ++y) {
    const bool is_over = held[y] > lo, is_same = held[y] == lo && held[y] != 0;
    if (is_over || (is_same && same < ties)) out[over + min(same, ties)] = static_cast<int32_t>(block[y]);
    over += is_over;
    same += is_same;
  }
  return true;
}

// What a lane has of 16 blocks from k0 on, but for their bounds: pages and exponents of blocks g and g + 8.
struct BoundPages {
  int32_t at[2];                        // below 0: no block here
  uint32_t byte[2];
  // The key of block k0 + g + 8 y for a row whose own block is `own`, from the whole number `score`, in units of 2^-kUnit.
  template <int kUnit>
  __device__ __forceinline__ uint32_t key(const SelectArgs& a, int y, int k, int own, float score) const {
    if (k > own || at[y] < 0) return 0;
    if (k < a.first || k > own - a.last) return kForced;
    return byte[y] == 255u ? kNotFinite : ordered(score, factor<kUnit>(y));
  }
  // 2^(e - 20): every score is a float.
  template <int kUnit>
  __device__ __forceinline__ float factor(int y) const {
    return power_of_two(max(static_cast<int>(byte[y]), 21) - 147 + kUnit);
  }
};

// And their bounds, pieces t, t + 4, ... of 16 bytes.
template <int D>
struct BoundTile : BoundPages {
  uint4 u[2][D / 32];
  __device__ __forceinline__ void load(const SelectArgs& a, int head, int t) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      if (at[y] >= a.n_pages) {
        report_error(a.status, DS_VIT_ERANGE);
        at[y] = -1;
      }
      const int64_t row = static_cast<int64_t>(max(at[y], 0)) * a.kv_heads + head;
      const uint4* from = reinterpret_cast<const uint4*>(a.hi_lo + row * 2 * D) + t;
      byte[y] = __ldg(a.exp + row);
#pragma unroll
      for (int j = 0; j < D / 32; ++j) u[y][j] = __ldg(from + 4 * j);
    }
  }
};

__device__ __forceinline__ int32_t page_entry(const int32_t* table, int k, int blocks) {
  return k < blocks ? __ldg(table + k) : -1;
}

// Up to sixteen rows of one sequence at a time, for one K/V head.  Bound by instructions and what they wait for: a
// quarter picks, the rest widens the bounds, multiplies, makes keys and shares queries.  Bytes go into the products as they are
// but for their sign (b + 128 in units of 2^-24), and the sums begin at -128 times that of w: whole
// numbers of at most 2^24 in any order, 127 |w| of the terms that are in and 128 |w| of the others.  2048 rows of 8
// heads over 532 blocks: 54 us, over 938 blocks (1024 rows) 48; 56 and 60 with bytes widened to fp16 by a subtraction, four CTAs
// an SM (64 registers) and each round's bounds loaded when it begins.  Thirty-two rows a CTA, with eight to
// sixteen warps: 54 to 57 and 53 to 56.  At head dim 128 the third CTA an SM costs 16 bytes
// of spills.
template <int D>
__global__ void __launch_bounds__(kSelectThreads, D == 128 ? 3 : 4) cache_select_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int kSteps = 2 * D / 64;                // 16-byte pieces of a block that a lane has, four MMAs each
  constexpr int kStep = 16 * kSelectWarps;
  extern __shared__ uint4 dynamic[];
  uint32_t* const keys = reinterpret_cast<uint32_t*>(dynamic);
  __shared__ __align__(16) __half w[kTileRows][2 * D + 8];
  __shared__ __align__(8) float bias[kTileRows];    // -128 times the sum of w
  uint2* const kept = reinterpret_cast<uint2*>(keys + a.tile_rows * a.places) + (threadIdx.x >> 5) * 32 * held_by_lane(a.top);
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int tile = static_cast<int>(blockIdx.x), head = tile % a.kv_heads;
  const int r_end = min(a.b.rows, (tile / a.kv_heads + 1) * a.tile_rows);
  const bf16* const queries = a.q + static_cast<int64_t>(head) * a.group * D;
  // The rows of one sequence after another.
  for (int ra = tile / a.kv_heads * a.tile_rows; ra < r_end;) {
    // Queries are on their way while the sequence is looked up, and the first pages' numbers while they are shared.
    constexpr int kOwn = (kTileRows + kSelectWarps - 1) / kSelectWarps;
    HeldHeads<D> held;
    auto hold = [&](int row) {
      held.load(queries + row * a.q_stride, row < r_end && a.group <= kHeldHeads ? a.group : 0, lane);
    };
    hold(ra + warp);
    const int s = find_seq(a.b, ra, lane);
    const Seq q = s < 0 ? Seq{0, 0, 0} : load_seq(a.b, a.page_shift, s, a.status);
    if (static_cast<unsigned>(ra - q.row0) >= static_cast<unsigned>(q.c)) {     // of no sequence, or refused
      ++ra;
      continue;
    }
    const int n_rows = min(r_end, q.row0 + q.c) - ra;
    const int p0 = q.kv - q.c + ra - q.row0;        // position of the first
    const int blocks = max(p0 + n_rows - 1 + (1 << a.page_shift), 0) >> a.page_shift;     // of the last
    const int32_t* table = a.b.table + static_cast<int64_t>(s) * a.b.table_cols;
    BoundTile<D> b;
    int32_t ahead[2];                               // the pages of the blocks after them
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      b.at[y] = page_entry(table, 16 * warp + g + 8 * y, blocks);
      ahead[y] = page_entry(table, 16 * warp + kStep + g + 8 * y, blocks);
    }
#pragma unroll
    for (int y = 0; y < kOwn; ++y) {
      const int i = warp + y * kSelectWarps;
      if (i >= n_rows) {
        if (i >= kTileRows) break;
        for (int x = lane; x < 2 * D; x += 32) w[i][x] = __half(0.f);
        continue;
      }
      const int sum = a.group <= kHeldHeads
                          ? shared_query<D>(a, held, w[i], lane)
                          : shared_query<D>(a, RowHeads<D, 8>{queries + static_cast<int64_t>(ra + i) * a.q_stride, a.group, lane}, w[i], lane);
      if (lane == 0) bias[i] = static_cast<float>(-128 * sum) * power_of_two(-kByteUnit);
      if (y + 1 < kOwn) hold(ra + i + kSelectWarps);
    }
    if (16 * warp < blocks) b.load(a, head, t);
    __syncthreads();
    for (int k0 = 16 * warp; k0 < blocks; k0 += kStep) {
      float c[kTileRows / 8][4];
#pragma unroll
      for (int z = 0; z < kTileRows / 8; ++z) {
        const float2 from = *reinterpret_cast<const float2*>(&bias[8 * z + 2 * t]);
        c[z][0] = c[z][2] = from.x;
        c[z][1] = c[z][3] = from.y;
      }
      auto products = [&](auto groups) {
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          const uint32_t b0[4] = {b.u[0][j].x, b.u[0][j].y, b.u[0][j].z, b.u[0][j].w};
          const uint32_t b1[4] = {b.u[1][j].x, b.u[1][j].y, b.u[1][j].z, b.u[1][j].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t v0 = b0[x] ^ 0x80808080u, v1 = b1[x] ^ 0x80808080u;
            const uint32_t m[4] = {f16_of_bytes(v0, 0x4140u), f16_of_bytes(v1, 0x4140u), f16_of_bytes(v0, 0x4342u),
                                   f16_of_bytes(v1, 0x4342u)};
            // The terms of rows g, g + 8, ... that go with the lane's piece of a block.
#pragma unroll
            for (int z = 0; z < decltype(groups)::value; ++z) {
              const uint2 wz = *reinterpret_cast<const uint2*>(&w[8 * z + g][64 * j + 16 * t + 4 * x]);
              mma_f16(c[z], m, wz.x, wz.y);
            }
          }
        }
      };
      if (n_rows > 8)
        products(std::integral_constant<int, kTileRows / 8>{});
      else
        products(std::integral_constant<int, 1>{});
      // The next bounds come while these scores become keys.
      const BoundPages here = b;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        b.at[y] = ahead[y];
        ahead[y] = page_entry(table, k0 + 2 * kStep + g + 8 * y, blocks);
      }
      if (k0 + kStep < blocks) b.load(a, head, t);
      // Blocks between all rows' forced ones, with pages and scores.
      const bool plain = n_rows % 8 == 0 && k0 >= a.first && k0 + 15 <= (p0 >> a.page_shift) - a.last &&
                         __all_sync(0xFFFFFFFFu, min(here.at[0], here.at[1]) >= 0 && max(here.byte[0], here.byte[1]) < 255u);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int k = k0 + g + 8 * y;
        const float factor = here.factor<kByteUnit>(y);
#pragma unroll
        for (int z = 0; z < kTileRows / 8; ++z) {
          if (8 * z >= n_rows) break;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int i = 2 * t + x + 8 * z;      // row
            if (plain)
              keys[i * a.places + k] = ordered(c[z][2 * y + x], factor);
            else if (i < n_rows && k < blocks)
              keys[i * a.places + k] = here.key<kByteUnit>(a, y, k, (p0 + i) >> a.page_shift, c[z][2 * y + x]);
          }
        }
      }
    }
    for (int i = warp; i < n_rows; i += kSelectWarps)
      if (blocks + lane < (blocks + 3) / 4 * 4) keys[i * a.places + blocks + lane] = 0;
    __syncthreads();
    for (int i = warp; i < n_rows; i += kSelectWarps) {
      const uint32_t* const mine = keys + i * a.places;
      int32_t* const out = a.blocks + static_cast<int64_t>(ra + i) * a.row_stride + head * a.head_stride;
      uint32_t lo = 1, hi = kForced;
      const int n = max(p0 + i + (1 << a.page_shift), 0) >> a.page_shift;       // blocks of this row
      const bool few = a.top <= 32 ? pick_few<1>(mine, n, a, out, kept, lo, hi)
                                   : a.top <= 128 && pick_few<6>(mine, n, a, out, kept, lo, hi);
      if (!few) pick<32>(mine, n, a.top, out, nullptr, lo, hi);
    }
    __syncthreads();
    ra += n_rows;
  }
}

// One row and K/V head, by a CTA or the CTAs of a cluster.  A row would leave seven eighths of an MMA empty: the
// products are 16-bit weights times the bytes, two at a time.  Bound by latency (row -> sequence -> table -> bounds,
// 3.6 us to the first score of 48 rows; then 2 us for every 128 blocks), so the first blocks' bounds are on their way while the query
// is made, and three CTAs an SM count for more than loads a round ahead (17 us; 20 with the
// next blocks' bounds in registers and two CTAs).  Two CTAs a row are slower where the rows fill
// the SMs (21 us): what comes before the first score is done twice.
template <int D>
__global__ void __launch_bounds__(kSelectThreads, 3) cache_select_row_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int kSteps = 2 * D / 64;
  extern __shared__ uint4 dynamic[];
  uint32_t* const keys = reinterpret_cast<uint32_t*>(dynamic);
  __shared__ __align__(16) int16_t w[2 * D];
  __shared__ __align__(16) int sums[2][kSelectWarps];
  __shared__ uint4 of_warps[kSelectWarps];
  __shared__ uint2 listed[kListed];
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(cluster_rank());
  uint32_t ranks;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  if (ranks > 1) cluster_arrive();
  const int64_t tile = blockIdx.x / ranks, row = tile / a.kv_heads;
  const int head = static_cast<int>(tile - row * a.kv_heads);
  if (warp == kSelectWarps - 1)
    shared_query<D>(a, RowHeads<D, 4>{a.q + row * a.q_stride + static_cast<int64_t>(head) * a.group * D, a.group, lane}, w, lane);
  const int s = find_seq(a.b, static_cast<int>(row), lane);
  const Seq q = s < 0 ? Seq{0, 0, 0} : load_seq(a.b, a.page_shift, s, a.status);
  const bool mine = static_cast<unsigned>(row - q.row0) < static_cast<unsigned>(q.c);     // else of no sequence, or refused
  const int p = q.kv - q.c + static_cast<int>(row - q.row0), own = p >> a.page_shift, blocks = mine ? max(own + 1, 0) : 0;
  const int32_t* table = a.b.table + static_cast<int64_t>(max(s, 0)) * a.b.table_cols;
  const int step = 16 * kSelectWarps * static_cast<int>(ranks);
  int k0 = 16 * (warp * static_cast<int>(ranks) + rank);
  BoundTile<D> b;
  int32_t next[2];                                  // the pages of the blocks after them
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    b.at[y] = page_entry(table, k0 + g + 8 * y, blocks);
    next[y] = page_entry(table, k0 + step + g + 8 * y, blocks);
  }
  if (k0 < blocks) b.load(a, head, t);
  if (ranks > 1) cluster_wait();                    // the first CTA's shared memory is there
  __syncthreads();
  for (; k0 < blocks; k0 += step) {
    int32_t ahead[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) ahead[y] = page_entry(table, k0 + 2 * step + g + 8 * y, blocks);
    int c[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const uint4* from = reinterpret_cast<const uint4*>(w + 64 * j + 16 * t);
      const uint4 w0 = from[0], w1 = from[1];
      const uint32_t wx[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t v[4] = {b.u[y][j].x, b.u[y][j].y, b.u[y][j].z, b.u[y][j].w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          c[y] = __dp2a_lo(static_cast<int>(wx[2 * x]), static_cast<int>(v[x]), c[y]);
          c[y] = __dp2a_hi(static_cast<int>(wx[2 * x + 1]), static_cast<int>(v[x]), c[y]);
        }
      }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      c[y] += __shfl_xor_sync(0xFFFFFFFFu, c[y], 1);
      c[y] += __shfl_xor_sync(0xFFFFFFFFu, c[y], 2);
      const int k = k0 + g + 8 * y;
      const uint32_t key = b.template key<0>(a, y, k, own, static_cast<float>(c[y]));
      if (t != 0 || k >= blocks) continue;
      if (ranks > 1) {
        const uint32_t to = mapa_shared(smem_u32(keys + k), 0);
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(key) : "memory");
      } else {
        keys[k] = key;
      }
    }
    b.at[0] = next[0], b.at[1] = next[1];
    if (k0 + step < blocks) b.load(a, head, t);
    next[0] = ahead[0], next[1] = ahead[1];
  }
  if (rank == 0 && blocks + static_cast<int>(threadIdx.x) < (blocks + 3) / 4 * 4) keys[blocks + threadIdx.x] = 0;
  if (ranks > 1)
    cluster_sync();
  else
    __syncthreads();
  if (rank != 0 || !mine) return;
  int32_t* const out = a.blocks + row * a.row_stride + head * a.head_stride;
  uint32_t lo, hi;
  if (!pick_some(keys, blocks, a.top, out, sums, of_warps, listed, lo, hi))
    pick<kSelectThreads>(keys, blocks, a.top, out, sums, lo, hi);
}

constexpr int kSelectKeyBytes = 200 * 1024;      // of shared memory, for scores
constexpr int kSharedOfSm = 228 * 1024, kSharedOfCta = 1024;      // there is; what the system takes of it for every CTA
constexpr int kept_bytes(int top) { return 8 * kSelectThreads * held_by_lane(top); }      // keys that are held while a list is picked
static_assert(4 * (DS_VIT_SELECT_MAX_COLS + 4) <= kSelectKeyBytes, "one row's scores");

bool bad_bounds(const ds_vit_key_bounds* b) { return !b || !b->hi_lo || !aligned(b->hi_lo, 16) || !b->exp; }

}  // namespace

}  // namespace dsvit

using namespace dsvit;

extern "C" {

int ds_vit_cache_bounds(const ds_vit_cache* cache, const ds_vit_chunks* chunks, const ds_vit_key_bounds* bounds,
                        int64_t rows, int32_t* status, void* stream) {
  BoundsArgs a{};
  if (const int rc = check_cache(cache, chunks, rows, &a.c, &a.b)) return rc;
  if (bad_bounds(bounds) || !status || !aligned(status, 4)) return DS_VIT_EINVAL;
  if (rows == 0) return DS_VIT_OK;
  a.hi_lo = bounds->hi_lo;
  a.exp = bounds->exp;
  a.status = reinterpret_cast<int*>(status);
  const int64_t most = (std::min<int64_t>(rows, chunks->max_rows) + cache->page - 1) / cache->page;   // of a sequence
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(most, 4096)), static_cast<unsigned>(chunks->n));
  const bool e4m3 = cache->kind == DS_VIT_CACHE_E4M3;
  auto* fn = cache->head_dim == 128 ? (e4m3 ? cache_bounds_kernel<128, true> : cache_bounds_kernel<128, false>)
                                    : (e4m3 ? cache_bounds_kernel<64, true> : cache_bounds_kernel<64, false>);
  return launched(launch_pdl(fn, grid, dim3(32 * kBoundWarps), 0, static_cast<cudaStream_t>(stream), a));
}

int ds_vit_cache_select(const ds_vit_cache* cache, const ds_vit_chunks* chunks, const ds_vit_key_bounds* bounds,
                        const void* q, int64_t q_stride, int64_t rows, int32_t heads, int32_t top, int32_t first,
                        int32_t last, int32_t* blocks, int64_t row_stride, int64_t head_stride, int32_t* status,
                        void* stream) {
  CacheView c;
  SelectArgs a{};
  if (const int rc = check_cache(cache, chunks, rows, &c, &a.b)) return rc;
  if (bad_bounds(bounds) || !status || !aligned(status, 4) || heads < 1 || heads % c.kv_heads != 0 ||
      heads / c.kv_heads > DS_VIT_CACHE_MAX_GROUP ||
      bad_rows(q, q_stride, static_cast<int64_t>(heads) * cache->head_dim) || first < 0 || last < 1 ||
      top > DS_VIT_SELECT_MAX_TOP || static_cast<int64_t>(first) + last > top ||
      bad_lists(blocks, row_stride, head_stride, rows, c.kv_heads, top))
    return DS_VIT_EINVAL;
  if (chunks->table_cols > DS_VIT_SELECT_MAX_COLS || rows > INT32_MAX / c.kv_heads) return DS_VIT_ERANGE;
  if (rows == 0) return DS_VIT_OK;
  a.n_pages = c.n_pages;
  a.kv_heads = c.kv_heads;
  a.page_shift = c.page_shift;
  a.hi_lo = bounds->hi_lo;
  a.exp = bounds->exp;
  a.q = static_cast<const bf16*>(q);
  a.q_stride = q_stride;
  a.group = heads / c.kv_heads;
  while (1 << a.log2_group < a.group) ++a.log2_group;
  a.top = top;
  a.first = first;
  a.last = last;
  a.blocks = blocks;
  a.row_stride = row_stride;
  a.head_stride = head_stride;
  a.status = reinterpret_cast<int*>(status);
  a.places = (chunks->table_cols + 31) / 32 * 32 + 4;
  // Rows of one sequence share the loads of its bounds where there are more than enough CTAs.
  const int64_t units = rows * c.kv_heads;
  const bool single = chunks->max_rows < 8 || units <= 4 * static_cast<int64_t>(num_sms()) || 8 * a.places > kSelectKeyBytes;
  // 64 sequences over 8000 to 60000 tokens, by single rows and by tiles: 2 rows each 32 and 90 us, 4 rows 52 and 49, 7 rows
  // 82 and 47.  A tile takes the sequences that its rows belong to one behind the other, and the choice is the call's: 60
  // single tokens beside a chunk of 1024 rows take 193 us, in a call of their own 19 (the chunk 41).
  a.tile_rows = 1;
  if (!single) {
    // Sixteen rows where two CTAs fit an SM (938 blocks: 16 rows 48 us, 8 rows 52; 1907 blocks: 139 and 112; lists of 64,
    // which take more to pick: 1400 blocks 76 and 81, 1450 blocks, where one CTA fits, 118 and 85), else eight as long as
    // one fits (3750 blocks: 8 rows 257 us, 4 rows 310).
    const int64_t fixed = 2 * kTileRows * (2 * cache->head_dim + 8) + 4 * kTileRows + kept_bytes(top) + kSharedOfCta;
    a.tile_rows = 2 * (4 * kTileRows * static_cast<int64_t>(a.places) + fixed) <= kSharedOfSm ? kTileRows : kTileRows / 2;
    while (4 * static_cast<int64_t>(a.tile_rows) * a.places > kSelectKeyBytes) a.tile_rows /= 2;
  }
  int ranks = 1;
  if (single)
    while (ranks < 8 && 2 * ranks * units <= 2 * static_cast<int64_t>(num_sms()) &&
           2 * ranks * 16 * kSelectWarps <= chunks->table_cols)
      ranks *= 2;
  const int bytes = 4 * a.tile_rows * a.places + (single ? 0 : kept_bytes(top));
  auto* fn = cache->head_dim == 128 ? (single ? cache_select_row_kernel<128> : cache_select_kernel<128>)
                                    : (single ? cache_select_row_kernel<64> : cache_select_kernel<64>);
  if (allow_smem(reinterpret_cast<const void*>(fn), kSelectKeyBytes + kept_bytes(DS_VIT_SELECT_MAX_TOP)) != cudaSuccess) return DS_VIT_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + a.tile_rows - 1) / a.tile_rows * c.kv_heads * ranks));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  return launched(cudaLaunchKernelEx(&cfg, fn, a));
}

}  // extern "C"
