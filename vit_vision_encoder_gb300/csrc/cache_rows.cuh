// Pieces shared by the attention kernels over the paged cache: the plan of a
// call's work, the records of results that several workers share, and the
// row computed key by key.
#pragma once

#include "cache.cuh"

namespace dsvit {

__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u; }

// A lane's D / 32 values of a row of keys (from c.k, its exponent from c.k_exp) or values.
template <int D, bool E4M3>
__device__ __forceinline__ void load_row(const uint8_t* held, const uint8_t* exps, int64_t row, int lane,
                                         float (&x)[D / 32]) {
  constexpr int kPer = D / 32;
  const int64_t at = row * D + lane * kPer;
  if constexpr (E4M3) {
    const float f = exp_factor(exps[row]);
#pragma unroll
    for (int y = 0; y < kPer; y += 2) {
      const float2 two = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(held + at + y));
      x[y] = two.x * f;
      x[y + 1] = two.y * f;
    }
  } else {
#pragma unroll
    for (int y = 0; y < kPer; y += 2) {
      const uint32_t two = *reinterpret_cast<const uint32_t*>(held + 2 * (at + y));
      x[y] = bf16lo(two);
      x[y + 1] = bf16hi(two);
    }
  }
}

// The matrix products give a hidden key the weight 0, and 0 times an infinity or NaN in its
// value is NaN.  Where rows of an item (positions p0 .. p1) see different keys and the
// result of the one at p is not finite: whether that may come from such a value, one
// that the item sees and the row does not.  By one warp.
template <int D, bool E4M3>
__device__ __forceinline__ bool hidden_not_finite(const AttentionArgs& a, int s, int kv_head, int p, int p0, int p1, int lane) {
  constexpr int kKeys = 2;
  bool bad = false;
  auto look = [&](int from, int to) {        // keys from .. to - 1
    for (int j = from; j < to; j += kKeys) {
      float v[kKeys][D / 32];
#pragma unroll
      for (int y = 0; y < kKeys; ++y) {
        const int64_t page = j + y < to ? page_of(a.b, a.c, s, j + y, a.status) : -1;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) v[y][x] = 0.f;
        if (page >= 0) load_row<D, E4M3>(a.c.v, a.c.v_exp, cache_row(a.c, page, kv_head, j + y), lane, v[y]);
      }
#pragma unroll
      for (int y = 0; y < kKeys; ++y)
#pragma unroll
        for (int x = 0; x < D / 32; ++x) bad |= not_finite(v[y][x]);
    }
  };
  look(p + 1, p1 + 1);
  look(max(window_start(a, p0), a.sinks), window_start(a, p));
  return __any_sync(0xFFFFFFFFu, bad);
}

// One row of the result from the keys that it does see, by one warp, two keys at a time.
template <int D, bool E4M3>
__device__ __forceinline__ void exact_row(const AttentionArgs& a, int s, int row0, int p, int i, int h, int lane) {
  constexpr int kPer = D / 32, kKeys = 2;
  const bf16* qr = a.q + (row0 + i) * a.q_stride + h * D + lane * kPer;
  float q[kPer], o[kPer];
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    q[x] = __bfloat162float(qr[x]);
    o[x] = 0.f;
  }
  const int lo = window_start(a, p), kv_head = h / a.group;
  float m = -INFINITY, l = 0.f;
  for (int j0 = 0; j0 <= p; j0 += kKeys) {
    if (j0 >= a.sinks && j0 + kKeys <= lo) j0 = lo & ~(kKeys - 1);
    const int64_t page = page_of(a.b, a.c, s, j0, a.status);      // a block lies in one page
    if (page < 0) return;
    const int64_t row = cache_row(a.c, page, kv_head, j0);
    float z[kKeys], v[kKeys][kPer];
    auto on = [&](int y) { return sees(a, p, j0 + y); };
#pragma unroll
    for (int y = 0; y < kKeys; ++y) {
      z[y] = 0.f;
      if (on(y)) {
        float k[kPer];
        load_row<D, E4M3>(a.c.k, a.c.k_exp, row + y, lane, k);
        load_row<D, E4M3>(a.c.v, a.c.v_exp, row + y, lane, v[y]);
#pragma unroll
        for (int x = 0; x < kPer; ++x) z[y] = fmaf(q[x], k[x], z[y]);
      }
    }
    float m_new = m;
#pragma unroll
    for (int y = 0; y < kKeys; ++y) {
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) z[y] += __shfl_xor_sync(0xFFFFFFFFu, z[y], x);
      z[y] *= a.scale_log2;
      if (on(y)) m_new = fmaxf(m_new, z[y]);
    }
    const float alpha = m == m_new ? 1.f : exp2f(m - m_new);
    l *= alpha;
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] *= alpha;
#pragma unroll
    for (int y = 0; y < kKeys; ++y) {
      if (!on(y)) continue;
      // A score of -inf weighs nothing, also while there is no other (NaN stays NaN).
      const float w = z[y] == -INFINITY ? 0.f : exp2f(z[y] - m_new);
      l += w;
#pragma unroll
      for (int x = 0; x < kPer; ++x) o[x] = fmaf(w, v[y][x], o[x]);
    }
    m = m_new;
    // Nothing more to find out: the row does see what makes it NaN throughout.
    bool lost = true;
#pragma unroll
    for (int x = 0; x < kPer; ++x) lost &= o[x] != o[x];
    if (__all_sync(0xFFFFFFFFu, lost)) break;
  }
  bf16* to = a.out + (row0 + i) * a.out_stride + h * D + lane * kPer;
#pragma unroll
  for (int x = 0; x < kPer; ++x) to[x] = __float2bfloat16_rn(o[x] / l);
}

// The row at p of an item (positions p0 .. p1) again, if its result is not finite because of
// a value that it does not see.  Long caches take their time (0.7 us a key), so this is
// done where nobody waits for the warp with a limit.  Out of line, and two keys at a time,
// for the registers of the kernels that call it (with four, every call of few rows took
// 2 us more).
template <int D, bool E4M3>
__device__ __noinline__ void mend_row(const AttentionArgs& a, int s, int row0, int p, int i, int h, int p0, int p1,
                                      int lane) {
  if (hidden_not_finite<D, E4M3>(a, s, h / a.group, p, p0, p1, lane)) exact_row<D, E4M3>(a, s, row0, p, i, h, lane);
}

// Whether a row of the output, written before, is not finite.
template <int D>
__device__ __forceinline__ bool row_not_finite(const AttentionArgs& a, int64_t row, int h, int lane) {
  const uint32_t* at = reinterpret_cast<const uint32_t*>(a.out + row * a.out_stride + h * D) + lane * (D / 64);
  bool bad = false;
#pragma unroll
  for (int x = 0; x < D / 64; ++x) bad |= not_finite(bf16lo(at[x])) || not_finite(bf16hi(at[x]));
  return __any_sync(0xFFFFFFFFu, bad);
}

// e4m3: the range of a softmax over values with exponents.  With scores z (log2 units) and a
// value's exponent e, the weights 2^z and the products' operands 2^(z + e), in fp16,
// need a reference each: the largest may differ by 2^237, and a row of zeros has the
// least exponent there is (-117) and any score.  m refers the weights and their sum l:
// l holds sum 2^(z - m), weights at most 2^kLag.  m + d refers the contributions, d an
// integer, and o holds sum 2^(z + e - m - d) v 2^-e: contributions at most 2^kLag too, the
// largest usually some 2^kLead.  Either one is raised when a block passes its lag.  (One
// reference for both, that of the contributions, lets the weights of zeros reach 2^131.)
// d is at least -110: contributions of the least exponents then stay under 2^7, and
// 2^kLag 2^-d is finite; and at most 120: no contribution is past 2^kLag, as e <= 120.
constexpr float kLag = 14.f, kLead = 6.f;
struct Raise {
  float m, d;             // the references from here on
  float l, o;             // factors of l and o
};
// From the block's largest score and contribution (-inf: none).
__device__ __forceinline__ bool must_raise(float m, float d, float score, float contribution) {
  return score > m + kLag || contribution > m + d + kLag;
}
__device__ __forceinline__ Raise raised(float m, float d, float score, float contribution) {
  if (!must_raise(m, d, score, contribution)) return Raise{m, d, 1.f, 1.f};
  Raise r;
  r.m = score > m + kLag ? score : m;
  const float to = contribution > m + d + kLag ? contribution - kLead : m + d;
  r.d = fminf(fmaxf(rintf(to - r.m), -110.f), 120.f);
  r.l = ex2_approx(m - r.m);
  r.o = ex2_approx((m - r.m) + (d - r.d));
  return r;
}
// 2^d, 2^-d of such a d.
__device__ __forceinline__ float shift_up(float d) { return __int_as_float((127 + static_cast<int>(d)) << 23); }
__device__ __forceinline__ float shift_down(float d) { return __int_as_float((127 - static_cast<int>(d)) << 23); }

// Results of a row are added up at the largest m and, next to it, the largest m + d (r):
// the d there, and the factors of a result's l and o.
__device__ __forceinline__ float shift_at(float m, float r) {
  return m == -INFINITY ? 0.f : fminf(fmaxf(rintf(r - m), -110.f), 120.f);
}
// (e4m3, with two of them a part: the approximation, off by 2^-22, 1 us of a tail chunk.)
template <bool E4M3>
__device__ __forceinline__ float sum_factor(float m, float to) {
  return m == to ? 1.f : E4M3 ? ex2_approx(m - to) : exp2f(m - to);
}
template <bool E4M3>
__device__ __forceinline__ float output_factor(float m, float d, float to_m, float to_d) {
  if constexpr (!E4M3) return sum_factor<false>(m, to_m);
  return m == -INFINITY ? 0.f : ex2_approx((m - to_m) + (d - to_d));
}

// Who shares the item that a worker begins and does not end: `parts` workers,
// the first of them that worker (0: none); the item's sequence, K/V head and
// first row among the rows of the two.  marked: rows of the worker's whole items may have
// to be computed again (many rows alone).
struct SplitHeader {
  int parts, s, head, rho0;
  Seq q;
  int marked;
};
static_assert(sizeof(SplitHeader) == 32, "read as two 16-byte words");

// Layout of the workspace: a header per worker, then two records per worker,
// 0 for the item that it found begun, 1 for the item that it leaves unended.  A record:
// unnormalised outputs [R][D], references of the weights [R], sums [R] and (e4m3) the
// outputs' shifts d [R], fp32.
struct Records {
  SplitHeader* headers;
  float* base;
  int rows;        // R
  int64_t size;    // floats per record (a multiple of 4)
  __device__ __forceinline__ float* at(int64_t worker, int which) const { return base + (2 * worker + which) * size; }
  __device__ __forceinline__ float* max_of(float* r, int d) const { return r + rows * d; }
  __device__ __forceinline__ float* sum_of(float* r, int d) const { return r + rows * d + rows; }
  __device__ __forceinline__ float* shift_of(float* r, int d) const { return r + rows * d + 2 * rows; }
};

inline int64_t record_floats(int rows, int d) { return (static_cast<int64_t>(rows) * (d + 3) + 3) & ~int64_t{3}; }
inline size_t records_bytes(int64_t workers, int rows, int d) {
  return static_cast<size_t>(workers) * (sizeof(SplitHeader) + 2 * record_floats(rows, d) * sizeof(float));
}
inline Records records_in(void* ws, int64_t workers, int rows, int d) {
  SplitHeader* h = static_cast<SplitHeader*>(ws);
  return Records{h, reinterpret_cast<float*>(h + workers), rows, record_floats(rows, d)};
}

// What a warp has of a row: references, sum, outputs 4 or 2 a lane.
template <int D>
struct Sum {
  float m = -INFINITY, d = 0.f, l = 0.f, o[D / 32] = {};
};

// Adds parts first, first + step, ... of one row of a split item to `sum`, loads of kBatch parts
// at a time.  The order is fixed, so a result depends on the lengths alone.
template <int D, bool E4M3, int kBatch>
__device__ __forceinline__ void join_parts(const Records& rec, int w, int parts, int row, int first, int step, int lane,
                                           Sum<D>& sum) {
  constexpr int kPer = D / 32;
  for (int p0 = first; p0 < parts; p0 += kBatch * step) {
    float mp[kBatch], dp[kBatch], lp[kBatch], op[kBatch][kPer];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int part = p0 + y * step;
      mp[y] = -INFINITY;
      dp[y] = lp[y] = 0.f;
#pragma unroll
      for (int x = 0; x < kPer; ++x) op[y][x] = 0.f;
      if (part < parts) {
        float* r = rec.at(w + part, part == 0 ? 1 : 0);
        mp[y] = rec.max_of(r, D)[row];
        lp[y] = rec.sum_of(r, D)[row];
        if constexpr (E4M3) dp[y] = rec.shift_of(r, D)[row];
        if constexpr (kPer == 4) {
          const float4 v = *reinterpret_cast<const float4*>(r + row * D + 4 * lane);
          op[y][0] = v.x, op[y][1] = v.y, op[y][2] = v.z, op[y][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(r + row * D + 2 * lane);
          op[y][0] = v.x, op[y][1] = v.y;
        }
      }
    }
    float m = sum.m, r = sum.m + sum.d;
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      m = fmaxf(m, mp[y]);
      r = fmaxf(r, mp[y] + dp[y]);
    }
    const float d = E4M3 ? shift_at(m, r) : 0.f;
    const float wa = output_factor<E4M3>(sum.m, sum.d, m, d);
    sum.l *= sum_factor<E4M3>(sum.m, m);
#pragma unroll
    for (int x = 0; x < kPer; ++x) sum.o[x] *= wa;
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const float wb = output_factor<E4M3>(mp[y], dp[y], m, d);
      sum.l += lp[y] * sum_factor<E4M3>(mp[y], m);
#pragma unroll
      for (int x = 0; x < kPer; ++x) sum.o[x] += op[y][x] * wb;
    }
    sum.m = m, sum.d = d;
  }
}

constexpr int kJoinWarps = 8;
// A row whose parts the warps of a block have added up: the warps' sums joined by the first.
template <int D, bool E4M3>
__device__ __forceinline__ void join_warps(int warp, int lane, Sum<D>& sum) {
  constexpr int kPer = D / 32;
  __shared__ float sm[kJoinWarps], sd[kJoinWarps], sl[kJoinWarps], so[kJoinWarps][D];
  __syncthreads();          // the previous row's results have been read
  if (lane == 0) {
    sm[warp] = sum.m;
    sd[warp] = sum.d;
    sl[warp] = sum.l;
  }
#pragma unroll
  for (int x = 0; x < kPer; ++x) so[warp][lane * kPer + x] = sum.o[x];
  __syncthreads();
  if (warp != 0) return;
  float r = sm[0] + sd[0];
  sum.m = sm[0];
#pragma unroll
  for (int y = 1; y < kJoinWarps; ++y) {
    sum.m = fmaxf(sum.m, sm[y]);
    r = fmaxf(r, sm[y] + sd[y]);
  }
  sum.d = E4M3 ? shift_at(sum.m, r) : 0.f;
  sum.l = 0.f;
#pragma unroll
  for (int x = 0; x < kPer; ++x) sum.o[x] = 0.f;
#pragma unroll
  for (int y = 0; y < kJoinWarps; ++y) {
    const float f = output_factor<E4M3>(sm[y], sd[y], sum.m, sum.d);
    sum.l += sl[y] * sum_factor<E4M3>(sm[y], sum.m);
#pragma unroll
    for (int x = 0; x < kPer; ++x) sum.o[x] += so[y][lane * kPer + x] * f;
  }
}

// One warp writes a joined row; positions(p0, p1): those of the rows that share its item's key blocks.
template <int D, bool E4M3, typename F>
__device__ __forceinline__ void join_finish(const AttentionArgs& a, const SplitHeader& hd, int rho, const Sum<D>& sum,
                                            int lane, F&& positions) {
  const int i = a.by_group(rho), h = hd.head * a.group + rho - i * a.group, p = hd.q.kv - hd.q.c + i;
  bf16* to = a.out + (hd.q.row0 + i) * a.out_stride + h * D + lane * (D / 32);
  const float inv = 1.f / sum.l, up = E4M3 ? shift_up(sum.d) : 1.f;
  bool bad = false;
  uint32_t w[D / 64];
#pragma unroll
  for (int x = 0; x < D / 64; ++x) {
    const float y0 = p < 0 ? 0.f : sum.o[2 * x] * inv * up, y1 = p < 0 ? 0.f : sum.o[2 * x + 1] * inv * up;
    bad |= not_finite(y0) || not_finite(y1);
    w[x] = pack_bf16x2(y0, y1);
  }
  if constexpr (D == 128)
    *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(to) = w[0];
  if (hd.q.c > 1 && __any_sync(0xFFFFFFFFu, bad)) {
    __syncwarp();
    int p0, p1;
    positions(p0, p1);
    mend_row<D, E4M3>(a, hd.s, hd.q.row0, p, i, h, p0, p1, lane);
  }
}

}  // namespace dsvit
