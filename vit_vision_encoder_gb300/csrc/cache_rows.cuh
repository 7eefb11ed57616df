// Pieces shared by the attention kernels over the paged cache: the plan of a
// call's work, the records of results that several workers share, and the
// row computed key by key.
#pragma once

#include "cache.cuh"
#include "cache_plan.h"

namespace dsvit {

// One row of the result, key by key, by one warp.  The matrix products give a
// hidden key the weight 0, and 0 times an infinity or NaN in its value is NaN;
// where a chunk's rows see different keys, a row whose result is not finite
// comes here and is computed from the keys that it does see.
template <int D, bool E4M3>
__device__ __noinline__ void exact_row(const AttentionArgs& a, int s, int row0, int p, int i, int h, int lane) {
  constexpr int kPer = D / 32;
  const bf16* qr = a.q + (row0 + i) * a.q_stride + h * D + lane * kPer;
  float q[kPer], o[kPer];
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    q[x] = __bfloat162float(qr[x]);
    o[x] = 0.f;
  }
  const int lo = a.window != 0 && p >= a.window ? p - a.window + 1 : 0;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j <= p; ++j) {
    if (j >= a.sinks && j < lo) j = lo;
    const int64_t page = page_of(a.b, a.c, s, j, a.status);
    if (page < 0) return;
    const int64_t row = cache_row(a.c, page, h / a.group, j);
    float kx[kPer], vx[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int64_t at = row * D + lane * kPer + x;
      if constexpr (E4M3) {
        kx[x] = e4m3x2_to_float2(a.c.k[at]).x * exp_factor(a.c.k_exp[row]);
        vx[x] = e4m3x2_to_float2(a.c.v[at]).x * exp_factor(a.c.v_exp[row]);
      } else {
        kx[x] = __bfloat162float(reinterpret_cast<const bf16*>(a.c.k)[at]);
        vx[x] = __bfloat162float(reinterpret_cast<const bf16*>(a.c.v)[at]);
      }
    }
    float d = 0.f;
#pragma unroll
    for (int x = 0; x < kPer; ++x) d = fmaf(q[x], kx[x], d);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, x);
    d *= a.scale_log2;
    const float m_new = fmaxf(m, d);
    const float alpha = m == m_new ? 1.f : exp2f(m - m_new);
    const float w = exp2f(d - m_new);
    l = l * alpha + w;
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] = o[x] * alpha + w * vx[x];
    m = m_new;
  }
  bf16* to = a.out + (row0 + i) * a.out_stride + h * D + lane * kPer;
#pragma unroll
  for (int x = 0; x < kPer; ++x) to[x] = __float2bfloat16_rn(p < 0 ? 0.f : o[x] / l);
}

__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u; }

// Who shares the item that a worker begins and does not end: `parts` workers,
// the first of them that worker (0: none).
struct SplitHeader {
  int parts, s, head, tile;
};

// Layout of the workspace: a header per worker, then two records per worker,
// 0 for the item that it found begun, 1 for the item that it leaves unended.  A record:
// unnormalised outputs [R][D], maxima [R], sums [R], fp32.
struct Records {
  SplitHeader* headers;
  float* base;
  int rows;        // R
  int64_t size;    // floats per record (a multiple of 4)
  __device__ __forceinline__ float* at(int64_t worker, int which) const { return base + (2 * worker + which) * size; }
  __device__ __forceinline__ float* max_of(float* r, int d) const { return r + rows * d; }
  __device__ __forceinline__ float* sum_of(float* r, int d) const { return r + rows * d + rows; }
};

inline int64_t record_floats(int rows, int d) { return (static_cast<int64_t>(rows) * (d + 2) + 3) & ~int64_t{3}; }
inline size_t records_bytes(int64_t workers, int rows, int d) {
  return static_cast<size_t>(workers) * (sizeof(SplitHeader) + 2 * record_floats(rows, d) * sizeof(float));
}
inline Records records_in(void* ws, int64_t workers, int rows, int d) {
  SplitHeader* h = static_cast<SplitHeader*>(ws);
  return Records{h, reinterpret_cast<float*>(h + workers), rows, record_floats(rows, d)};
}

// Joins the parts of every split item: O = sum_p 2^(m_p - M) O_p, L alike.  One
// block per (group of workers, row): its warps share the parts, each with a
// running maximum, and are joined through shared memory in a fixed order, so
// a result depends on the lengths alone.  Worker groups: blockIdx.x, then every
// gridDim.x-th worker.
constexpr int kJoinWarps = 8;

template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kJoinWarps)
    join_kernel(const __grid_constant__ AttentionArgs a, const Records rec, int workers) {
  constexpr int kPer = D / 32;
  __shared__ float sm[kJoinWarps], sl[kJoinWarps], so[kJoinWarps][D];
  grid_dep_launch();
  grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int w = blockIdx.x; w < workers; w += gridDim.x) {
    const SplitHeader hd = rec.headers[w];
    if (hd.parts == 0) continue;
    const Seq sq = load_seq(a.b, a.c.page_shift, hd.s, nullptr);
    const int row = static_cast<int>(blockIdx.y), rho = hd.tile * rec.rows + row;
    if (rho >= sq.c * a.group) continue;
    float m = -INFINITY, l = 0.f, o[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] = 0.f;
    for (int part = warp; part < hd.parts; part += kJoinWarps) {
      float* r = rec.at(w + part, part == 0 ? 1 : 0);
      const float mp = rec.max_of(r, D)[row], lp = rec.sum_of(r, D)[row];
      float op[kPer];
#pragma unroll
      for (int x = 0; x < kPer; ++x) op[x] = r[row * D + lane * kPer + x];
      const float m_new = fmaxf(m, mp);
      const float wa = m == m_new ? 1.f : exp2f(m - m_new), wb = mp == m_new ? 1.f : exp2f(mp - m_new);
      l = l * wa + lp * wb;
#pragma unroll
      for (int x = 0; x < kPer; ++x) o[x] = o[x] * wa + op[x] * wb;
      m = m_new;
    }
    __syncthreads();      // the previous item's results have been read
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
#pragma unroll
    for (int x = 0; x < kPer; ++x) so[warp][lane * kPer + x] = o[x];
    __syncthreads();
    if (warp == 0) {
      float M = sm[0];
#pragma unroll
      for (int x = 1; x < kJoinWarps; ++x) M = fmaxf(M, sm[x]);
      float L = 0.f;
#pragma unroll
      for (int x = 0; x < kPer; ++x) o[x] = 0.f;
#pragma unroll
      for (int y = 0; y < kJoinWarps; ++y) {
        const float f = sm[y] == M ? 1.f : exp2f(sm[y] - M);
        L += sl[y] * f;
#pragma unroll
        for (int x = 0; x < kPer; ++x) o[x] += so[y][lane * kPer + x] * f;
      }
      const int i = rho / a.group, h = hd.head * a.group + rho % a.group, p = sq.kv - sq.c + i;
      bool bad = false;
      bf16* to = a.out + (sq.row0 + i) * a.out_stride + h * D + lane * kPer;
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        const float y = p < 0 ? 0.f : o[x] / L;
        bad |= not_finite(y);
        to[x] = __float2bfloat16_rn(y);
      }
      if (sq.c > 1 && __any_sync(0xFFFFFFFFu, bad)) {
        __syncwarp();
        exact_row<D, E4M3>(a, hd.s, sq.row0, p, i, h, lane);
      }
    }
  }
}

}  // namespace dsvit
