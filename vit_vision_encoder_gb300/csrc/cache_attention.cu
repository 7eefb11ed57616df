// Attention of new tokens over the paged K/V cache (include/dsvit.h,
// ds_vit_cache_attention).
#include "cache.cuh"

namespace dsvit {

namespace {

// One warp per (packed row, query head), keys one after the other: scores by
// a warp sum, running maximum and sum of the softmax in fp32.
template <int D, bool E4M3>
__global__ void __launch_bounds__(128) row_attention_kernel(const __grid_constant__ AttentionArgs a) {
  constexpr int kPer = D / 32;
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0)
    for (int s = threadIdx.x; s < a.b.n; s += 128) load_seq(a.b, a.c.page_shift, s, a.status);
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (item >= static_cast<int64_t>(a.b.rows) * a.heads) return;
  const int r = static_cast<int>(item / a.heads), h = static_cast<int>(item % a.heads);
  const int s = find_seq(a.b, r, lane);
  if (s < 0) return;
  const Seq sq = load_seq(a.b, a.c.page_shift, s, a.status);
  if (static_cast<unsigned>(r - sq.row0) >= static_cast<unsigned>(sq.c)) return;
  const int p = sq.kv - sq.c + (r - sq.row0);
  float q[kPer], o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = __bfloat162float(a.q[r * a.q_stride + h * D + lane * kPer + i]);
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j <= p; ++j) {
    if (!sees(a, p, j)) continue;
    const int64_t page = page_of(a.b, a.c, s, j, a.status);
    if (page < 0) return;
    const int64_t row = cache_row(a.c, page, h / a.group, j);
    float kx[kPer], vx[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t at = row * D + lane * kPer + i;
      if constexpr (E4M3) {
        kx[i] = e4m3x2_to_float2(a.c.k[at]).x * exp_factor(a.c.k_exp[row]);
        vx[i] = e4m3x2_to_float2(a.c.v[at]).x * exp_factor(a.c.v_exp[row]);
      } else {
        kx[i] = __bfloat162float(reinterpret_cast<const bf16*>(a.c.k)[at]);
        vx[i] = __bfloat162float(reinterpret_cast<const bf16*>(a.c.v)[at]);
      }
    }
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) d = fmaf(q[i], kx[i], d);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, x);
    d *= a.scale_log2;
    const float m_new = fmaxf(m, d);
    const float alpha = m == m_new ? 1.f : exp2f(m - m_new);
    const float w = exp2f(d - m_new);
    l = l * alpha + w;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * alpha + w * vx[i];
    m = m_new;
  }
  const float inv = p < 0 ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    a.out[r * a.out_stride + h * D + lane * kPer + i] = __float2bfloat16_rn(o[i] * inv);
}

}  // namespace

size_t cache_attention_workspace(int head_dim, int group, int max_rows) {
  const int64_t rows = static_cast<int64_t>(max_rows) * group;
  return rows <= kDecodeRows ? cache_decode_workspace(head_dim, static_cast<int>(rows)) : 256;
}

int launch_cache_attention(const AttentionArgs& a, int head_dim, bool e4m3, void* ws, cudaStream_t stream) {
  if (static_cast<int64_t>(a.b.max_rows) * a.group <= kDecodeRows)
    return launch_cache_decode(a, head_dim, e4m3, ws, stream);
  auto* fn = head_dim == 128 ? (e4m3 ? row_attention_kernel<128, true> : row_attention_kernel<128, false>)
                             : (e4m3 ? row_attention_kernel<64, true> : row_attention_kernel<64, false>);
  const int64_t items = static_cast<int64_t>(a.b.rows) * a.heads;
  const cudaError_t e = launch_pdl(fn, dim3(static_cast<unsigned>((items + 3) / 4)), dim3(128), 0, stream, a);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? DS_VIT_OK : DS_VIT_ECUDA;
}

}  // namespace dsvit
