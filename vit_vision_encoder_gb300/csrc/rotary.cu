// Norms of queries and keys for each head and their rotation by position, in one
// pass (include/dsvit.h, ds_vit_qk_norm_rope).
//
// Every byte is read once and written once: bound by memory at prompt lengths and by
// the chain load -> norm -> store at one token a sequence.  D / 16 lanes hold one head, 16
// values each: the 16-byte pieces l and l + D / 16 of the row, so that both loads
// of a warp are whole lines and both members of every pair lie in one lane under either
// pairing (the norm's sum is the only exchange between lanes).  A pass is the 512 / D heads that a
// warp holds at a time; a warp takes up to kBatch passes of a row's queries or of its keys together, one pass where
// there are few rows.  The norm's weights go into the row's sines and cosines once a batch:
//   y_a = f (x_a [g_a cos] - x_b [g_b sin]),  y_b = f (x_b [g_b cos] + x_a [g_a sin]).
// 8500 rows of 40 and 8 heads of 128: 36.5 us, 84% of the rate of a plain copy; batches of 4 passes 38.5, of 6 38.0 (as many as
// the registers of four CTAs an SM hold), queries and keys mixed in a batch and the weights
// multiplied into each head 41; the next batch's loads ahead of the work gained nothing.  48 rows 3.1 us, a
// launch and three dependent trips to memory.
//
// Angles: positions are whole numbers, so the fraction of a turn is
// pos * (freq / 2 pi) modulo 1 in 64-bit fixed point, exact but for the frequency's own
// rounding, with no reduction of large arguments; sincospif takes its upper 32 bits.
// A lane works out D / 64 pairs' sines and cosines for the whole warp.
#include <algorithm>
#include <cmath>

#include "cache.cuh"

namespace dsvit {

namespace {

constexpr int kWarps = 4;
constexpr int kBatch = 5;    // passes whose loads are in flight together
constexpr int kWarpsPerSm = 16;

struct RotaryArgs {
  ds_vit_rotary r;
  const bf16* x[2];          // q, k
  bf16* y[2];
  int64_t x_stride[2], y_stride[2];
  const bf16* norm[2];
  int heads[2];
  const int32_t* pos;
  int64_t pos_stride;
  int64_t rows;
  int batches[2];            // of a row's q, k: batch b has passes b, b + batches, ...
  int64_t each;              // batches of a warp, one behind the other
  float eps;
};

// Pair j of a lane's eight, of those of a head: pieces l and l + D / 16 hold them as
// halves of pairs, or as four pairs each.
template <int D, bool kAdjacent>
__device__ __forceinline__ int pair_of(int l, int j) {
  if constexpr (!kAdjacent) return 8 * l + j;
  return j < 4 ? 4 * l + j : D / 4 + 4 * l + j - 4;
}

template <int D, bool kAdjacent>
__global__ void __launch_bounds__(32 * kWarps, kWarpsPerSm / kWarps) qk_norm_rope_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes, kOwn = D / 64;
  grid_dep_launch();
  const int lane = threadIdx.x & 31, l = lane % kLanes, h0 = lane / kLanes;
  uint64_t turn[kOwn];
  int axis[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    turn[i] = a.r.turn[lane * kOwn + i];
    axis[i] = a.r.axis[lane * kOwn + i];
  }
  grid_dep_wait();
  const int per_row = a.batches[0] + a.batches[1];
  const int64_t begin = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * a.each;
  const int64_t end = min(begin + a.each, a.rows * per_row);
  if (begin >= end) return;
  int64_t row = begin / per_row;
  int batch = static_cast<int>(begin - row * per_row);
  bool turned = false;                  // whether c and s are the row's
  float c[8], s[8];
  for (int64_t u = begin; u < end; ++u) {
    const int x = batch >= a.batches[0], first = x ? batch - a.batches[0] : batch;
    const int heads = x ? a.heads[1] : a.heads[0], step = x ? a.batches[1] : a.batches[0];
    const bf16* const from = (x ? a.x[1] + row * a.x_stride[1] : a.x[0] + row * a.x_stride[0]) + 8 * l;
    bf16* const to = (x ? a.y[1] + row * a.y_stride[1] : a.y[0] + row * a.y_stride[0]) + 8 * l;
    const bf16* const norm = x ? a.norm[1] : a.norm[0];
    uint4 lo[kBatch], hi[kBatch];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int h = (first + y * step) * kHeads + h0;
      lo[y] = hi[y] = make_uint4(0, 0, 0, 0);
      if (h < heads) {
        lo[y] = *reinterpret_cast<const uint4*>(from + h * D);
        hi[y] = *reinterpret_cast<const uint4*>(from + h * D + D / 2);
      }
    }
    uint4 g[2] = {make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u),      // ones
                  make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u)};
    if (norm != nullptr) {
      g[0] = __ldg(reinterpret_cast<const uint4*>(norm) + l);
      g[1] = __ldg(reinterpret_cast<const uint4*>(norm) + l + kLanes);
    }
    if (!turned) {
      float co[kOwn], so[kOwn];
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int32_t at = __ldg(a.pos + axis[i] * a.pos_stride + row);
        const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(at)) * turn[i];
        sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-31f, &so[i], &co[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int p = pair_of<D, kAdjacent>(l, j), i = kOwn == 2 ? j & 1 : 0;
        c[j] = __shfl_sync(0xFFFFFFFFu, co[i], p / kOwn);
        s[j] = __shfl_sync(0xFFFFFFFFu, so[i], p / kOwn);
      }
    }
    const uint32_t gw[8] = {g[0].x, g[0].y, g[0].z, g[0].w, g[1].x, g[1].y, g[1].z, g[1].w};
    float gc[16], gs[16];                // of each value: g times the pair's cosine, sine
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int j = kAdjacent ? i / 2 : i & 7;
      const float gi = i & 1 ? bf16hi(gw[i / 2]) : bf16lo(gw[i / 2]);
      gc[i] = gi * c[j];
      gs[i] = gi * s[j];
    }
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      if ((first + y * step) * kHeads >= heads) break;
      const int h = (first + y * step) * kHeads + h0;
      const uint32_t w[8] = {lo[y].x, lo[y].y, lo[y].z, lo[y].w, hi[y].x, hi[y].y, hi[y].z, hi[y].w};
      float v[16], f = 1.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[2 * i] = bf16lo(w[i]);
        v[2 * i + 1] = bf16hi(w[i]);
      }
      if (norm != nullptr) {
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i & 1] = fmaf(v[i], v[i], sum[i & 1]);
        float all = sum[0] + sum[1];
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
        f = rsqrtf(all * (1.f / D) + a.eps);
      }
      float r[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // Pair j's members among the lane's values: (j, j + 8), or (2j, 2j + 1).
        const int m0 = kAdjacent ? 2 * j : j, m1 = kAdjacent ? 2 * j + 1 : j + 8;
        r[m0] = (v[m0] * gc[m0] - v[m1] * gs[m1]) * f;
        r[m1] = (v[m1] * gc[m1] + v[m0] * gs[m0]) * f;
      }
      if (h < heads) {
        *reinterpret_cast<uint4*>(to + h * D) =
            make_uint4(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]), pack_bf16x2(r[4], r[5]), pack_bf16x2(r[6], r[7]));
        *reinterpret_cast<uint4*>(to + h * D + D / 2) = make_uint4(pack_bf16x2(r[8], r[9]), pack_bf16x2(r[10], r[11]),
                                                                   pack_bf16x2(r[12], r[13]), pack_bf16x2(r[14], r[15]));
      }
    }
    turned = true;
    if (++batch == per_row) {
      batch = 0;
      ++row;
      turned = false;
    }
  }
}

// f / 2 pi modulo 1 in units of 2^-64, rounded down, f positive and finite.  f is m 2^(x - 53) with m whole and under 2^53;
// 1 / 2 pi goes in as 128 bits, whose error is f 2^-128 turns.  Whole numbers throughout: the same on every machine.
uint64_t turns_of(double f) {
  constexpr uint64_t kHigh = 0x28BE60DB9391054Au, kLow = 0x7F09D5F47D4D3770u;    // 2^128 / 2 pi, rounded down
  int x;
  const uint64_t m = static_cast<uint64_t>(std::ldexp(std::frexp(f, &x), 53));
  const int right = 53 - x + 64;            // m kHigh:kLow is in units of 2^(x - 53 - 128) turns: 2^-right of those wanted
  const unsigned __int128 low = static_cast<unsigned __int128>(m) * kLow;
  const unsigned __int128 high = static_cast<unsigned __int128>(m) * kHigh + static_cast<uint64_t>(low >> 64);
  const uint64_t words[4] = {static_cast<uint64_t>(low), static_cast<uint64_t>(high), static_cast<uint64_t>(high >> 64), 0};
  if (right <= 0) return right > -64 ? words[0] << -right : 0;
  if (right >= 192) return 0;
  const int word = right / 64, bit = right % 64;
  return words[word] >> bit | (bit ? words[word + 1] << (64 - bit) : 0);
}

}  // namespace

}  // namespace dsvit

using namespace dsvit;

extern "C" {

int ds_vit_rotary_init(int32_t head_dim, double theta, const double* inv_freq, int32_t axes,
                       const int32_t* sections, int32_t interleaved, int32_t pairing, ds_vit_rotary* out) {
  if (!out || (head_dim != 64 && head_dim != 128) || (axes != 1 && axes != 3) ||
      (pairing != DS_VIT_ROPE_HALF_VECTOR && pairing != DS_VIT_ROPE_ADJACENT) || (axes == 3 && !sections) ||
      (!inv_freq && !(theta > 1.0 && std::isfinite(theta))))
    return DS_VIT_EINVAL;
  const int pairs = head_dim / 2;
  if (axes == 3) {
    int64_t sum = 0;
    for (int a = 0; a < 3; ++a) {
      if (sections[a] < 0 || (interleaved && a > 0 && 3 * static_cast<int64_t>(sections[a]) > pairs + 2 - a))
        return DS_VIT_EINVAL;
      sum += sections[a];
    }
    if (sum != pairs) return DS_VIT_EINVAL;
  }
  ds_vit_rotary r{};
  r.head_dim = head_dim;
  r.axes = axes;
  r.pairing = pairing;
  for (int i = 0; i < pairs; ++i) {
    const double f = inv_freq ? inv_freq[i] : std::pow(theta, -static_cast<double>(i) / pairs);
    if (!(f > 0.0 && std::isfinite(f))) return DS_VIT_EINVAL;
    r.turn[i] = turns_of(f);
    if (axes == 3 && interleaved)
      r.axis[i] = static_cast<uint8_t>(i % 3 && i < 3 * sections[i % 3] ? i % 3 : 0);
    else if (axes == 3)
      r.axis[i] = static_cast<uint8_t>((i >= sections[0]) + (i >= sections[0] + sections[1]));
  }
  *out = r;
  return DS_VIT_OK;
}

int ds_vit_qk_norm_rope(const ds_vit_rotary* rotary, const void* q, int64_t q_stride, int32_t heads,
                        const void* k, int64_t k_stride, int32_t kv_heads, int64_t rows, const int32_t* pos,
                        int64_t pos_stride, const void* q_norm, const void* k_norm, float eps, void* q_out,
                        int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  if (!rotary || (rotary->head_dim != 64 && rotary->head_dim != 128) || (rotary->axes != 1 && rotary->axes != 3) ||
      (rotary->pairing != DS_VIT_ROPE_HALF_VECTOR && rotary->pairing != DS_VIT_ROPE_ADJACENT) || heads < 1 ||
      heads > DS_VIT_CACHE_MAX_HEADS * DS_VIT_CACHE_MAX_GROUP || kv_heads < 1 || kv_heads > DS_VIT_CACHE_MAX_HEADS ||
      rows < 0)
    return DS_VIT_EINVAL;
  const int d = rotary->head_dim;
  for (int i = 0; i < d / 2; ++i)
    if (rotary->axis[i] >= rotary->axes) return DS_VIT_EINVAL;
  const int64_t qw = static_cast<int64_t>(heads) * d, kw = static_cast<int64_t>(kv_heads) * d;
  if (bad_rows(q, q_stride, qw) || bad_rows(k, k_stride, kw) || bad_rows(q_out, q_out_stride, qw) ||
      bad_rows(k_out, k_out_stride, kw) || !pos || !aligned(pos, 4) || (rotary->axes > 1 && pos_stride < rows) ||
      !aligned(q_norm, 16) || !aligned(k_norm, 16) || ((q_norm || k_norm) && !(eps > 0.f && std::isfinite(eps))))
    return DS_VIT_EINVAL;
  if (rows > INT32_MAX / 2) return DS_VIT_ERANGE;
  if (rows == 0) return DS_VIT_OK;
  RotaryArgs a{};
  a.r = *rotary;
  a.x[0] = static_cast<const bf16*>(q), a.x[1] = static_cast<const bf16*>(k);
  a.y[0] = static_cast<bf16*>(q_out), a.y[1] = static_cast<bf16*>(k_out);
  a.x_stride[0] = q_stride, a.x_stride[1] = k_stride;
  a.y_stride[0] = q_out_stride, a.y_stride[1] = k_out_stride;
  a.norm[0] = static_cast<const bf16*>(q_norm), a.norm[1] = static_cast<const bf16*>(k_norm);
  a.heads[0] = heads, a.heads[1] = kv_heads;
  a.pos = pos;
  a.pos_stride = rotary->axes > 1 ? pos_stride : 0;
  a.rows = rows;
  a.eps = eps;
  // Few rows: a pass a warp, as long as that is no more warps than run at once.
  const int64_t warps = kWarpsPerSm * static_cast<int64_t>(num_sms());
  int per_batch = kBatch, per_row;
  for (;; --per_batch) {
    per_row = 0;
    for (int x = 0; x < 2; ++x) {
      const int passes = (a.heads[x] + 512 / d - 1) / (512 / d);
      a.batches[x] = (passes + per_batch - 1) / per_batch;
      per_row += a.batches[x];
    }
    if (per_batch == 1 || 2 * rows * per_row > warps) break;
  }
  const int64_t batches = rows * per_row;
  a.each = (batches + warps - 1) / warps;
  const unsigned blocks = static_cast<unsigned>(((batches + a.each - 1) / a.each + kWarps - 1) / kWarps);
  const bool adj = rotary->pairing == DS_VIT_ROPE_ADJACENT;
  auto* fn = d == 128 ? (adj ? qk_norm_rope_kernel<128, true> : qk_norm_rope_kernel<128, false>)
                      : (adj ? qk_norm_rope_kernel<64, true> : qk_norm_rope_kernel<64, false>);
  return launched(launch_pdl(fn, dim3(blocks), dim3(32 * kWarps), 0, static_cast<cudaStream_t>(stream), a));
}

}  // extern "C"
