// Attention over the paged cache for few rows: at most 32 query rows (new
// tokens times query heads per K/V head) share a K/V head, as in decoding.
//
// Bound by the cache's bytes: each key and value is read once and meets at
// most 32 rows, 64 flops a byte of bf16.  That is under a tenth of the tensor
// rate the bytes could feed, so the products run as warp MMAs (m16n8k16),
// whose fragments come straight from shared memory; what counts is bytes in
// flight and few instructions per key.
//
// Work: the unit is a block of 16 keys (always inside one page) of one item
// (sequence, K/V head).  All units of a call are counted from the lengths on
// the device and dealt in order to the workers, the warps of the grid, in
// equal shares (cache_plan.h), so a batch of unequal lengths and a single long
// sequence both keep every SM reading.  A worker streams its blocks through
// its own ring of TMA tiles, with its own barriers and running softmax; warps
// never wait for one another.  Items that lie within one worker's share are
// finished there, the others leave records that join_kernel adds up.
//
// bf16: S = Q K^T with K fragments by ldmatrix, P V with V fragments by
// ldmatrix.trans.  e4m3: a lane loads 16 bytes of a key (16 dims) or of two
// values' rows and widens pairs to fp16 in registers (one conversion a pair,
// exact; bf16 has no such conversion, and bit operations to the same end took
// five instructions a pair and 437 us where these take REPLACED).  The order
// of dims within a product is free as long as both operands share it, and so is
// the order of output columns, so a lane's bytes are used where they lie.
// fp16's range is kept by powers of two: each query row is scaled to a largest
// magnitude in [2^14, 2^15) (the scores are scaled back), and the weights carry
// the values' exponents and are taken against the running maximum of score
// plus exponent, the size of a key's contribution, so that the largest stay in
// [2^6, 2^14]; contributions under 2^-20 of the largest lose bits.
#include "cache_rows.cuh"

namespace dsvit {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlockShift = 4;             // 16 keys
constexpr int kRingBytes = 24 * 1024;      // per warp
// A row's reference m (log2) is raised when a block's maximum passes m + kLag,
// to kLead below that maximum; weights are 2^(x - m).
template <bool E4M3>
struct Reference {
  static constexpr float kLag = E4M3 ? 14.f : 8.f;
  static constexpr float kLead = E4M3 ? 6.f : 0.f;
};

template <int D, bool E4M3>
struct Shape {
  static constexpr int kRow = E4M3 ? D : 2 * D;            // bytes of a key
  static constexpr int kTile = 16 * kRow;
  static constexpr int kStage = 2 * kTile;                 // K, then V
  static constexpr int kStages = kRingBytes / kStage;
  static constexpr int kExp = E4M3 ? 32 : 0;               // exponents of a stage: 16 K, 16 V
  static constexpr int kSmem = 1024 + kWarps * (kRingBytes + kStages * (8 + kExp)) + 8 * (DS_VIT_MAX_SEQS + 1);
};

// An item and the part of its blocks that a worker takes.
struct Item {
  int s, head;
  Seq q;
  KeyBlocks kb;
  int b, end;      // next block, end of the worker's part
};

struct Plan {
  const int64_t* pre;   // [n + 1]: units of the sequences before each
  int64_t begin, end;   // the worker's units
};

__device__ __forceinline__ KeyBlocks seq_blocks(const AttentionArgs& a, const Seq& q) {
  KeyBlocks kb = key_blocks(q.kv - q.c, q.kv - 1, a.window, a.sinks, kBlockShift);
  if (q.c > 0 && kb.count == 0) kb.count = 1;   // nothing visible: one block without keys, so that zeros get written
  return kb;
}

// The item of unit u and the worker's part of it.
__device__ __forceinline__ Item item_at(const AttentionArgs& a, const Plan& pl, int64_t u) {
  int lo = 0, hi = a.b.n - 1;              // the last s with pre[s] <= u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pl.pre[mid] <= u)
      lo = mid;
    else
      hi = mid - 1;
  }
  Item it;
  it.s = lo;
  it.q = load_seq(a.b, a.c.page_shift, lo, nullptr);
  it.kb = seq_blocks(a, it.q);
  const int64_t r = u - pl.pre[lo];
  it.head = static_cast<int>(r / it.kb.count);
  it.b = static_cast<int>(r - static_cast<int64_t>(it.head) * it.kb.count);
  const int64_t left = pl.end - u;
  it.end = left < it.kb.count - it.b ? it.b + static_cast<int>(left) : it.kb.count;
  return it;
}

template <int D, bool E4M3, int MT>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ AttentionArgs a, const Records rec) {
  using S = Shape<D, E4M3>;
  constexpr int kSteps = D / 16;           // k steps of S, and half the column tiles of O
  constexpr int kCols = D / 8;             // column tiles of O
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * kRingBytes;
  uint8_t* tail = smem + kWarps * kRingBytes;
  const uint32_t exps = smem_u32(tail) + warp * S::kStages * S::kExp;
  tail += kWarps * S::kStages * S::kExp;
  const uint32_t bar0 = smem_u32(tail) + warp * S::kStages * 8;
  tail += kWarps * S::kStages * 8;
  int64_t* pre = reinterpret_cast<int64_t*>(tail);
  __shared__ int64_t part[kWarps];

  if (lane == 0) {
    for (int i = 0; i < S::kStages; ++i) mbar_init(bar0 + 8 * i, 1);
    if (warp == 0) {
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
    }
  }
  fence_barrier_init();
  grid_dep_launch();
  grid_dep_wait();

  // ---- plan: units before each sequence
  int64_t total = 0;
  for (int s0 = 0; s0 < a.b.n; s0 += kThreads) {
    const int s = s0 + threadIdx.x;
    int64_t x = 0;
    if (s < a.b.n) {
      const Seq q = load_seq(a.b, a.c.page_shift, s, blockIdx.x == 0 ? a.status : nullptr);
      x = static_cast<int64_t>(seq_blocks(a, q).count) * (q.c > 0 ? a.c.kv_heads : 0);
    }
    int64_t inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    int64_t before = total;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += part[w];
      total += part[w];
    }
    if (s < a.b.n) pre[s] = before + inc - x;
    __syncthreads();
  }
  if (threadIdx.x == 0) pre[a.b.n] = total;
  __syncthreads();

  const int64_t all = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t W = total < all ? total : all;
  const int64_t me = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
  if (me >= W) {
    if (lane == 0) rec.headers[me] = SplitHeader{0, 0, 0, 0};
    return;
  }
  const Plan pl{pre, share_begin(me, W, total), share_begin(me + 1, W, total)};

  // ---- the ring: lane 0 loads blocks, kStages ahead of their use
  int64_t load_u = pl.begin;
  Item ld = item_at(a, pl, load_u);
  int pg = 0, pg_from = -32;               // table entries of blocks pg_from + lane of ld
  int slot_ld = 0;
  auto load_next = [&]() {
    if (load_u >= pl.end) return;
    if (ld.b >= ld.end) {
      ld = item_at(a, pl, load_u);
      pg_from = -32;
    }
    if (ld.b >= pg_from + 32 || pg_from < 0) {
      pg_from = ld.b;
      const int b = ld.b + lane;
      pg = -1;
      if (b < ld.end && ld.q.kv > ld.kb.at(b) << kBlockShift)
        pg = static_cast<int>(page_of(a.b, a.c, ld.s, ld.kb.at(b) << kBlockShift, a.status));
    }
    const int page = __shfl_sync(0xFFFFFFFFu, pg, ld.b - pg_from);
    if (lane == 0) {
      const uint32_t bar = bar0 + 8 * slot_ld, to = ring + slot_ld * S::kStage;
      if (page < 0) {
        mbar_arrive(bar);                  // no such page (reported), or an item without keys
      } else {
        const int row = static_cast<int>(cache_row(a.c, page, ld.head, ld.kb.at(ld.b) << kBlockShift));
        mbar_expect_tx(bar, S::kStage + S::kExp);
        if constexpr (E4M3) {
          tma_load_2d(to, &tm_k, bar, 0, row);
          bulk_load(exps + slot_ld * S::kExp, a.c.k_exp + row, 16, bar);
          tma_load_2d(to + S::kTile, &tm_v, bar, 0, row);
          bulk_load(exps + slot_ld * S::kExp + 16, a.c.v_exp + row, 16, bar);
        } else {
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            tma_load_2d(to + 2048 * x, &tm_k, bar, 64 * x, row);
            tma_load_2d(to + S::kTile + 2048 * x, &tm_v, bar, 64 * x, row);
          }
        }
      }
    }
    ++ld.b;
    ++load_u;
    if (++slot_ld == S::kStages) slot_ld = 0;
  };
  for (int i = 0; i < S::kStages; ++i) load_next();

  // ---- the worker's items
  int slot = 0;
  uint32_t phase = 0;
  SplitHeader header{0, 0, 0, 0};
  bool ok = true;
  int64_t used_u = pl.begin;               // blocks used so far
  for (int64_t u = pl.begin; u < pl.end;) {
    const Item it = item_at(a, pl, u);
    const int R = it.q.c * a.group;
    // Q fragments and positions of rows g, g + 8 of each row tile.
    uint32_t qf[MT][kSteps][4];
    int pos[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int rho = 16 * mt + 8 * x + g;
        const int i = rho / a.group;
        pos[mt][x] = rho < R ? it.q.kv - it.q.c + i : -1;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            a.q + (it.q.row0 + i) * a.q_stride + (it.head * a.group + rho - i * a.group) * D);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          // Dims of the k step held by this lane: 2t, 2t + 1 and 2t + 8, 2t + 9
          // of 16, or (e4m3) four consecutive ones of its 16-byte piece.
          const int d0 = E4M3 ? 16 * (D == 128 ? 2 * t + (k >> 2) : t) + 4 * (k & 3) : 16 * k + 2 * t;
          const int d1 = E4M3 ? d0 + 2 : d0 + 8;
          qf[mt][k][x] = rho < R ? __ldg(src + d0 / 2) : 0u;
          qf[mt][k][2 + x] = rho < R ? __ldg(src + d1 / 2) : 0u;
        }
      }
    }
    float qscale[MT][2];                   // scale_log2, and what scales an fp16 row back
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        qscale[mt][x] = a.scale_log2;
        if constexpr (E4M3) {
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
            top = __vmaxu2(top, __vmaxu2(qf[mt][k][x] & 0x7FFF7FFFu, qf[mt][k][2 + x] & 0x7FFF7FFFu));
          top = max(top & 0xFFFFu, top >> 16);
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          // The largest's exponent field E: times 2^(141 - E), in two steps of normal powers of two.
          const int E = max(static_cast<int>(top >> 7), 1), up = 141 - E, half = up / 2;
          const float f0 = __int_as_float((127 + half) << 23), f1 = __int_as_float((127 + up - half) << 23);
          const float g0 = __int_as_float((127 - half) << 23), g1 = __int_as_float((127 - up + half) << 23);
          qscale[mt][x] = a.scale_log2 * g0 * g1;
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            qf[mt][k][x] = pack_f16x2(bf16lo(qf[mt][k][x]) * f0 * f1, bf16hi(qf[mt][k][x]) * f0 * f1);
            qf[mt][k][2 + x] = pack_f16x2(bf16lo(qf[mt][k][2 + x]) * f0 * f1, bf16hi(qf[mt][k][2 + x]) * f0 * f1);
          }
        }
      }
    }
    float o[MT][kCols][4], m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
    }
    const int p_first = it.q.kv - it.q.c, p_last = it.q.kv - 1;
    // First keys of the first and the last row's windows.
    const int lo_first = a.window != 0 && p_first >= a.window ? p_first - a.window + 1 : 0;
    const int lo_last = a.window != 0 && p_last >= a.window ? p_last - a.window + 1 : 0;

    for (int b = it.b; b < it.end; ++b) {
      const uint32_t bar = bar0 + 8 * slot, tk = ring + slot * S::kStage, tv = tk + S::kTile;
      const int key0 = it.kb.at(b) << kBlockShift;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar, phase, a.status));
      if (!ok) break;
      // ---- S = Q K^T, 16 rows x 16 keys per row tile
      float sc[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[mt][n][e] = 0.f;
      if constexpr (E4M3) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int row = 8 * n + g;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            const uint32_t piece = D == 128 ? (2 * t + h) ^ (row & 7) : t ^ ((row >> 1) & 3);
            const uint4 w = lds128(tk + row * S::kRow + piece * 16);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t b0 = e4m3x2_to_f16x2(ww[x] & 0xFFFFu), b1 = e4m3x2_to_f16x2(ww[x] >> 16);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma_f16(sc[mt][n], qf[mt][4 * h + x], b0, b1);
            }
          }
        }
      } else {
        const int row = (lane & 7) + ((lane >> 4) << 3);
        const uint32_t at = tk + row * 128;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t f[4];
          const int piece = 2 * (k & 3) + ((lane >> 3) & 1);
          ldmatrix_x4(at + (k >> 2) * 2048 + ((piece ^ (row & 7)) << 4), f);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma_bf16(sc[mt][0], qf[mt][k], f[0], f[1]);
            mma_bf16(sc[mt][1], qf[mt][k], f[2], f[3]);
          }
        }
      }
      // ---- softmax of the block
      float kf[2][2], vf[2][2], ve[2][2];  // factors of keys and values, exponents of values
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if constexpr (E4M3) {
          const uint32_t ek = lds_u16(exps + slot * S::kExp + 8 * n + 2 * t);
          const uint32_t ev = lds_u16(exps + slot * S::kExp + 16 + 8 * n + 2 * t);
          kf[n][0] = exp_factor(ek & 255u);
          kf[n][1] = exp_factor(ek >> 8);
          vf[n][0] = exp_factor(ev & 255u);
          vf[n][1] = exp_factor(ev >> 8);
          // byte - 127: the byte in the last bits of 2^23
          ve[n][0] = __uint_as_float(0x4B000000u | (ev & 255u)) - 8388735.f;
          ve[n][1] = __uint_as_float(0x4B000000u | (ev >> 8)) - 8388735.f;
        }
      }
      // Keys that every row sees: no later than the first row, inside the last row's window or all sinks.
      const bool open = key0 + 15 <= p_first && (key0 >= lo_last || key0 + 16 <= a.sinks);
      uint32_t vmask[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
      if (!open) {
        // Values that no row sees (behind the last token, before every window)
        // may be anything: zeros stand in for them.
        auto any = [&](int j) { return j <= p_last && (j >= lo_first || j < a.sinks); };
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int j = key0 + 8 * n + 2 * t;
          vmask[n] = (any(j) ? 0xFFFFu : 0u) | (any(j + 1) ? 0xFFFF0000u : 0u);
        }
      }
      uint32_t pf[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float top[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          top[x] = -INFINITY;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& z = sc[mt][n][2 * x + e];
              z *= E4M3 ? qscale[mt][x] * kf[n][e] : qscale[mt][x];
              if (!open && !sees(a, pos[mt][x], key0 + 8 * n + 2 * t + e)) z = -INFINITY;
              top[x] = fmaxf(top[x], E4M3 ? z + ve[n][e] : z);
            }
          top[x] = fmaxf(top[x], __shfl_xor_sync(0xFFFFFFFFu, top[x], 1));
          top[x] = fmaxf(top[x], __shfl_xor_sync(0xFFFFFFFFu, top[x], 2));
        }
        // The reference is raised (and O rescaled) rarely: weights stay below 2^kLag.
        const bool up0 = top[0] > m[mt][0] + Reference<E4M3>::kLag, up1 = top[1] > m[mt][1] + Reference<E4M3>::kLag;
        if (__any_sync(0xFFFFFFFFu, up0 || up1)) {
          float f[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float old = m[mt][x];
            if (x == 0 ? up0 : up1) m[mt][x] = top[x] - Reference<E4M3>::kLead;
            f[x] = old == m[mt][x] ? 1.f : ex2_approx(old - m[mt][x]);
            l[mt][x] *= f[x];
          }
#pragma unroll
          for (int n = 0; n < kCols; ++n) {
            o[mt][n][0] *= f[0];
            o[mt][n][1] *= f[0];
            o[mt][n][2] *= f[1];
            o[mt][n][3] *= f[1];
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float base = m[mt][x] == -INFINITY ? 0.f : m[mt][x];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float w0 = ex2_approx(sc[mt][n][2 * x] - base), w1 = ex2_approx(sc[mt][n][2 * x + 1] - base);
            l[mt][x] += w0 + w1;
            if constexpr (E4M3) {
              w0 *= vf[n][0];
              w1 *= vf[n][1];
            }
            // The product's operand: weights in 16 bits (their sum stays in fp32).
            pf[mt][2 * n + x] = E4M3 ? pack_f16x2(w0, w1) : pack_bf16x2(w0, w1);
          }
        }
      }
      // ---- O += P V
      if constexpr (E4M3) {
        if (!open) {
          // Such a value's exponent may be the NaN byte: the weight is zero, not NaN.
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x) pf[mt][x] &= vmask[x >> 1];
        }
        uint32_t w[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = 8 * (x >> 1) + 2 * t + (x & 1);
          if constexpr (D == 128) {
            const uint4 v = lds128(tv + row * S::kRow + ((g ^ (row & 7)) << 4));
            w[x][0] = v.x;
            w[x][1] = v.y;
            w[x][2] = v.z;
            w[x][3] = v.w;
          } else {
            const uint2 v = lds64(tv + row * S::kRow + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + 8 * (g & 1));
            w[x][0] = v.x;
            w[x][1] = v.y;
          }
        }
#pragma unroll
        for (int y = 0; y < kCols / 4; ++y) {
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            // Bytes e, e + 1 of both keys' words, side by side per dim.
            const uint32_t sel = e == 0 ? 0x5140u : 0x7362u;
            const uint32_t p0 = __byte_perm(w[0][y], w[1][y], sel), p1 = __byte_perm(w[2][y], w[3][y], sel);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t b0 = e4m3x2_to_f16x2(z == 0 ? p0 & 0xFFFFu : p0 >> 16) & vmask[0];
              const uint32_t b1 = e4m3x2_to_f16x2(z == 0 ? p1 & 0xFFFFu : p1 >> 16) & vmask[1];
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma_f16(o[mt][4 * y + e + z], pf[mt], b0, b1);
            }
          }
        }
      } else {
        const int row = lane & 15;
        const uint32_t at = tv + row * 128;
#pragma unroll
        for (int n = 0; n < kCols; n += 2) {
          uint32_t f[4];
          const int piece = (n & 7) + (lane >> 4);
          ldmatrix_x4_trans(at + (n >> 3) * 2048 + ((piece ^ (row & 7)) << 4), f);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma_bf16(o[mt][n], pf[mt], f[0] & vmask[0], f[1] & vmask[1]);
            mma_bf16(o[mt][n + 1], pf[mt], f[2] & vmask[0], f[3] & vmask[1]);
          }
        }
      }
      __syncwarp();                        // the stage has been read by every lane
      load_next();
      ++used_u;
      if (++slot == S::kStages) {
        slot = 0;
        phase ^= 1;
      }
    }
    if (!ok) break;

    // ---- the item's end: finished here, or a record for the join
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[mt][x] += __shfl_xor_sync(0xFFFFFFFFu, l[mt][x], 1);
        l[mt][x] += __shfl_xor_sync(0xFFFFFFFFu, l[mt][x], 2);
      }
    const bool begun = it.b > 0, whole = !begun && it.end == it.kb.count;
    if (!begun && !whole) {
      const int64_t last = u - it.b + it.kb.count - 1;
      header = SplitHeader{static_cast<int>(share_of(last, W, total) - me) + 1, it.s, it.head, 0};
    }
    float* r = rec.at(me, begun ? 0 : 1);
    uint32_t redo = 0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int rho = 16 * mt + 8 * x + g;
        bool bad = false;
        if (rho < R) {
          const int i = rho / a.group;
          bf16* dst = a.out + (it.q.row0 + i) * a.out_stride + (it.head * a.group + rho - i * a.group) * D;
          const float inv = pos[mt][x] < 0 ? 0.f : 1.f / l[mt][x];
          float* rr = r + rho * D;
          if (!whole && t == 0) {
            rec.max_of(r, D)[rho] = m[mt][x];
            rec.sum_of(r, D)[rho] = l[mt][x];
          }
          // bf16: columns 8n + 2t, + 1.  e4m3: column tile n holds dim n of
          // each lane group's D / 8, so this lane has dims (2t) D/8 + n and (2t + 1) D/8 + n.
          if constexpr (E4M3) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d0 = (2 * t + e) * kCols;
#pragma unroll
              for (int n = 0; n < kCols; n += 4) {
                float4 y = make_float4(o[mt][n][2 * x + e], o[mt][n + 1][2 * x + e], o[mt][n + 2][2 * x + e],
                                       o[mt][n + 3][2 * x + e]);
                if (whole) {
                  y = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
                  bad |= not_finite(y.x) || not_finite(y.y) || not_finite(y.z) || not_finite(y.w);
                  *reinterpret_cast<uint2*>(dst + d0 + n) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
                } else {
                  *reinterpret_cast<float4*>(rr + d0 + n) = y;
                }
              }
            }
          } else {
#pragma unroll
            for (int n = 0; n < kCols; ++n) {
              const float y0 = o[mt][n][2 * x], y1 = o[mt][n][2 * x + 1];
              if (whole) {
                bad |= not_finite(y0 * inv) || not_finite(y1 * inv);
                *reinterpret_cast<uint32_t*>(dst + 8 * n + 2 * t) = pack_bf16x2(y0 * inv, y1 * inv);
              } else {
                *reinterpret_cast<float2*>(rr + 8 * n + 2 * t) = make_float2(y0, y1);
              }
            }
          }
        }
        if (it.q.c > 1) {
          const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, bad);
#pragma unroll
          for (int y = 0; y < 8; ++y)
            if ((lanes >> (4 * y)) & 15u) redo |= 1u << (16 * mt + 8 * x + y);
        }
      }
    }
    while (redo) {
      __syncwarp();
      const int rho = __ffs(static_cast<int>(redo)) - 1;
      redo &= redo - 1;
      const int i = rho / a.group;
      exact_row<D, E4M3>(a, it.s, it.q.row0, it.q.kv - it.q.c + i, i, it.head * a.group + rho - i * a.group, lane);
    }
    u += it.end - it.b;
  }
  // After a timeout: wait (bounded) for the loads still in flight.
  for (; !ok && used_u < load_u; ++used_u) {
    if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar0 + 8 * slot, phase, nullptr))) break;
    if (++slot == S::kStages) {
      slot = 0;
      phase ^= 1;
    }
  }
  if (lane == 0) rec.headers[me] = ok ? header : SplitHeader{0, 0, 0, 0};
}

int decode_workers() { return num_sms() * kWarps; }

template <int D, bool E4M3, int MT>
int launch(const AttentionArgs& a, void* ws, cudaStream_t stream) {
  using S = Shape<D, E4M3>;
  CUtensorMap tk, tv;
  const uint64_t rows = static_cast<uint64_t>(a.c.n_pages) * a.c.kv_heads << a.c.page_shift;
  const uint64_t cols = S::kRow / 2;      // in 16-bit units
  auto map = [&](CUtensorMap* m, const void* p) {
    return cols == 32 ? make_tmap_bf16_sw64(m, p, rows, cols, 16) : make_tmap_bf16(m, p, rows, cols, 16);
  };
  if (!map(&tk, a.c.k) || !map(&tv, a.c.v)) return DS_VIT_ECUDA;
  if (allow_smem(reinterpret_cast<const void*>(decode_kernel<D, E4M3, MT>), S::kSmem) != cudaSuccess)
    return DS_VIT_ECUDA;
  const int R = a.b.max_rows * a.group, grid = num_sms();
  const Records rec = records_in(ws, decode_workers(), R, D);
  cudaError_t e = launch_pdl(decode_kernel<D, E4M3, MT>, dim3(grid), dim3(kThreads), S::kSmem, stream, tk, tv, a, rec);
  if (e == cudaSuccess)
    e = launch_pdl(join_kernel<D, E4M3>, dim3(grid, R), dim3(32 * kJoinWarps), 0, stream, a, rec, decode_workers());
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? DS_VIT_OK : DS_VIT_ECUDA;
}

}  // namespace

size_t cache_decode_workspace(int head_dim, int rows) { return records_bytes(decode_workers(), rows, head_dim); }

int launch_cache_decode(const AttentionArgs& a, int head_dim, bool e4m3, void* ws, cudaStream_t stream) {
  const int R = a.b.max_rows * a.group;
  if (R > kDecodeRows) return DS_VIT_EINVAL;
  if (head_dim == 128) {
    if (R <= 16) return e4m3 ? launch<128, true, 1>(a, ws, stream) : launch<128, false, 1>(a, ws, stream);
    return e4m3 ? launch<128, true, 2>(a, ws, stream) : launch<128, false, 2>(a, ws, stream);
  }
  if (R <= 16) return e4m3 ? launch<64, true, 1>(a, ws, stream) : launch<64, false, 1>(a, ws, stream);
  return e4m3 ? launch<64, true, 2>(a, ws, stream) : launch<64, false, 2>(a, ws, stream);
}

}  // namespace dsvit
