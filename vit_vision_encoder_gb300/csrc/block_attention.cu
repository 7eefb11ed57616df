// Attention over the blocks of a paged cache that each row lists
// (include/dsvit.h, ds_vit_cache_attention_blocks).
//
// Every row and K/V head has keys of its own, which the 8 or so query heads of the group
// share: 2 * 8 flops a byte of bf16.  There is nothing for a CTA's warps to share and no use for a tile
// larger than the group, so keys and values go from the pages straight into
// registers as fragments of warp MMAs (m16n8k16), 16 keys at a time, with no
// shared memory and nobody to wait for:
//   S^T = K Q^T:  16 keys in the place of M, 8 query heads in that of N (the usual order would
//                 leave half of M empty);
//   O^T += V^T P^T: dims in the place of M.  P^T comes out of S^T's accumulators by a transposing
//                 move between lanes (movmatrix).
// The order of dims inside a product is free as long as both sides share it, and so
// are the order of keys and that of output rows, so each lane uses what it loads where it lies; values, of
// which a product pairs keys, are loaded by whole lines (eight lanes a key) and passed on between
// lanes, since a load in which neighbouring lanes read different keys takes L1 a cycle for each.
// The next tile's keys are loaded behind the scores' products, its values behind the outputs'.
//
// What bounds it, 40 query and 8 K/V heads of 128:
//   rows of different sequences, by memory: 48 rows over 4096 tokens each, bf16, 122 us (97% of the rate of a
//   plain copy); e4m3, 84 us (71%): twelve warps an SM have 48 KB in flight, and conversions come on top.
//   Sixteen warps with the queries in shared memory 95, with the next values in registers too 84.
//   rows of one prompt, by the SM itself: 2048 rows over 1024 tokens each, e4m3, 493 us, bf16 579 to 603; all rows over
//   one block, which L1 then holds, 475 and 541.  316 instructions a tile of 16 keys, more than half of them in the ALU
//   (conversions, masks, addresses), and L1's data path (with values read as the products want them
//   503 and 687).  Two tiles a step (604), four CTAs an SM (529) and scores from e4m3 MMAs with the queries in
//   two parts (579) were slower.
//
// Work: an item is a row, a K/V head and up to 8 (16) of its query heads.  One warp takes
// an item while there are enough of them; with fewer, up to 4 warps of a CTA, then the
// CTAs of a cluster, take its tiles in turn and join their sums through (distributed)
// shared memory in a fixed order.  One launch, no workspace.
//
// Weights are rounded where they meet the values, as in the dense attention: to bf16, 2^-8 of each at most, over bf16
// pages, whose type the product has to share, and to fp16 over e4m3 pages, whose values widen to it exactly.  Their sum
// takes them whole, in fp32.  Measured beside 64 bits, of the outputs' norm: 48 single rows over bf16 pages 0.0023, where
// weights in fp32 give 0.0017 from the outputs' rounding alone; e4m3 0.0017.
//
// e4m3: keys widen exactly to fp16, queries are scaled to at most 2^15 by a power of two;
// the softmax multiplies by each key's factor.  Values widen to fp16, and the weights that meet them
// carry the values' exponents against a reference r of their own, that of the contributions
// (score + exponent), while the weights' sum refers to the scores' maximum m.
#include <algorithm>

#include "cache.cuh"

namespace dsvit {

namespace {

struct BlockArgs {
  CacheView c;
  ChunkView b;
  const bf16* q;
  int64_t q_stride;
  bf16* out;
  int64_t out_stride;
  int group, head_tiles;     // query heads per K/V head; items that share them
  float scale_log2;
  const int32_t* blocks;
  int64_t row_stride, head_stride;
  int top;
  int* status;
  int64_t items;
  bool wide;                 // keys begin on 32-byte boundaries
  int warp_shift;            // warps of a CTA per item: 1 << warp_shift
};

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kLag16 = 8.f;                    // bf16: a reference is raised when it is passed by this (log2)
constexpr float kLag8 = 14.f, kLead8 = 6.f;      // e4m3: fp16 weights in (0, 2^14], 2^6 after a raise

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr));
  return x;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(addr));
  return x;
}

// A reference before anything has been seen: every finite score is at or above it.
constexpr float kNone = -3.402823466e38f;

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 32 bytes by one load.
__device__ __forceinline__ void ldg256(const uint4* from, uint4& a, uint4& b) {
  asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
      : "l"(from));
}

// The two e4m3 values in the upper half of a register as fp16.
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t four) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(four));
  return r;
}

template <int D, bool E4M3, int NT>
struct Frag {
  static constexpr int kK = E4M3 ? D / 64 : D / 32;      // 16-byte pieces of a key that a lane holds
  static constexpr int kV = D == 128 && !E4M3 ? 2 : 1;   // pieces of a value
  static constexpr int kM = D / 16;                      // row tiles of the output
  // The first 16 bytes of a key are piece 0 of lane group member t = 0; pieces 2i and 2i + 1 of a lane lie side by side.
  static __device__ __forceinline__ int piece(int t, int j) { return kK == 1 ? t : 8 * (j >> 1) + 2 * t + (j & 1); }
  // A dim of accumulator row tile m, rows g and g + 8, of lane group g.
  static __device__ __forceinline__ int dim(int g, int m, int half) {
    return kV == 2 ? 64 * half + 8 * g + m : (D / 8) * g + 2 * m + half;
  }
};

// A warp's sums of an item, in shared memory: outputs of head n at n * (D + 4), then m, r, l of each head.
template <int D, int NT>
struct Record {
  static constexpr int kHeads = 8 * NT, kPitch = D + 4, kM = kHeads * kPitch, kR = kM + kHeads, kL = kR + kHeads,
                       kSeen = kL + kHeads, kFloats = kSeen + 4;
};

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kThreads, NT == 2 ? 2 : D == 128 ? 3 : 4) block_attention_kernel(const __grid_constant__ BlockArgs a) {
  using F = Frag<D, E4M3, NT>;
  using R = Record<D, NT>;
  constexpr int kK = F::kK, kV = F::kV, kM = F::kM, kChains = 2;
  __shared__ __align__(16) float records[kWarps][R::kFloats];
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  uint32_t rank = cluster_rank(), ranks;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int sub = warp & ((1 << a.warp_shift) - 1);
  const int64_t item = (static_cast<int64_t>(blockIdx.x / ranks) << (2 - a.warp_shift)) + (warp >> a.warp_shift);
  const int sharers = static_cast<int>(ranks) << a.warp_shift, me = (static_cast<int>(rank) << a.warp_shift) + sub;

  // The item: neighbouring warps have neighbouring rows of one K/V head.
  int64_t row = 0;
  int kv_head = 0, head0 = 0, heads = 0, s = -1, p = -1;
  bool mine = item < a.items;
  if (mine) {
    const int64_t tile = item / a.b.rows;
    row = item - tile * a.b.rows;
    kv_head = static_cast<int>(tile / a.head_tiles);
    head0 = static_cast<int>(tile - static_cast<int64_t>(kv_head) * a.head_tiles) * 8 * NT;
    heads = min(8 * NT, a.group - head0);
    head0 += kv_head * a.group;
    s = find_seq(a.b, static_cast<int>(row), lane);
    const Seq q = s < 0 ? Seq{0, 0, 0} : load_seq(a.b, a.c.page_shift, s, a.status);
    const int i = static_cast<int>(row) - q.row0;
    mine = static_cast<unsigned>(i) < static_cast<unsigned>(q.c);
    p = mine ? q.kv - q.c + i : -1;
  }

  // Queries, B fragments of S^T: lane (g, t) has of head g what it has of a key.
  uint32_t qf[NT][kK][E4M3 ? 8 : 4];
  float unit[NT][2];                       // what an accumulated score of heads 2t, 2t + 1 counts (log2)
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const bool on = mine && 8 * n + g < heads;
    const uint4* from = reinterpret_cast<const uint4*>(a.q + row * a.q_stride + static_cast<int64_t>(head0 + 8 * n + g) * D);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if constexpr (!E4M3) {
#pragma unroll
      for (int j = 0; j < kK; ++j) {
        const uint4 u = on ? __ldg(from + F::piece(t, j)) : zero;
        qf[n][j][0] = u.x, qf[n][j][1] = u.y, qf[n][j][2] = u.z, qf[n][j][3] = u.w;
      }
    } else {
      uint4 u[kK][2];
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < kK; ++j)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          u[j][y] = on ? __ldg(from + 2 * F::piece(t, j) + y) : zero;
          const uint32_t m = __vmaxu2(__vmaxu2(u[j][y].x & 0x7FFF7FFFu, u[j][y].y & 0x7FFF7FFFu),
                                      __vmaxu2(u[j][y].z & 0x7FFF7FFFu, u[j][y].w & 0x7FFF7FFFu));
          top = max(top, max(m & 0xFFFFu, m >> 16));
        }
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      // The largest magnitude to [2^14, 2^15): exponent field E to 141.  Infinities and NaN stay.
      const int E = min(max(static_cast<int>(top >> 7), 15), 254);
      const float f = __int_as_float((268 - E) << 23);
      const float undo = __int_as_float((E - 14) << 23);
#pragma unroll
      for (int j = 0; j < kK; ++j)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t w[4] = {u[j][y].x, u[j][y].y, u[j][y].z, u[j][y].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) qf[n][j][4 * y + x] = pack_f16x2(bf16lo(w[x]) * f, bf16hi(w[x]) * f);
        }
      unit[n][0] = fminf(__shfl_sync(0xFFFFFFFFu, undo, 8 * t) * a.scale_log2, 3e38f);
      unit[n][1] = fminf(__shfl_sync(0xFFFFFFFFu, undo, 8 * t + 4) * a.scale_log2, 3e38f);
    }
  }

  float m[NT][2], r[NT][2], l[NT][2], acc[NT][kM][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int x = 0; x < 2; ++x) m[n][x] = r[n][x] = kNone, l[n][x] = 0.f;
#pragma unroll
    for (int y = 0; y < kM; ++y)
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[n][y][x] = 0.f;
  }
  bool seen = false;

  // The list, 32 entries at a time: a lane has one entry's block and page.
  const int tile_shift = a.c.page_shift - 4;
  const int32_t* const list = a.blocks + row * a.row_stride + kv_head * a.head_stride;
  int base = 0, block = -1, at = -1;
  auto window = [&](int e0) {
    base = e0;
    const int e = e0 + lane;
    block = e < a.top ? __ldg(list + e) : -1;
    if (static_cast<unsigned>(block) > static_cast<unsigned>(p >> a.c.page_shift)) block = -1;
    at = -1;
    if (block >= 0) {
      at = __ldg(a.b.table + static_cast<int64_t>(s) * a.b.table_cols + block);
      if (!page_there(at, a.c.n_pages)) {
        report_error(a.status, DS_VIT_ERANGE);
        at = -1;
      }
    }
  };
  // The next tile of this warp's: its first row in the pages and its keys (0: none is left).
  const int tiles = p < 0 ? 0 : a.top << tile_shift;
  int x_next = me;
  int64_t row0 = 0;
  auto next = [&]() {
    while (x_next < tiles) {
      const int x = x_next, e = x >> tile_shift;
      x_next += sharers;
      if (e >= base + 32) window(e & ~31);
      const int from = e - base;
      const int page = __shfl_sync(0xFFFFFFFFu, at, from), blk = __shfl_sync(0xFFFFFFFFu, block, from);
      if (page < 0) continue;
      const int off = (x & ((1 << tile_shift) - 1)) * 16;
      const int n = min(p + 1 - (blk << a.c.page_shift) - off, 16);
      if (n <= 0) continue;
      row0 = cache_row(a.c, page, kv_head, off);
      return n;
    }
    return 0;
  };

  constexpr int kRow = E4M3 ? D : 2 * D;      // bytes of a key
  // Rows g and g + 8 of the scores are keys key0 and key0 + 8, so that their rows 2t, 2t + 1, 8 + 2t and 9 + 2t are
  // keys t, t + 4, t + 8 and t + 12: whose values lane group member t is given (below).
  const int key0 = (g >> 1) + 4 * (g & 1);
  uint4 k[2][kK];
  uint4 v[4][kV];                             // e4m3 at D 64: 8 bytes of each
  uint32_t kb[2], vb[2];                      // exponents of keys key0, key0 + 8
  // Whole tiles, all but the last of a row's own block, are loaded without conditions.
  const uint8_t* const k_lane = a.c.k + key0 * kRow + 16 * F::piece(t, 0);
  // Values: eight lanes read a line of one key; what lane (g, t) needs of key 4y + t is with lane 8t + g.
  const uint8_t* const v_lane = a.c.v + (lane >> 3) * kRow + (E4M3 && D == 64 ? 8 : 16) * (lane & 7);
  const int v_from = 8 * t + g;
  auto load_k = [&](int64_t r0, int n) {
    auto load = [&](bool whole, auto on) {
      const uint8_t* const from = k_lane + r0 * kRow;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint4* const at_y = reinterpret_cast<const uint4*>(from + 8 * y * kRow);
        if (kK > 1 && whole && a.wide) {
#pragma unroll
          for (int j = 0; j + 1 < kK; j += 2) ldg256(at_y + 4 * j, k[y][j], k[y][j + 1]);
        } else {
#pragma unroll
          for (int j = 0; j < kK; ++j) k[y][j] = on(key0 + 8 * y) ? __ldg(at_y + F::piece(0, j)) : make_uint4(0, 0, 0, 0);
        }
        if constexpr (E4M3) {
          kb[y] = on(key0 + 8 * y) ? __ldg(a.c.k_exp + r0 + key0 + 8 * y) : 127u;
          vb[y] = on(key0 + 8 * y) ? __ldg(a.c.v_exp + r0 + key0 + 8 * y) : 127u;
        }
      }
    };
    if (n == 16)
      load(true, [](int) { return true; });
    else
      load(false, [n](int key) { return key < n; });
  };
  auto load_v = [&](int64_t r0, int n) {
    auto load = [&](auto on) {
      const uint8_t* const from = v_lane + r0 * kRow;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const bool here = on(4 * y + (lane >> 3));
        if constexpr (E4M3 && D == 64) {
          const uint2 u = here ? __ldg(reinterpret_cast<const uint2*>(from + 4 * y * kRow)) : make_uint2(0, 0);
          v[y][0] = make_uint4(u.x, u.y, 0, 0);
        } else {
#pragma unroll
          for (int z = 0; z < kV; ++z)
            v[y][z] = here ? __ldg(reinterpret_cast<const uint4*>(from + 4 * y * kRow) + 8 * z) : make_uint4(0, 0, 0, 0);
        }
      }
    };
    if (n == 16)
      load([](int) { return true; });
    else
      load([n](int key) { return key < n; });
  };
  auto word = [](const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; };

  if (tiles > 0) window(0);
  int n_keys = next();
  if (n_keys > 0) {
    load_k(row0, n_keys);
    load_v(row0, n_keys);
  }
  while (n_keys > 0) {
    seen = true;
    const int n_here = n_keys;
    // Products that follow one another into the same sum wait for each other: kChains sums.
    float part[kChains][NT][4];
#pragma unroll
    for (int i = 0; i < kChains; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) part[i][n][0] = part[i][n][1] = part[i][n][2] = part[i][n][3] = 0.f;
#pragma unroll
    for (int j = 0; j < kK; ++j) {
      if constexpr (E4M3) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t k0 = word(k[0][j], x), k1 = word(k[1][j], x);
          const uint32_t af[4] = {e4m3x2_to_f16x2(k0), e4m3x2_to_f16x2(k1), e4m3x2_hi_to_f16x2(k0), e4m3x2_hi_to_f16x2(k1)};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(part[x % kChains][n], af, qf[n][j][2 * x], qf[n][j][2 * x + 1]);
        }
      } else {
        const uint32_t a0[4] = {k[0][j].x, k[1][j].x, k[0][j].y, k[1][j].y};
        const uint32_t a1[4] = {k[0][j].z, k[1][j].z, k[0][j].w, k[1][j].w};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_bf16(part[2 * j % kChains][n], a0, qf[n][j][0], qf[n][j][1]);
          mma_bf16(part[(2 * j + 1) % kChains][n], a1, qf[n][j][2], qf[n][j][3]);
        }
      }
    }
    float c[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        c[n][x] = part[0][n][x];
#pragma unroll
        for (int i = 1; i < kChains; ++i) c[n][x] += part[i][n][x];
      }
    float kf[2] = {1.f, 1.f}, ve[2] = {0.f, 0.f};
    if constexpr (E4M3) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        kf[y] = exp_factor(kb[y]);
        ve[y] = vb[y] == 255u ? __int_as_float(0x7FC00000) : static_cast<float>(static_cast<int>(vb[y]) - 127);
      }
    }
    n_keys = next();
    if (n_keys > 0) load_k(row0, n_keys);

    // Scores (log2) of keys key0 (0, 1) and key0 + 8 (2, 3), heads 2t and 2t + 1.
    bool raise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        // (0 times a factor past all floats stays 0, NaN stays.)
        float z = c[n][x] * (E4M3 ? min_nan(kf[x >> 1] * unit[n][x & 1], 3e38f) : a.scale_log2);
        if (n_here < 16 && key0 + 8 * (x >> 1) >= n_here) z = -INFINITY;
        c[n][x] = z;
        raise |= z > m[n][x & 1] + (E4M3 ? kLag8 : kLag16);
        if constexpr (E4M3) raise |= z + ve[x >> 1] > r[n][x & 1] + kLag8;
      }
    if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float top = fmaxf(c[n][x], c[n][x + 2]), most = fmaxf(c[n][x] + ve[0], c[n][x + 2] + ve[1]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            if constexpr (E4M3) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
          }
          const float to = fmaxf(m[n][x], top), lf = ex2_approx(m[n][x] - to);
          float of = lf;
          if constexpr (E4M3) {
            // Contributions may lie up to kLag8 over their reference: it moves when one is further up.
            const float ref = most > r[n][x] + kLag8 ? most - kLead8 : r[n][x];
            of = ex2_approx(r[n][x] - ref);
            r[n][x] = ref;
          }
          m[n][x] = to;
          l[n][x] *= lf;
#pragma unroll
          for (int y = 0; y < kM; ++y) {
            acc[n][y][x] *= of;
            acc[n][y][x + 2] *= of;
          }
        }
    }
    uint32_t pf[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float y = ex2_approx(c[n][x] - m[n][x & 1]);
        l[n][x & 1] += y;
        w[x] = E4M3 ? ex2_approx(c[n][x] + ve[x >> 1] - r[n][x & 1]) : y;
      }
      pf[n][0] = transposed(E4M3 ? pack_f16x2(w[0], w[1]) : pack_bf16x2(w[0], w[1]));
      pf[n][1] = transposed(E4M3 ? pack_f16x2(w[2], w[3]) : pack_bf16x2(w[2], w[3]));
    }
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
      for (int z = 0; z < kV; ++z) {
        v[y][z].x = __shfl_sync(0xFFFFFFFFu, v[y][z].x, v_from);
        v[y][z].y = __shfl_sync(0xFFFFFFFFu, v[y][z].y, v_from);
        if constexpr (!E4M3 || D != 64) {
          v[y][z].z = __shfl_sync(0xFFFFFFFFu, v[y][z].z, v_from);
          v[y][z].w = __shfl_sync(0xFFFFFFFFu, v[y][z].w, v_from);
        }
      }
#pragma unroll
    for (int y = 0; y < kM; ++y) {
      uint32_t af[4];
      if constexpr (E4M3) {
        const uint32_t sel = y & 1 ? 0x7362u : 0x5140u;
        const uint32_t u0 = __byte_perm(word(v[0][0], y >> 1), word(v[1][0], y >> 1), sel);
        const uint32_t u1 = __byte_perm(word(v[2][0], y >> 1), word(v[3][0], y >> 1), sel);
        af[0] = e4m3x2_to_f16x2(u0), af[1] = e4m3x2_hi_to_f16x2(u0);
        af[2] = e4m3x2_to_f16x2(u1), af[3] = e4m3x2_hi_to_f16x2(u1);
      } else if constexpr (kV == 2) {
        const uint32_t sel = y & 1 ? 0x7632u : 0x5410u;
        af[0] = __byte_perm(word(v[0][0], y >> 1), word(v[1][0], y >> 1), sel);
        af[1] = __byte_perm(word(v[0][kV - 1], y >> 1), word(v[1][kV - 1], y >> 1), sel);
        af[2] = __byte_perm(word(v[2][0], y >> 1), word(v[3][0], y >> 1), sel);
        af[3] = __byte_perm(word(v[2][kV - 1], y >> 1), word(v[3][kV - 1], y >> 1), sel);
      } else {
        af[0] = __byte_perm(word(v[0][0], y), word(v[1][0], y), 0x5410u);
        af[1] = __byte_perm(word(v[0][0], y), word(v[1][0], y), 0x7632u);
        af[2] = __byte_perm(word(v[2][0], y), word(v[3][0], y), 0x5410u);
        af[3] = __byte_perm(word(v[2][0], y), word(v[3][0], y), 0x7632u);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (E4M3)
          mma_f16(acc[n][y], af, pf[n][0], pf[n][1]);
        else
          mma_bf16(acc[n][y], af, pf[n][0], pf[n][1]);
      }
    }
    if (n_keys > 0) load_v(row0, n_keys);
  }

#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[n][x] += __shfl_xor_sync(0xFFFFFFFFu, l[n][x], o);

  bf16* const out = a.out + row * a.out_stride + static_cast<int64_t>(head0) * D;
  // The sum of an item, o at reference r over l at reference m; zeros where nothing was seen.
  auto factors = [](float mm, float rr, float ll, bool any, float& f0, float& f1) {
    f0 = any ? 1.f / ll : 0.f;
    f1 = E4M3 && any ? ex2_approx(0.5f * (rr - mm)) : 1.f;      // twice: 2^(r - m) may be no float
  };
  if (sharers == 1) {
    if (!mine) return;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int h = 8 * n + 2 * t + x;
        float f0, f1;
        factors(m[n][x], r[n][x], l[n][x], seen, f0, f1);
        float o[2][kM];
#pragma unroll
        for (int y = 0; y < kM; ++y) {
          o[0][y] = seen ? acc[n][y][x] * f0 * f1 * f1 : 0.f;
          o[1][y] = seen ? acc[n][y][x + 2] * f0 * f1 * f1 : 0.f;
        }
        if (h >= heads) continue;
        uint4* to = reinterpret_cast<uint4*>(out + h * D);
        if constexpr (kV == 2) {
#pragma unroll
          for (int z = 0; z < 2; ++z)
            to[8 * z + g] = make_uint4(pack_bf16x2(o[z][0], o[z][1]), pack_bf16x2(o[z][2], o[z][3]),
                                       pack_bf16x2(o[z][4], o[z][5]), pack_bf16x2(o[z][6], o[z][7]));
        } else {
#pragma unroll
          for (int z = 0; z < kM / 4; ++z)
            to[(kM / 4) * g + z] =
                make_uint4(pack_bf16x2(o[0][4 * z], o[1][4 * z]), pack_bf16x2(o[0][4 * z + 1], o[1][4 * z + 1]),
                           pack_bf16x2(o[0][4 * z + 2], o[1][4 * z + 2]), pack_bf16x2(o[0][4 * z + 3], o[1][4 * z + 3]));
        }
      }
    return;
  }

  float* rec = records[warp];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int h = 8 * n + 2 * t + x;
#pragma unroll
      for (int y = 0; y < kM; ++y) {
        rec[h * R::kPitch + F::dim(g, y, 0)] = acc[n][y][x];
        rec[h * R::kPitch + F::dim(g, y, 1)] = acc[n][y][x + 2];
      }
      if (g == 0) {
        rec[R::kM + h] = m[n][x];
        rec[R::kR + h] = E4M3 ? r[n][x] : m[n][x];
        rec[R::kL + h] = l[n][x];
      }
    }
  if (lane == 0) rec[R::kSeen] = seen ? 1.f : 0.f;
  if (ranks > 1)
    cluster_sync();
  else
    __syncthreads();
  if (mine) {
    // Four outputs a thread, the item's threads in all CTAs; records in the order of the sharers.
    const uint32_t first = smem_u32(records[warp - sub]);
    constexpr uint32_t kBytes = R::kFloats * 4;
    for (int w = 32 * me + lane; w < heads * (D / 4); w += 32 * sharers) {
      const int h = w / (D / 4), d = 4 * (w - h * (D / 4));
      float mm = kNone, rr = kNone;
      bool any = false;
      auto part = [&](int y) {
        return mapa_shared(first + (y & ((1 << a.warp_shift) - 1)) * kBytes, y >> a.warp_shift);
      };
#pragma unroll 4
      for (int y = 0; y < sharers; ++y) {
        const uint32_t at_y = part(y);
        mm = fmaxf(mm, ld_cluster(at_y + 4 * (R::kM + h)));
        rr = fmaxf(rr, ld_cluster(at_y + 4 * (R::kR + h)));
        any |= ld_cluster(at_y + 4 * R::kSeen) != 0.f;
      }
      float ll = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int y = 0; y < sharers; ++y) {
        const uint32_t at_y = part(y);
        const float lf = ex2_approx(ld_cluster(at_y + 4 * (R::kM + h)) - mm);
        const float of = ex2_approx(ld_cluster(at_y + 4 * (R::kR + h)) - rr);
        const float4 oy = ld_cluster4(at_y + 4 * (h * R::kPitch + d));
        // A part that saw nothing has the lowest references, and zeros.
        ll = fmaf(ld_cluster(at_y + 4 * (R::kL + h)), lf, ll);
        o.x = fmaf(oy.x, of, o.x), o.y = fmaf(oy.y, of, o.y), o.z = fmaf(oy.z, of, o.z), o.w = fmaf(oy.w, of, o.w);
      }
      float f0, f1;
      factors(mm, rr, ll, any, f0, f1);
      uint2 u = make_uint2(0, 0);
      if (any) {
        u.x = pack_bf16x2(o.x * f0 * f1 * f1, o.y * f0 * f1 * f1);
        u.y = pack_bf16x2(o.z * f0 * f1 * f1, o.w * f0 * f1 * f1);
      }
      *reinterpret_cast<uint2*>(out + h * D + d) = u;
    }
  }
  if (ranks > 1) cluster_sync();         // the others have read this CTA's records
}

template <int D, bool E4M3>
int launch_blocks(BlockArgs a, void* stream) {
  const int nt = a.group > 8 ? 2 : 1;
  a.head_tiles = (a.group + 8 * nt - 1) / (8 * nt);
  a.items = static_cast<int64_t>(a.b.rows) * a.c.kv_heads * a.head_tiles;
  // Warps that share an item: as many as fill the SMs with twelve each, of two tiles at least.
  const int64_t room = (nt == 2 ? 24 : 12) * static_cast<int64_t>(num_sms());
  const int tiles = a.top << (a.c.page_shift - 4);
  int sharers = 1;
  while (sharers < 8 * kWarps && 2 * sharers * a.items <= room && 4 * sharers <= tiles) sharers *= 2;
  while (1 << a.warp_shift < std::min(sharers, kWarps)) ++a.warp_shift;
  const int ranks = std::max(sharers / kWarps, 1);
  const int64_t per_cta = kWarps >> a.warp_shift;
  const int64_t ctas = (a.items + per_cta - 1) / per_cta * ranks;
  if (ctas > INT32_MAX) return DS_VIT_ERANGE;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
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
  auto* fn = nt == 2 ? block_attention_kernel<D, E4M3, 2> : block_attention_kernel<D, E4M3, 1>;
  return launched(cudaLaunchKernelEx(&cfg, fn, a));
}

}  // namespace

}  // namespace dsvit

using namespace dsvit;

extern "C" int ds_vit_cache_attention_blocks(const ds_vit_cache* cache, const ds_vit_chunks* chunks, const void* q,
                                             int64_t q_stride, int64_t rows, int32_t heads, float scale,
                                             const int32_t* blocks, int64_t row_stride, int64_t head_stride,
                                             int32_t top, void* out, int64_t out_stride, int32_t* status,
                                             void* stream) {
  BlockArgs a{};
  if (const int rc = check_cache(cache, chunks, rows, &a.c, &a.b)) return rc;
  if (heads < 1 || heads % a.c.kv_heads != 0 || heads / a.c.kv_heads > DS_VIT_CACHE_MAX_GROUP || !(scale > 0.f) ||
      !(scale <= 1e30f) || top < 1 || top > DS_VIT_SELECT_MAX_TOP ||
      bad_lists(blocks, row_stride, head_stride, rows, a.c.kv_heads, top))
    return DS_VIT_EINVAL;
  const int64_t width = static_cast<int64_t>(heads) * cache->head_dim;
  if (!status || !aligned(status, 4) || bad_rows(q, q_stride, width) || bad_rows(out, out_stride, width))
    return DS_VIT_EINVAL;
  if (rows > INT32_MAX / heads) return DS_VIT_ERANGE;
  if (rows == 0) return DS_VIT_OK;
  a.q = static_cast<const bf16*>(q);
  a.q_stride = q_stride;
  a.out = static_cast<bf16*>(out);
  a.out_stride = out_stride;
  a.group = heads / a.c.kv_heads;
  a.scale_log2 = 1.4426950408889634f * scale;
  a.blocks = blocks;
  a.row_stride = row_stride;
  a.head_stride = head_stride;
  a.top = top;
  a.status = reinterpret_cast<int*>(status);
  a.wide = aligned(cache->k, 32);
  const bool e4m3 = cache->kind == DS_VIT_CACHE_E4M3;
  return cache->head_dim == 128 ? (e4m3 ? launch_blocks<128, true>(a, stream) : launch_blocks<128, false>(a, stream))
                                : (e4m3 ? launch_blocks<64, true>(a, stream) : launch_blocks<64, false>(a, stream));
}
