// Attention over the paged cache for few rows, as in decoding: the query rows
// that share a K/V head (new tokens times query heads per K/V head) are taken
// 16 at a time, up to decode_rows of them.
//
// Bound by the cache's bytes: each key and value read meets at most 16 rows, 32
// flops a byte of bf16, a twentieth of the tensor rate the bytes could feed.  So the
// products run as warp MMAs (m16n8k16), whose fragments come straight from shared
// memory; what counts is bytes in flight and a short chain of instructions per key.
// Measured at 40 query and 8 K/V heads of 128: 32 sequences of 400 to 16000 tokens,
// bf16, 88 us (5.7 TB/s; the loads alone 85); 64 of 2000 to 30000, e4m3, 224 us (6.1
// TB/s, the loads alone 216: the rest is conversions and products of twice the keys
// a byte); one of 1500 tokens 11.8 us, three quarters of it fixed (launches, plan, join).
//
// Work: the unit is a block of kKeys keys of one item (sequence, K/V head, 16
// rows).  All units of a call are counted from the lengths on the device and dealt in
// order to the workers, the consumer warps of the grid, in equal shares
// (cache_plan.h), so a batch of unequal lengths and a single long sequence both
// keep every SM reading.  A worker streams its blocks through its own ring of
// TMA tiles with its own running softmax; consumer warps never wait for one
// another.  One producer warp per CTA fills the rings, lane i that of warp i
// (issued by the consumers themselves, the loads took 660 of the 2260 cycles a
// block of 16 keys cost a warp).  bf16: a consumer takes a stage's fragments into
// registers at once and gives the stage back before it computes.  Items that
// lie within one worker's share are finished there, the others leave records
// that join_kernel adds up.
//
// bf16: blocks of 16 keys (inside one page); S = Q K^T with K fragments by
// ldmatrix, P V with V fragments by ldmatrix.trans.  e4m3: blocks of 32 keys (64 at
// head dim 64: 660 thousand tokens 137 us, 208 in blocks of 32); a
// lane loads 16 bytes of a key (16 dims) or of two values' rows and widens
// pairs to fp16 in registers (one conversion a pair, exact; bf16 has no such
// conversion, and bit operations to the same end took five instructions a
// pair).  The order of dims within a product is free as long as both operands
// share it, and so is the order of output columns, so a lane's bytes are used
// where they lie.  fp16's range is kept by powers of two: each query row is
// scaled to a largest magnitude in [2^14, 2^15) (the scores are scaled back),
// and the weights carry the values' exponents and are taken against the running
// maximum of score plus exponent, the size of a key's contribution, so that the
// largest stay in [2^6, 2^14]; contributions under 2^-20 of the largest lose
// bits.  The weights' sum has a reference of its own (Raise in cache_rows.cuh).
#include "cache_rows.cuh"

#include <algorithm>

namespace dsvit {

namespace {

// bf16: a row's reference m (log2) is raised when a block's maximum passes m + kLag16, to
// that maximum; weights are 2^(z - m).  e4m3: Raise in cache_rows.cuh.
constexpr float kLag16 = 8.f;

template <int D, bool E4M3>
struct Shape {
  // Consumer warps: with the producer a multiple of four, and as many registers
  // as the fragments need (D 128: 255 each).
  static constexpr int kWarps = D == 64 ? 11 : 7;
  static constexpr int kThreads = 32 * kWarps + 32;
  static constexpr int kRingBytes = (D == 64 ? 16 : 24) * 1024;      // per consumer warp
  static constexpr int kKeyShift = E4M3 ? (D == 64 ? 6 : 5) : 4;
  static constexpr int kKeys = 1 << kKeyShift;             // keys of a block
  static constexpr int kRow = E4M3 ? D : 2 * D;            // bytes of a key
  static constexpr int kTile = kKeys * kRow;
  static constexpr int kPlane = kKeys * 128;               // bf16, D = 128: two planes of 64 dims
  static constexpr int kStage = 2 * kTile;                 // K, then V
  static constexpr int kStages = kRingBytes / kStage;
  static constexpr int kExp = E4M3 ? 2 * kKeys : 0;        // exponents of a stage: K, then V
  static constexpr int kPieces = kKeys / 16;               // pages of a block at most
  static constexpr int kSmem = 1024 + kWarps * (kRingBytes + kStages * (16 + kExp)) +
                               8 * (DS_VIT_MAX_SEQS + 1) + static_cast<int>(sizeof(Seq)) * DS_VIT_MAX_SEQS;
};

// An item and the part of its blocks that a worker takes.
struct Item {
  int s, head, rho0;   // rho0: its first row among the rows that share the K/V head
  Seq q;
  KeyBlocks kb;
  int b, end;      // next block, end of the worker's part
};

struct Plan {
  const int64_t* pre;   // [n + 1]: units of the sequences before each
  const Seq* seqs;      // [n]
  int64_t begin, end;   // the worker's units
};

template <int kKeyShift>
__device__ __forceinline__ KeyBlocks seq_blocks(const AttentionArgs& a, const Seq& q) {
  KeyBlocks kb = key_blocks(q.kv - q.c, q.kv - 1, a.window, a.sinks, kKeyShift);
  if (q.c > 0 && kb.count == 0) kb.count = 1;   // nothing visible: one block without keys, so that zeros get written
  return kb;
}

constexpr int kRows = 16;   // rows of an item

__device__ __forceinline__ int row_tiles(const AttentionArgs& a, const Seq& q) {
  return (q.c * a.group + kRows - 1) / kRows;
}

// The item of unit u and the worker's part of it.
template <int kKeyShift>
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
  it.q = pl.seqs[lo];
  it.kb = seq_blocks<kKeyShift>(a, it.q);
  const int64_t r = u - pl.pre[lo];
  const int n = static_cast<int>(r / it.kb.count), tiles = row_tiles(a, it.q);
  it.head = n / tiles;
  it.rho0 = (n - it.head * tiles) * kRows;
  it.b = static_cast<int>(r - static_cast<int64_t>(n) * it.kb.count);
  const int64_t left = pl.end - u;
  it.end = left < it.kb.count - it.b ? it.b + static_cast<int>(left) : it.kb.count;
  return it;
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    mma_f16(c, a, b0, b1);
  else
    mma_bf16(c, a, b0, b1);
}

// bf16, head dim 128: both 64-dim planes of a tile by one copy for pages up to this, by
// two for larger ones.  64 sequences of 10 thousand tokens, one copy / two, us: pages of
// 16 tokens 404 / 435, 32 403 / 414, 64 402 / 397, 128 404 / 389 (2.7 GB at 6.7 to 7.0 TB/s).
constexpr int kPlanesShift = 5;

// The producer warp: lane i loads the blocks of consumer warp i into its ring as
// stages come free.  The lanes look at their rings in turn and stay together
// (each waiting for its own ring, they fell apart and held one another up).
// Lanes without a worker have an empty plan.  After two seconds without a free
// stage a lane stops loading, and its consumer times out on its own.  The exponents
// come by per-lane copies: a bulk or tensor copy costs the warp some 75 cycles a lane
// (e4m3, head dim 128, 64 sequences of 10 thousand tokens, pages of 64 / 16 tokens: 240
// / 384 us with bulk copies of the exponents, 224 / 311 so).
template <int D, bool E4M3>
__device__ __forceinline__ void produce(const CUtensorMap* tm_k, const CUtensorMap* tm_v, const AttentionArgs& a,
                                        const Plan& pl, uint32_t ring, uint32_t exps, uint32_t full, uint32_t empty) {
  using S = Shape<D, E4M3>;
  const int step = min(1 << a.c.page_shift, S::kKeys), pieces = S::kKeys / step;   // keys of a piece, pieces of a block
  int slot = 0;
  uint32_t phase = 1;                      // a new barrier's preceding phase counts as complete
  int64_t u = pl.begin;
  Item it{};
  int p_last = 0, lo = 0, next[S::kPieces] = {};
  // Table entries are read a block ahead.  Of a block's pages only those that some row sees are needed.
  auto look = [&](int b) {
    const int key0 = it.kb.at(b) << S::kKeyShift;
#pragma unroll
    for (int h = 0; h < S::kPieces; ++h) {
      const int k0 = key0 + h * step, k1 = k0 + step - 1;
      next[h] = -2;                        // not needed
      if (h < pieces && k0 <= p_last && (k1 >= lo || k0 < a.sinks))
        next[h] = __ldg(a.b.table + static_cast<int64_t>(it.s) * a.b.table_cols + (k0 >> a.c.page_shift));
    }
  };
  auto item = [&]() {
    it = item_at<S::kKeyShift>(a, pl, u);
    u += it.end - it.b;
    p_last = it.q.kv - 1;
    lo = window_start(a, it.q.kv - it.q.c);
    look(it.b);
  };
  bool active = u < pl.end;
  if (active) item();
  unsigned long long since = global_timer();
  while (__any_sync(0xFFFFFFFFu, active)) {
    if (active && mbar_test(empty + 8 * slot, phase)) {
      int page[S::kPieces];
#pragma unroll
      for (int h = 0; h < S::kPieces; ++h) page[h] = next[h];
      const int key0 = it.kb.at(it.b) << S::kKeyShift, head = it.head;
      if (++it.b < it.end)
        look(it.b);
      else if (u < pl.end)
        item();
      else
        active = false;
      const uint32_t bar = full + 8 * slot, to = ring + slot * S::kStage, ex = exps + slot * S::kExp;
      bool on[S::kPieces];
      int loads = 0;
#pragma unroll
      for (int h = 0; h < S::kPieces; ++h) {
        on[h] = page_there(page[h], a.c.n_pages);
        if (!on[h] && page[h] != -2) report_error(a.status, DS_VIT_ERANGE);
        loads += on[h];
      }
      mbar_expect_tx(bar, S::kStage / pieces * loads);
#pragma unroll
      for (int h = 0; h < S::kPieces; ++h) {
        if (!on[h]) continue;
        const int row = static_cast<int>(cache_row(a.c, page[h], head, key0 + h * step));
        if constexpr (E4M3) {
          tma_load_2d(to + h * step * S::kRow, tm_k, bar, 0, row);
          tma_load_2d(to + S::kTile + h * step * S::kRow, tm_v, bar, 0, row);
          for (int i = 0; i < step; i += 16) {
            cp_async_16(ex + h * step + i, a.c.k_exp + row + i, 16);
            cp_async_16(ex + S::kKeys + h * step + i, a.c.v_exp + row + i, 16);
          }
        } else {
          if (D == 128 && a.c.page_shift <= kPlanesShift) {
            tma_load_3d(to, tm_k, bar, 0, row, 0);
            tma_load_3d(to + S::kTile, tm_v, bar, 0, row, 0);
          } else {
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
              tma_load_2d(to + S::kPlane * x, tm_k, bar, 64 * x, row);
              tma_load_2d(to + S::kTile + S::kPlane * x, tm_v, bar, 64 * x, row);
            }
          }
        }
      }
      if constexpr (E4M3) cp_async_arrive(bar);
      if (++slot == S::kStages) {
        slot = 0;
        phase ^= 1;
      }
      since = global_timer();
    } else if (active && global_timer() - since > kWaitLimitNs) {
      report_error(a.status, kErrTimeout);
      active = false;
    }
  }
  if constexpr (E4M3) cp_async_wait<0>();   // no copy lands after the CTA has exited
}

// kRowHalves: 1 when at most 8 rows share a K/V head (rows 8 .. 15 of the
// MMAs' 16 are then zeros nobody looks at), else 2.
template <int D, bool E4M3, int kRowHalves>
__global__ void __launch_bounds__(Shape<D, E4M3>::kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ AttentionArgs a, const Records rec) {
  using S = Shape<D, E4M3>;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads, kRingBytes = S::kRingBytes;
  constexpr int kSteps = D / 16;           // k steps of S
  constexpr int kCols = D / 8;             // column tiles of O
  constexpr int kN = S::kKeys / 8;         // column tiles of S
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // Per ring: tiles, exponents, full and empty barriers.
  const uint32_t rings = smem_u32(smem);
  const uint32_t exps0 = rings + kWarps * kRingBytes;
  const uint32_t bars0 = exps0 + kWarps * S::kStages * S::kExp;
  int64_t* pre = reinterpret_cast<int64_t*>(smem + kWarps * (kRingBytes + S::kStages * (S::kExp + 16)));
  Seq* seqs = reinterpret_cast<Seq*>(pre + DS_VIT_MAX_SEQS + 1);
  auto full_of = [&](int w) { return bars0 + w * S::kStages * 16; };
  auto empty_of = [&](int w) { return full_of(w) + S::kStages * 8; };
  __shared__ int64_t part[kWarps + 1];

  if (warp == kWarps) {
    if (lane < kWarps)
      for (int i = 0; i < S::kStages; ++i) {
        mbar_init(full_of(lane) + 8 * i, E4M3 ? 2 : 1);     // the tiles' bytes, the exponents' copies
        mbar_init(empty_of(lane) + 8 * i, 1);
      }
    if (lane == 0) {
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
      seqs[s] = q;
      x = static_cast<int64_t>(seq_blocks<S::kKeyShift>(a, q).count) * row_tiles(a, q) * a.c.kv_heads;
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
    for (int w = 0; w <= kWarps; ++w) {
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
  const Shares shares = deal(total, W);
  // Neighbouring shares go to different SMs.
  auto worker = [&](int w) { return static_cast<int64_t>(w) * gridDim.x + blockIdx.x; };
  if (warp == kWarps) {
    Plan pl{pre, seqs, 0, 0};
    if (lane < kWarps && worker(lane) < W) {
      pl.begin = shares.begin(worker(lane));
      pl.end = shares.begin(worker(lane) + 1);
    }
    produce<D, E4M3>(&tm_k, &tm_v, a, pl, rings + lane * kRingBytes, exps0 + lane * S::kStages * S::kExp,
                     full_of(lane), empty_of(lane));
    return;
  }
  const int64_t me = worker(warp);
  if (me >= W) {
    if (lane == 0) rec.headers[me] = SplitHeader{};
    return;
  }
  const Plan pl{pre, seqs, shares.begin(me), shares.begin(me + 1)};
  const uint32_t ring = rings + warp * kRingBytes, exps = exps0 + warp * S::kStages * S::kExp;
  const uint32_t full = full_of(warp), empty = empty_of(warp);

  // ---- the worker's items
  int slot = 0;
  uint32_t phase = 0;
  SplitHeader header{};
  bool dead = false;                       // a wait gave up
  bool marked = false;                     // whole items have rows that may be to compute again
  for (int64_t u = pl.begin; u < pl.end;) {
    const Item it = item_at<S::kKeyShift>(a, pl, u);
    const int R = min(it.q.c * a.group - it.rho0, kRows);       // rows of this item
    // Q fragments and positions of rows g, g + 8; what scales an fp16 row's scores back, times scale_log2.
    uint32_t qf[kSteps][4];
    int pos[kRowHalves];
    float qscale[kRowHalves];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int rho = it.rho0 + 8 * x + g;
      const int i = a.by_group(rho);
      const bool on = x < kRowHalves && 8 * x + g < R;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          a.q + (it.q.row0 + i) * a.q_stride + (it.head * a.group + rho - i * a.group) * D);
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        // Dims of the k step held by this lane: 2t, 2t + 1 and 2t + 8, 2t + 9
        // of 16, or (e4m3) four consecutive ones of its 16-byte piece.
        const int d0 = E4M3 ? 16 * (D == 128 ? 2 * t + (k >> 2) : t) + 4 * (k & 3) : 16 * k + 2 * t;
        const int d1 = E4M3 ? d0 + 2 : d0 + 8;
        qf[k][x] = on ? __ldg(src + d0 / 2) : 0u;
        qf[k][2 + x] = on ? __ldg(src + d1 / 2) : 0u;
      }
      if (x >= kRowHalves) continue;
      pos[x] = on ? it.q.kv - it.q.c + i : -1;
      qscale[x] = a.scale_log2;
      if constexpr (E4M3) {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
          top = __vmaxu2(top, __vmaxu2(qf[k][x] & 0x7FFF7FFFu, qf[k][2 + x] & 0x7FFF7FFFu));
        top = max(top & 0xFFFFu, top >> 16);
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // The largest's exponent field E: times 2^(141 - E), in two steps of normal powers of two.
        const int E = max(static_cast<int>(top >> 7), 1), up = 141 - E, half = up / 2;
        const float f0 = __int_as_float((127 + half) << 23), f1 = __int_as_float((127 + up - half) << 23);
        const float g0 = __int_as_float((127 - half) << 23), g1 = __int_as_float((127 - up + half) << 23);
        qscale[x] = a.scale_log2 * g0 * g1;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          qf[k][x] = pack_f16x2(bf16lo(qf[k][x]) * f0 * f1, bf16hi(qf[k][x]) * f0 * f1);
          qf[k][2 + x] = pack_f16x2(bf16lo(qf[k][2 + x]) * f0 * f1, bf16hi(qf[k][2 + x]) * f0 * f1);
        }
      }
    }
    float o[kCols][4], m[kRowHalves], l[kRowHalves], d[kRowHalves];   // d: e4m3, see Raise
#pragma unroll
    for (int x = 0; x < kRowHalves; ++x) {
      m[x] = -INFINITY;
      l[x] = d[x] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < kCols; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    // Positions of the sequence's first and last rows (its items share the key blocks).
    const int p_first = it.q.kv - it.q.c, p_last = it.q.kv - 1;
    const int lo_first = window_start(a, p_first), lo_last = window_start(a, p_last);

    for (int b = it.b; b < it.end; ++b) {
      const uint32_t tk = ring + slot * S::kStage, tv = tk + S::kTile, ex = exps + slot * S::kExp;
      const int key0 = it.kb.at(b) << S::kKeyShift;
      // Every row sees all keys of the block.
      const bool open = key0 + S::kKeys - 1 <= p_first && (key0 >= lo_last || key0 + S::kKeys <= a.sinks);
      auto any = [&](int j) { return j <= p_last && (j >= lo_first || j < a.sinks); };   // some row sees key j
      dead |= !mbar_wait(full + 8 * slot, phase, a.status);
      if (!open) {
        // Values that no row sees (behind the last token, before every window)
        // may be anything: zeros take their place, in the tile and (below) as weights.
#pragma unroll 1
        for (int x = lane; x < S::kTile / 16; x += 32) {
          const int row = E4M3 ? x / (S::kRow / 16) : (x >> 3) & (S::kKeys - 1);
          if (!any(key0 + row)) sts128(tv + 16 * x, make_uint4(0, 0, 0, 0));
        }
        fence_proxy_async_smem();          // before the loads that will follow into the tile
        __syncwarp();
      }
      // ---- S = Q K^T, 16 rows x kKeys keys.  bf16: the block's fragments, all at once,
      // then the stage is free again; e4m3: key tile by key tile, the values later.
      constexpr int kWords = E4M3 ? 1 : D / 4;
      uint32_t kw[kWords], vw[kWords], ke[kN], ve[kN];
      float sc[kN][4];
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
      auto release = [&]() {
        // The reads come before the loads that the stage's return lets in.
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * slot);
        if (++slot == S::kStages) {
          slot = 0;
          phase ^= 1;
        }
      };
      if constexpr (E4M3) {
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          ke[n] = lds_u16(ex + 8 * n + 2 * t);
          ve[n] = lds_u16(ex + S::kKeys + 8 * n + 2 * t);
        }
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          const int row = 8 * n + g;         // this lane's key of the tile
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            const uint32_t piece = D == 128 ? (2 * t + h) ^ (row & 7) : t ^ ((row >> 1) & 3);
            const uint4 w = lds128(tk + row * S::kRow + piece * 16);
            mma<true>(sc[n], qf[4 * h], e4m3x2_to_f16x2(w.x & 0xFFFFu), e4m3x2_to_f16x2(w.x >> 16));
            mma<true>(sc[n], qf[4 * h + 1], e4m3x2_to_f16x2(w.y & 0xFFFFu), e4m3x2_to_f16x2(w.y >> 16));
            mma<true>(sc[n], qf[4 * h + 2], e4m3x2_to_f16x2(w.z & 0xFFFFu), e4m3x2_to_f16x2(w.z >> 16));
            mma<true>(sc[n], qf[4 * h + 3], e4m3x2_to_f16x2(w.w & 0xFFFFu), e4m3x2_to_f16x2(w.w >> 16));
          }
        }
      } else {
        const int kr = (lane & 7) + ((lane >> 4) << 3), vr = lane & 15;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const int piece = 2 * (k & 3) + ((lane >> 3) & 1);
          ldmatrix_x4(tk + kr * 128 + (k >> 2) * S::kPlane + ((piece ^ (kr & 7)) << 4),
                      *reinterpret_cast<uint32_t(*)[4]>(kw + 4 * k));
        }
#pragma unroll
        for (int n = 0; n < kCols; n += 2) {
          const int piece = (n & 7) + (lane >> 4);
          ldmatrix_x4_trans(tv + vr * 128 + (n >> 3) * S::kPlane + ((piece ^ (vr & 7)) << 4),
                            *reinterpret_cast<uint32_t(*)[4]>(vw + 2 * n));
        }
        release();
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
#pragma unroll
          for (int n = 0; n < kN; ++n) mma<false>(sc[n], qf[k], kw[4 * k + 2 * n], kw[4 * k + 2 * n + 1]);
      }
      // ---- softmax of the block: scores z = sc f (log2 units), f the scale and
      // the key's factor; contributions z + the value's exponent
      float add[kN][2], vf[kN][2], top[kRowHalves], most[kRowHalves];   // most: the largest contribution
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          add[n][e] = 0.f;
          vf[n][e] = 1.f;
          if constexpr (E4M3) {
            // Rows with the NaN byte hold NaN elements, so plain shifts do for the factors.
            const uint32_t kb = e == 0 ? ke[n] & 255u : ke[n] >> 8, vb = e == 0 ? ve[n] & 255u : ve[n] >> 8;
            const float kf = __uint_as_float(kb << 23);
            vf[n][e] = __uint_as_float(vb << 23);
            add[n][e] = __uint_as_float(0x4B000000u | vb) - 8388735.f;   // byte - 127: the byte in the last bits of 2^23
#pragma unroll
            for (int x = 0; x < kRowHalves; ++x) sc[n][2 * x + e] *= qscale[x] * kf;
          }
        }
#pragma unroll
      for (int x = 0; x < kRowHalves; ++x) {
        if (!open) {
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!sees(a, pos[x], key0 + 8 * n + 2 * t + e)) sc[n][2 * x + e] = -INFINITY;
        }
        top[x] = most[x] = -INFINITY;
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[x] = fmaxf(top[x], sc[n][2 * x + e]);
            if constexpr (E4M3) most[x] = fmaxf(most[x], sc[n][2 * x + e] + add[n][e]);
          }
        if constexpr (!E4M3) {
          top[x] *= qscale[x];
          top[x] = fmaxf(top[x], __shfl_xor_sync(0xFFFFFFFFu, top[x], 1));
          top[x] = fmaxf(top[x], __shfl_xor_sync(0xFFFFFFFFu, top[x], 2));
        }
      }
      // References are raised (and O rescaled) rarely.
      bool some = dead;
#pragma unroll
      for (int x = 0; x < kRowHalves; ++x)
        some |= E4M3 ? must_raise(m[x], d[x], top[x], most[x]) : top[x] > m[x] + kLag16;
      if (__any_sync(0xFFFFFFFFu, some)) {
        if (__any_sync(0xFFFFFFFFu, dead)) {
          dead = true;
          break;
        }
#pragma unroll
        for (int x = 0; x < kRowHalves; ++x) {
          float fl, fo;
          if constexpr (E4M3) {
#pragma unroll
            for (int y = 1; y < 4; y <<= 1) {      // over the row's four lanes
              top[x] = fmaxf(top[x], __shfl_xor_sync(0xFFFFFFFFu, top[x], y));
              most[x] = fmaxf(most[x], __shfl_xor_sync(0xFFFFFFFFu, most[x], y));
            }
            const Raise r = raised(m[x], d[x], top[x], most[x]);
            m[x] = r.m, d[x] = r.d, fl = r.l, fo = r.o;
          } else {
            const float old = m[x];
            if (top[x] > old + kLag16) m[x] = top[x];
            fl = fo = old == m[x] ? 1.f : ex2_approx(old - m[x]);
          }
          l[x] *= fl;
#pragma unroll
          for (int n = 0; n < kCols; ++n) {
            o[n][2 * x] *= fo;
            o[n][2 * x + 1] *= fo;
          }
        }
      }
      uint32_t pf[kN / 2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        constexpr int kLast = kRowHalves - 1;
        const int y = x < kLast ? x : kLast;
        const float base = m[y] != -INFINITY ? -m[y] : 0.f, down = E4M3 ? shift_down(d[y]) : 1.f;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          uint32_t& p = pf[n / 2][2 * (n & 1) + x];
          p = 0;
          if (x >= kRowHalves) continue;
          const float f = E4M3 ? 1.f : qscale[y];
          float w0 = ex2_approx(fmaf(sc[n][2 * x], f, base));
          float w1 = ex2_approx(fmaf(sc[n][2 * x + 1], f, base));
          l[y] += w0 + w1;
          // The product's operand: weights in 16 bits (their sum stays in fp32).
          p = E4M3 ? pack_f16x2(w0 * down * vf[n][0], w1 * down * vf[n][1]) : pack_bf16x2(w0, w1);
          if (E4M3 && !open) {
            // The exponent of a value that nobody sees may be the NaN byte.
            const int j = key0 + 8 * n + 2 * t;
            p &= (any(j) ? 0xFFFFu : 0u) | (any(j + 1) ? 0xFFFF0000u : 0u);
          }
        }
      }
      // ---- O += P V
      if constexpr (E4M3) {
#pragma unroll
        for (int h = 0; h < kN / 2; ++h) {
          // w[4 y + x]: word y of the rows of keys 16h + 2t, + 1, + 8, + 9
          uint32_t w[kCols];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = 16 * h + 8 * (x >> 1) + 2 * t + (x & 1);
            if constexpr (D == 128) {
              const uint4 v = lds128(tv + row * S::kRow + ((g ^ (row & 7)) << 4));
              w[x] = v.x, w[4 + x] = v.y, w[8 + x] = v.z, w[12 + x] = v.w;
            } else {
              const uint2 v = lds64(tv + row * S::kRow + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + 8 * (g & 1));
              w[x] = v.x, w[4 + x] = v.y;
            }
          }
#pragma unroll
          for (int y = 0; y < kCols / 4; ++y)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              // Bytes e, e + 1 of both keys' words, side by side per dim.
              const uint32_t sel = e == 0 ? 0x5140u : 0x7362u;
              const uint32_t p0 = __byte_perm(w[4 * y], w[4 * y + 1], sel), p1 = __byte_perm(w[4 * y + 2], w[4 * y + 3], sel);
              mma<true>(o[4 * y + e], pf[h], e4m3x2_to_f16x2(p0 & 0xFFFFu), e4m3x2_to_f16x2(p1 & 0xFFFFu));
              mma<true>(o[4 * y + e + 1], pf[h], e4m3x2_to_f16x2(p0 >> 16), e4m3x2_to_f16x2(p1 >> 16));
            }
        }
        release();
      } else {
#pragma unroll
        for (int n = 0; n < kCols; ++n) mma<false>(o[n], pf[0], vw[2 * n], vw[2 * n + 1]);
      }
    }
    if (dead) break;

    // ---- the item's end: finished here, or a record for the join
#pragma unroll
    for (int x = 0; x < kRowHalves; ++x) {
      l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], 1);
      l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], 2);
    }
    const bool begun = it.b > 0, whole = !begun && it.end == it.kb.count;
    if (!begun && !whole) {
      const int64_t last = u - it.b + it.kb.count - 1;
      header = SplitHeader{static_cast<int>(shares.owner(last) - me) + 1, it.s, it.head, it.rho0, it.q, 0};
    }
    float* r = rec.at(me, begun ? 0 : 1);
    bool redo = false;                     // a row that may be to compute again
#pragma unroll
    for (int x = 0; x < kRowHalves; ++x) {
      const int rr0 = 8 * x + g, rho = it.rho0 + rr0;
      bool bad = false;
      if (rr0 < R) {
        const int i = a.by_group(rho);
        bf16* dst = a.out + (it.q.row0 + i) * a.out_stride + (it.head * a.group + rho - i * a.group) * D;
        const float inv = 1.f / l[x], up = E4M3 ? shift_up(d[x]) : 1.f;
        auto value = [&](float y) { return pos[x] < 0 ? 0.f : y * inv * up; };
        float* rr = r + rr0 * D;
        if (!whole && t == 0) {
          rec.max_of(r, D)[rr0] = m[x];
          rec.sum_of(r, D)[rr0] = l[x];
          if constexpr (E4M3) rec.shift_of(r, D)[rr0] = d[x];
        }
        // bf16: columns 8n + 2t, + 1.  e4m3: column tile n holds dim n of each
        // lane group's D / 8, so this lane has dims (2t) D/8 + n and (2t + 1) D/8 + n.
        if constexpr (E4M3) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int d0 = (2 * t + e) * kCols;
#pragma unroll
            for (int n = 0; n < kCols; n += 4) {
              float4 y = make_float4(o[n][2 * x + e], o[n + 1][2 * x + e], o[n + 2][2 * x + e], o[n + 3][2 * x + e]);
              if (whole) {
                y = make_float4(value(y.x), value(y.y), value(y.z), value(y.w));
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
            float y0 = o[n][2 * x], y1 = o[n][2 * x + 1];
            if (whole) {
              y0 = value(y0), y1 = value(y1);
              bad |= not_finite(y0) || not_finite(y1);
              *reinterpret_cast<uint32_t*>(dst + 8 * n + 2 * t) = pack_bf16x2(y0, y1);
            } else {
              *reinterpret_cast<float2*>(rr + 8 * n + 2 * t) = make_float2(y0, y1);
            }
          }
        }
      }
      redo |= bad && it.q.c > 1;
    }
    marked |= redo;
    u += it.end - it.b;
  }
  if (dead) {
    // After a timeout: wait (bounded) for the loads that may still be in flight.
    for (int i = 0; i < S::kStages; ++i) {
      if (!mbar_wait(full + 8 * slot, phase, nullptr)) break;
      if (++slot == S::kStages) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
  if (lane == 0) rec.headers[me] = dead ? SplitHeader{} : header;
  // Rows to compute again, now that the producer has nothing left to wait for.
  __syncwarp();                            // what the lanes wrote is there for all of them
  if (!dead && __any_sync(0xFFFFFFFFu, marked))
    for (int64_t u = pl.begin; u < pl.end;) {
      const Item it = item_at<S::kKeyShift>(a, pl, u);
      u += it.end - it.b;
      if (it.b != 0 || it.end != it.kb.count || it.q.c <= 1) continue;
      const int p0 = it.q.kv - it.q.c, p1 = it.q.kv - 1, end = min(it.rho0 + kRows, it.q.c * a.group);
      for (int rho = it.rho0; rho < end; ++rho) {
        const int i = a.by_group(rho), h = it.head * a.group + rho - i * a.group;
        if (row_not_finite<D>(a, it.q.row0 + i, h, lane))
          mend_row<D, E4M3>(a, it.s, it.q.row0, p0 + i, i, h, p0, p1, lane);
      }
    }
}

// Joins the parts of every split item.  Block (y, x) looks after workers x, x +
// gridDim.y, ... and rows y, y + gridDim.x, ... of their items (rows in the grid's
// fast dimension: the blocks of the few workers with something to join then lie on
// many SMs).  One warp adds up a row; where many parts meet few rows (a token over
// a long cache) the parts are shared between the block's warps.
constexpr int kJoinItems = 16;    // workers per block at most
constexpr int kJoinRows = 8;      // grid rows at most

template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kJoinWarps, 4)
    join_kernel(const __grid_constant__ AttentionArgs a, const Records rec, int workers) {
  __shared__ SplitHeader heads[kJoinItems];
  grid_dep_launch();
  grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = blockIdx.y, groups = gridDim.y;
  const int mine = (workers - group + groups - 1) / groups;
  if (threadIdx.x < 2 * mine)
    reinterpret_cast<int4*>(heads)[threadIdx.x] =
        reinterpret_cast<const int4*>(rec.headers + group + (threadIdx.x >> 1) * groups)[threadIdx.x & 1];
  __syncthreads();
  int turn = 0;                       // rows dealt to the warps so far
  for (int k = 0; k < mine; ++k) {
    const SplitHeader& hd = heads[k];
    if (hd.parts == 0) continue;
    const int w = group + k * groups;
    const int64_t left = static_cast<int64_t>(hd.q.c) * a.group - hd.rho0;
    const int rows = left < rec.rows ? static_cast<int>(left) : rec.rows;
    auto positions = [&](int& p0, int& p1) {         // a sequence's items share the key blocks
      p0 = hd.q.kv - hd.q.c;
      p1 = hd.q.kv - 1;
    };
    for (int row = blockIdx.x; row < rows; row += gridDim.x) {
      Sum<D> sum;
      if (hd.parts <= kJoinWarps) {
        if (turn++ % kJoinWarps != warp) continue;
        join_parts<D, E4M3, 4>(rec, w, hd.parts, row, 0, 1, lane, sum);
        join_finish<D, E4M3>(a, hd, hd.rho0 + row, sum, lane, positions);
        continue;
      }
      join_parts<D, E4M3, 4>(rec, w, hd.parts, row, warp, kJoinWarps, lane, sum);
      join_warps<D, E4M3>(warp, lane, sum);
      if (warp == 0) join_finish<D, E4M3>(a, hd, hd.rho0 + row, sum, lane, positions);
    }
  }
}

template <int D, bool E4M3, int kRowHalves>
int launch(const AttentionArgs& a, void* ws, cudaStream_t stream) {
  using S = Shape<D, E4M3>;
  CUtensorMap tk, tv;
  const uint64_t rows = static_cast<uint64_t>(a.c.n_pages) * a.c.kv_heads << a.c.page_shift;
  const uint64_t cols = S::kRow / 2;      // in 16-bit units
  const uint32_t box = std::min(1 << a.c.page_shift, S::kKeys);
  auto map = [&](CUtensorMap* m, const void* p) {
    if (cols == 128 && a.c.page_shift <= kPlanesShift) return make_tmap_bf16_planes(m, p, rows, box);
    return cols == 32 ? make_tmap_bf16_sw64(m, p, rows, cols, box) : make_tmap_bf16(m, p, rows, cols, box);
  };
  if (!map(&tk, a.c.k) || !map(&tv, a.c.v)) return DS_VIT_ECUDA;
  if (allow_smem(reinterpret_cast<const void*>(decode_kernel<D, E4M3, kRowHalves>), S::kSmem) != cudaSuccess)
    return DS_VIT_ECUDA;
  const int R = std::min(a.b.max_rows * a.group, kRows), grid = num_sms();
  const int workers = grid * S::kWarps;
  const Records rec = records_in(ws, workers, R, D);
  cudaError_t e = launch_pdl(decode_kernel<D, E4M3, kRowHalves>, dim3(grid), dim3(S::kThreads), S::kSmem, stream, tk, tv,
                             a, rec);
  if (e == cudaSuccess)
    e = launch_pdl(join_kernel<D, E4M3>, dim3(rec.rows < kJoinRows ? rec.rows : kJoinRows, grid),
                   dim3(32 * kJoinWarps), 0, stream, a, rec, workers);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? DS_VIT_OK : DS_VIT_ECUDA;
}

}  // namespace

size_t cache_decode_workspace(int head_dim, int rows) {
  // The larger of the two kinds': the size depends on head_dim and rows alone.
  const int warps = head_dim == 64 ? std::max(Shape<64, false>::kWarps, Shape<64, true>::kWarps)
                                   : std::max(Shape<128, false>::kWarps, Shape<128, true>::kWarps);
  return records_bytes(static_cast<int64_t>(num_sms()) * warps, std::min(rows, kRows), head_dim);
}

int launch_cache_decode(const AttentionArgs& a, int head_dim, bool e4m3, void* ws, cudaStream_t stream) {
  const int R = a.b.max_rows * a.group;
  if (head_dim == 128) {
    if (R <= 8) return e4m3 ? launch<128, true, 1>(a, ws, stream) : launch<128, false, 1>(a, ws, stream);
    return e4m3 ? launch<128, true, 2>(a, ws, stream) : launch<128, false, 2>(a, ws, stream);
  }
  if (R <= 8) return e4m3 ? launch<64, true, 1>(a, ws, stream) : launch<64, false, 1>(a, ws, stream);
  return e4m3 ? launch<64, true, 2>(a, ws, stream) : launch<64, false, 2>(a, ws, stream);
}

}  // namespace dsvit
