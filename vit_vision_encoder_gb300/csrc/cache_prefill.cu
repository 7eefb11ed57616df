// Attention over the paged cache for many rows (chunks of a prompt) on tcgen05.
//
// The query rows that share a K/V head (new tokens times query heads per K/V
// head, token by token) are taken 256 at a time, as two 128-row tiles A and B
// that share every tile of 128 keys; an item is one such group of rows, and the
// unit of work is one key tile of an item.  All units are counted from the
// lengths on the device and dealt to the CTAs, one per SM, in equal shares
// (cache_plan.h): causal items of unequal depth, short chunks over long caches
// and ragged batches all end together.  A CTA finishes the items that lie within
// its share; the others leave records that join_items_kernel adds up.
//
// Bound by the tensor pipe and the chain S -> softmax -> P V of a tile, of which two
// (A's and B's) overlap: 2048 rows over 34 thousand tokens, 40 query and 8 K/V heads
// of 128, bf16, take 863 us (1.60 PFLOP/s; 2820 cycles a step of two tiles, 2048 of
// them tensor work), 940 to 1000 us in calls back to back, where power lowers the
// clock.  Short calls are bound by what comes before and after: launch, plan, first loads
// (9 us) and join (2.5 us where nothing is split) of the 37 us that 1090 rows with
// nothing cached take.
//
// Roles: warps 0-7 run the softmax of tile A and warps 8-15 that of tile B, two
// threads a row (16x32bx2 TMEM accesses, as in the bidirectional kernel); warp
// 16 loads pages by TMA (a box per page and 64 dims) into a ring of key and
// value tiles; warp 17 issues the MMAs:
//   S_X = Q_X K_j^T     (M 128, N 128, K D)    smem x smem -> TMEM
//   O_X += P_X V_j      (M 128, N D,   K 128)  TMEM x smem -> TMEM
// P_X (16-bit pairs) takes the first half of S_X's columns, so S_X of the next
// tile waits for P_X V_j; the other tile's MMAs and softmax fill that time.  At head
// dim 64 TMEM has room for a third score tile, and A and B take the three in turn
// (e4m3, windowed chunks of 31 to 1008 rows, 55 us now: 3.6 us less by it).
// Rows of Q are loaded by the softmax warps, so any group size fills the tiles.
// Warp 18 walks the CTA's items and hands them to the other roles through a
// ring in shared memory.  The rows' way in and out of the tiles is through
// 16-byte pieces that lie side by side in memory (by way of the row's place in
// the Q tile on the way out): as accesses of a thread to its own row, they took
// 6000 cycles in and 10000 out an item.
//
// An item of at most 128 rows leaves tile B without rows of its own: it then
// takes the same rows and every other key tile, and the two results are added up
// in TMEM (32 sequences of 8000 tokens, 32 rows, bf16, D 64: 130 us without, 105
// with).
//
// e4m3 pages: warps 20-27 widen the raw tiles to fp16 in shared memory (the
// conversion is exact; the rows of a tile are scaled by powers of two to the
// tile's largest exponent E, those of a tile whose exponents lie far apart are not:
// kFar).  Scores are
// scaled by 2^E(K); the weights are taken against the running maximum of score
// plus E(V), the size of a contribution, and their sum is scaled back to a reference
// of its own (Raise in cache_rows.cuh).  Query rows are scaled to fp16's range like
// in the kernel for few rows.
//
// Keys that a row does not see are masked in its scores.  Value rows that no row
// of the item sees are zeroed in shared memory (they may hold anything); where
// rows of an item see different keys and a result is not finite because of a value
// hidden from it, the row is computed again from the keys that it does see (mend_row):
// by the join, as waits here have a limit.
#include "cache_rows.cuh"

#include <type_traits>

namespace dsvit {

namespace {

constexpr int kTile = 128;                  // rows of a query tile, keys of a key tile
constexpr int kTileShift = 7;
constexpr int kItemRows = 2 * kTile;
constexpr int kWarpTma = 16, kWarpMma = 17, kWarpJobs = 18;
constexpr int kWarpConvert = 20;            // 20 .. 23: key tiles, 24 .. 27: value tiles (e4m3)
constexpr uint32_t kTmemCols = 512;
// e4m3: a tile whose rows (those that some row of the item sees) lie further apart than
// this is taken as it is, and the softmax multiplies by each key's own factors (kFar in
// place of the tile's exponent).  Keys scaled by 2^-15 are still exact in fp16 (multiples of
// 2^-9 2^-15).  A row's reference follows the tile's exponent E(V): where the value that has
// it is hidden from the row, or its weight is nothing, it lies up to kSpanV above the row's
// largest contribution, and those under 2^(kSpanV - 20) of that one lose bits.  Rows of zeros
// count, with their exponent of -117: the score of one may be the tile's largest, and E(V)
// then says nothing about the contributions.
constexpr int kSpanK = 15, kSpanV = 8, kFar = 1024;

template <int D, bool E4M3>
struct Cfg {
  static constexpr int kThreads = E4M3 ? 896 : 608;
  static constexpr int kBytes = kTile * D * 2;             // a 16-bit tile of 128 rows
  static constexpr int kHalf = kTile * 128;                // 64 dims of it
  static constexpr int kRawBytes = kTile * D;              // an e4m3 tile
  static constexpr int kRing = E4M3 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 8);
  // The converters of keys and those of values each wait for every use of their raw
  // places and for no other (a wait by parity must not skip a use): an even number.
  static constexpr int kRaw = E4M3 ? 4 : 0;
  // Tile B takes part in items without rows for it (with a ring of three tiles it would wait for A's).
  static constexpr bool kShare = kRing > 3;
  // Score tiles in TMEM, 128 columns each, then O_A and O_B: one each for A and B, or
  // (where O leaves room) three for the two of them in turn.
  static constexpr int kScores = D == 64 ? 3 : 2;
  static constexpr uint32_t kTmemO = 128 * kScores;
  static constexpr int kOffKv = 2 * kBytes;                // after Q_A, Q_B
  static constexpr int kOffRaw = kOffKv + kRing * kBytes;
  static constexpr int kOffExp = kOffRaw + kRaw * kRawBytes;   // exponents of the raw tiles
  static constexpr int kOffBar = kOffExp + kRaw * kTile;
  static constexpr int kSmem = kOffBar + 1024 + 1024;
  static_assert(kSmem + 512 <= 232448, "shared memory, the static part included");
  static constexpr float kLag16 = 8.f;                     // bf16: see the kernel for few rows
};

// Barrier slots.
enum : int {
  kBarQ = 0,                // [2] tile X's query rows are in shared memory
  kBarKvFull = 2,           // [8]
  kBarKvEmpty = 10,         // [8]
  kBarRawFull = 18,         // [4]
  kBarRawEmpty = 22,        // [4]
  // By score tile, whose next scores wait for the product of its last weights: with
  // three of them a softmax may be two steps ahead of the issuer, which a barrier by
  // query tile would lose count of.
  kBarSFull = 26,           // [3]
  kBarPFull = 29,           // [3]
  kBarPvDone = 32,          // [2]
  kBarRagged = 34,          // a value tile with rows to zero has landed
  kBarDrain = 35,
  kBarJobFull = 36,         // [4]
  kBarJobEmpty = 40,        // [4]
  kBarOther = 44,           // tile B's share of the keys is summed up
  kBarMerged = 45,          // and has been read
  kBarCount = 46
};

// Where a CTA's share of the units begins, and how many it has; how far
// borders move to an item's end.
struct Start {
  int s, k, head, off;        // off: units of the item before the share
  int64_t units, total, first;
  int snap;
};
struct PrefillArgs {
  AttentionArgs a;
  Records rec;
};

// Shares are counted in key tiles, an item weighing kItemCost more than it has:
// what its rows' way in and out takes (5 us; a tile takes 1.4).
constexpr int kItemCost = 4;
// A split costs what some six tiles do (the second load of the rows, records of
// 128 KB a part, their sum), so borders move to an item's end within six; and
// where even the longest item is short and not much over a share, no item is split.
constexpr int kSnap = 6, kUnsplit = 16 + kItemCost;

__device__ __forceinline__ int items_of(const AttentionArgs& a, const Seq& q) {
  return (q.c * a.group + kItemRows - 1) / kItemRows;
}

// Positions of the first and the last row of item k of a sequence.
__device__ __forceinline__ void item_positions(const AttentionArgs& a, const Seq& q, int k, int& p0, int& p1) {
  const int r0 = k * kItemRows, r1 = min(r0 + kItemRows, q.c * a.group) - 1;
  p0 = q.kv - q.c + a.by_group(r0);
  p1 = q.kv - q.c + a.by_group(r1);
}

__device__ __forceinline__ KeyBlocks item_blocks(const AttentionArgs& a, const Seq& q, int k) {
  int p0, p1;
  item_positions(a, q, k, p0, p1);
  KeyBlocks kb = key_blocks(p0, p1, a.window, a.sinks, kTileShift);
  if (kb.count == 0) kb.count = 1;          // nothing visible: one tile without keys, so that zeros get written
  return kb;
}

// What the roles need to know of an item, and the CTA's part of its tiles.
struct alignas(16) Job {
  int s, head;
  int rho0;                   // first of its rows among those that share the K/V head
  int whole;                  // 1: all tiles are the CTA's; 0: a record is left, 2: for an item begun elsewhere
  Seq q;
  int b;
  KeyBlocks kb;
  int end;                    // tiles b .. end - 1; none: no more items
};
constexpr int kJobs = 4;

// The CTA's items in the order sequence, item, head.
struct Walk {
  int s, k, head, b, end;
  Seq q;
  KeyBlocks kb;
  int take;                   // units of this item
  int64_t left;               // units left, this item's included

  // Into the item at unit `off`, which is 0 or behind its first kItemCost.
  __device__ __forceinline__ void enter(const AttentionArgs& a, int off) {
    kb = item_blocks(a, q, k);
    const int rest = kb.count + kItemCost - off;
    take = left < rest ? static_cast<int>(left) : rest;
    b = off == 0 ? 0 : off - kItemCost;
    end = off + take - kItemCost;
  }
  __device__ __forceinline__ void start(const AttentionArgs& a, const Start& st) {
    s = st.s, k = st.k, head = st.head;
    left = st.units;
    q = left > 0 ? load_seq(a.b, a.c.page_shift, s, nullptr) : Seq{0, 0, 0};
    if (left <= 0) return;
    enter(a, st.off);
    if (b >= kb.count) step(a);             // the border moved to this item's end
  }
  // To the next item; left must be positive afterwards for it to exist.
  __device__ __forceinline__ void next(const AttentionArgs& a) {
    left -= take;
    if (left > 0) step(a);
  }
  __device__ __noinline__ void step(const AttentionArgs& a) {
    if (++head == a.c.kv_heads) {
      head = 0;
      if (++k == items_of(a, q)) {
        k = 0;
        do {
          q = load_seq(a.b, a.c.page_shift, ++s, nullptr);
        } while (q.c == 0);
      }
    }
    enter(a, 0);
  }
};

// The plan of the call, by all threads of a CTA in scratch shared memory: a
// flat list of (sequence, item) pairs, each thread adding up a run of it.
template <int kThreads>
__device__ __forceinline__ Start make_plan(const AttentionArgs& a, uint8_t* scratch, int* status) {
  int* items = reinterpret_cast<int*>(scratch);                                 // [n + 1] items before each sequence
  Start* found = reinterpret_cast<Start*>(scratch + 4 * (DS_VIT_MAX_SEQS + 2));
  constexpr int kWarps = kThreads / 32;
  __shared__ int64_t warp_sum[kWarps];
  __shared__ int64_t border[2];
  __shared__ int longest;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto scan = [&](int64_t x, int64_t& total) {      // exclusive prefix over the block
    auto inclusive = [&](int64_t v) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += y;
      }
      return v;
    };
    const int64_t inc = inclusive(x);
    __syncthreads();                        // warp_sum's last readers are done
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    const int64_t sums = inclusive(lane < kWarps ? warp_sum[lane] : 0);
    total = __shfl_sync(0xFFFFFFFFu, sums, kWarps - 1);
    const int64_t before = __shfl_sync(0xFFFFFFFFu, sums, (warp + 31) & 31);
    return (warp > 0 ? before : 0) + inc - x;
  };
  int all = 0;
  for (int s0 = 0; s0 < a.b.n; s0 += kThreads) {
    const int s = s0 + tid;
    int64_t x = 0, t;
    if (s < a.b.n) x = items_of(a, load_seq(a.b, a.c.page_shift, s, status));
    const int64_t before = scan(x, t);
    if (s < a.b.n) items[s] = all + static_cast<int>(before);
    all += static_cast<int>(t);
  }
  if (tid == 0) {
    items[a.b.n] = all;
    longest = 0;
  }
  __syncthreads();
  // This thread's run of the list, and its units.
  const int per = (all + kThreads - 1) / kThreads, i0 = min(all, tid * per), i1 = min(all, i0 + per);
  int s_run = 0;
  if (i0 < i1) {
    int lo = 0, hi = a.b.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (items[mid] <= i0)
        lo = mid;
      else
        hi = mid - 1;
    }
    s_run = lo;
  }
  auto walk = [&](auto&& each) {
    int s = s_run;
    Seq q = load_seq(a.b, a.c.page_shift, s, nullptr);
    for (int i = i0; i < i1; ++i) {
      while (i >= items[s + 1]) q = load_seq(a.b, a.c.page_shift, ++s, nullptr);
      each(s, i - items[s], item_blocks(a, q, i - items[s]).count);
    }
  };
  int64_t mine = 0, total;
  if (i0 < i1) {
    int most = 0;
    walk([&](int, int, int count) {
      mine += static_cast<int64_t>(count + kItemCost) * a.c.kv_heads;
      most = max(most, count + kItemCost);
    });
    atomicMax(&longest, most);
  }
  int64_t at = scan(mine, total);            // its barriers also settle `longest`
  // This CTA's borders, moved to an item's end where one is near.
  const int64_t W = total < gridDim.x ? total : gridDim.x, w = blockIdx.x;
  const Shares shares = deal(total, W);
  const int64_t near = 3 * shares.each / 8;
  const int snap = longest <= kUnsplit && longest <= shares.each + 8 ? kUnsplit
                   : near < kSnap                                    ? static_cast<int>(near)
                                                                     : kSnap;
  const int64_t x0 = w < W ? shares.begin(w) : total, x1 = w < W ? shares.begin(w + 1) : total;
  if (tid == 0) {
    border[0] = border[1] = total;
    *found = Start{};
  }
  __syncthreads();
  if (mine > 0 && ((x0 >= at && x0 < at + mine) || (x1 >= at && x1 < at + mine)))
    walk([&](int s, int k, int count) {
      const int weight = count + kItemCost;
      const int64_t here = static_cast<int64_t>(weight) * a.c.kv_heads;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t x = e == 0 ? x0 : x1;
        if (x < at || x >= at + here) continue;
        const int head = static_cast<int>(x - at < INT32_MAX ? static_cast<uint32_t>(x - at) / static_cast<uint32_t>(weight)
                                                             : (x - at) / weight);
        const int64_t i0 = at + static_cast<int64_t>(head) * weight;
        const int64_t y = snap_border(x, i0, i0 + weight, snap, kItemCost);
        border[e] = y;
        if (e == 0) {
          found->s = s;
          found->k = k;
          found->head = head;
          found->off = static_cast<int>(y - i0);
        }
      }
      at += here;
    });
  __syncthreads();
  Start st = *found;
  st.first = border[0];
  st.units = border[1] - border[0];
  st.total = total;
  st.snap = snap;
  __syncthreads();
  return st;
}

__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The lowest n bits (none for n <= 0, all for n >= 64).
__device__ __forceinline__ uint64_t bits_below(int n) {
  return n <= 0 ? 0 : n >= 64 ? ~uint64_t{0} : (uint64_t{1} << n) - 1;
}

// Address of 16-byte piece `piece` (of D / 8) of row r in a 16-bit tile.
template <int D, bool E4M3>
__device__ __forceinline__ uint32_t tile_piece(uint32_t tile, int r, int piece) {
  return tile + (piece >> 3) * Cfg<D, E4M3>::kHalf + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
}

// The exponent bytes of keys j .. j + 7 of a sequence, from the pages.
__device__ __forceinline__ uint2 exponent_bytes(const AttentionArgs& a, const uint8_t* exps, int s, int head, int j) {
  const int page = __ldg(a.b.table + static_cast<int64_t>(s) * a.b.table_cols + (j >> a.c.page_shift));
  if (!page_there(page, a.c.n_pages)) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  return __ldg(reinterpret_cast<const uint2*>(exps + cache_row(a.c, page, head, j)));
}
__device__ __forceinline__ uint32_t byte_of(uint2 b, int y) { return ((y < 4 ? b.x : b.y) >> (8 * (y & 3))) & 255u; }

template <int D, bool E4M3>
__global__ void __launch_bounds__(Cfg<D, E4M3>::kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ PrefillArgs p) {
  using C = Cfg<D, E4M3>;
  constexpr int kHalves = D / 64;
  const AttentionArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBarCount);
  volatile int* tile_exp = reinterpret_cast<volatile int*>(bars + kBarCount + 1);   // [8] K, [8] V: E of recent tiles
  Job* jobs = reinterpret_cast<Job*>(smem + C::kOffBar + 512);
  const uint32_t base = smem_u32(smem), bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  auto sQ = [&](int x) { return base + x * C::kBytes; };
  auto sKv = [&](int i) { return base + C::kOffKv + i * C::kBytes; };
  auto sRaw = [&](int i) { return base + C::kOffRaw + i * C::kRawBytes; };
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // alike in a warp's lanes

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(kBarQ + x), 256);
      mbar_init(bar(kBarPvDone + x), 1);
    }
    for (int i = 0; i < C::kScores; ++i) {
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarPFull + i), 256);
    }
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(bar(kBarKvFull + i), E4M3 ? 4 : 1);
      mbar_init(bar(kBarKvEmpty + i), 1);
    }
    for (int i = 0; i < C::kRaw; ++i) {
      mbar_init(bar(kBarRawFull + i), 33);       // the tile's bytes, the lanes' copies of exponents
      mbar_init(bar(kBarRawEmpty + i), 4);
    }
    for (int i = 0; i < kJobs; ++i) {
      mbar_init(bar(kBarJobFull + i), 1);
      mbar_init(bar(kBarJobEmpty + i), 18 + (E4M3 ? 8 : 0));   // softmax, TMA, MMA and converter warps
    }
    mbar_init(bar(kBarRagged), 1);
    mbar_init(bar(kBarDrain), 1);
    mbar_init(bar(kBarOther), 256);
    mbar_init(bar(kBarMerged), 256);
    fence_barrier_init();
  }
  if (warp == kWarpTma) {
    if (lane == 0) {
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
    }
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_launch();
  grid_dep_wait();
  const Start st = make_plan<C::kThreads>(a, smem + C::kOffKv, blockIdx.x == 0 ? a.status : nullptr);
  __shared__ int consumed, marked;
  if (threadIdx.x == 0) marked = 0;
  fence_proxy_async_smem();                 // the scratch becomes the ring
  __syncthreads();
  // Job n of the ring: every thread of a role's warp reads it, then one of them hands the slot back.
  auto take = [&](int n, Job& j) {
    const int i = n % kJobs;
    const bool ok = mbar_wait(bar(kBarJobFull + i), (n / kJobs) & 1, a.status);
    const int4* src = reinterpret_cast<const int4*>(jobs + i);
    int4* dst = reinterpret_cast<int4*>(&j);
    dst[0] = src[0], dst[1] = src[1], dst[2] = src[2];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarJobEmpty + i));
    return ok && j.b < j.end;
  };
  float4* other = reinterpret_cast<float4*>(smem + C::kBytes);   // tile B's references and sums, in place of its query rows
  int issued = 0;                           // ring or raw tiles whose loads were issued

  // e4m3: 28 warps start with 72 registers each; 16 x 96 + 12 x 40 is the same sum.
  if (warp >= kWarpTma && (!E4M3 || warp < kWarpConvert)) {
    if constexpr (E4M3) registers_dec<40>();
  if (warp == kWarpTma) {
    // ------------------------------------------------------------ TMA producer
    // Lane i loads page i of a tile (of 128 / page pages).
    const int page = 1 << a.c.page_shift, pages = kTile >> a.c.page_shift;
    constexpr int kDepth = E4M3 ? C::kRaw : C::kRing;
    constexpr int kFull = E4M3 ? kBarRawFull : kBarKvFull, kEmpty = E4M3 ? kBarRawEmpty : kBarKvEmpty;
    int slot = 0, ragged = 0;
    uint32_t phase = 1;
    bool ok = true;
    Job w;
    for (int n = 0; ok && take(n, w); ++n) {
      const int p0 = w.q.kv - w.q.c + a.by_group(w.rho0);
      const int p1 = w.q.kv - w.q.c + a.by_group(min(w.rho0 + kItemRows, w.q.c * a.group) - 1);
      const int lo = window_start(a, p0);
      auto any = [&](int j0, int j1) { return j0 <= p1 && (j1 >= lo || j0 < a.sinks); };   // a key of j0 .. j1 is seen
      auto look = [&](int b) {
        const int key0 = w.kb.at(b) << kTileShift, j = key0 + lane * page;
        if (lane >= pages || !any(j, j + page - 1)) return -2;
        return __ldg(a.b.table + static_cast<int64_t>(w.s) * a.b.table_cols + (j >> a.c.page_shift));
      };
      int next = look(w.b);
      for (int b = w.b; b < w.end; ++b) {
        const int entry = next;
        if (b + 1 < w.end) next = look(b + 1);
        const bool on = page_there(entry, a.c.n_pages);
        if (!on && entry != -2) report_error(a.status, DS_VIT_ERANGE);
        const int loaded = __popc(__ballot_sync(0xFFFFFFFFu, on));
        const int key0 = w.kb.at(b) << kTileShift;
        const int row = on ? static_cast<int>(cache_row(a.c, entry, w.head, 0)) : 0;
        // A value tile with rows that nobody sees: they are zeroed before it is used.
        const bool whole = any(key0, key0) && key0 + kTile - 1 <= p1 && (key0 >= lo || key0 + kTile <= a.sinks) &&
                           loaded == pages;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(kEmpty + slot), phase, a.status));
          if (!ok) break;
          const bool fix = !E4M3 && kv == 1 && !whole;
          const uint32_t full = fix ? bar(kBarRagged) : bar(kFull + slot);
          const uint32_t per = page * D * (E4M3 ? 1 : 2);
          if (lane == 0) mbar_expect_tx(full, loaded * per);
          __syncwarp();
          if (on) {
            const CUtensorMap* tm = kv == 0 ? &tm_k : &tm_v;
            if constexpr (E4M3) {
              tma_load_2d(sRaw(slot) + lane * page * D, tm, full, 0, row);
              const uint8_t* from = (kv == 0 ? a.c.k_exp : a.c.v_exp) + row;
              for (int i = 0; i < page; i += 16) cp_async_16(base + C::kOffExp + slot * kTile + lane * page + i, from + i, 16);
            } else {
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                tma_load_2d(sKv(slot) + h * C::kHalf + lane * page * 128, tm, full, 64 * h, row);
            }
          }
          if constexpr (E4M3) cp_async_arrive(full);
          __syncwarp();
          if (fix) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(kBarRagged), ragged & 1, a.status));
            if (!ok) break;
            ++ragged;
            const uint32_t loads = __ballot_sync(0xFFFFFFFFu, on);
            for (int x = lane; x < kTile * 8 * kHalves; x += 32) {
              const int r = (x >> 3) & (kTile - 1), j = key0 + r;
              if (!any(j, j) || !((loads >> (r >> a.c.page_shift)) & 1u)) sts128(sKv(slot) + 16 * x, make_uint4(0, 0, 0, 0));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kFull + slot));
            __syncwarp();
          }
          ++issued;
          if (++slot == kDepth) {
            slot = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
      }
    }
    if constexpr (E4M3) cp_async_wait<0>();  // no copy lands after the CTA has exited
  } else if (warp == kWarpJobs) {
    // ------------------------------------------------------------ the items
    if (lane == 0) {
      SplitHeader header{};
      Walk w;
      w.start(a, st);
      for (int n = 0;; ++n) {
        const int i = n % kJobs;
        if (!mbar_wait(bar(kBarJobEmpty + i), ((n / kJobs) & 1) ^ 1, a.status)) break;
        const bool more = w.left > 0;
        const bool whole = more && w.b == 0 && w.end == w.kb.count;
        jobs[i] = more ? Job{w.s, w.head, w.k * kItemRows, whole ? 1 : w.b > 0 ? 2 : 0, w.q, w.b, w.kb, w.end} : Job{};
        mbar_arrive(bar(kBarJobFull + i));
        if (!more) break;
        if (!whole && w.b == 0) {
          const Shares shares = deal(st.total, st.total < gridDim.x ? st.total : gridDim.x);
          const int64_t i0 = st.first + st.units - w.left, i1 = i0 + w.kb.count + kItemCost;
          int64_t last = shares.owner(i1 - 1);       // the last worker whose border is not at or behind the end
          while (last > blockIdx.x && snap_border(shares.begin(last), i0, i1, st.snap, kItemCost) >= i1) --last;
          header = SplitHeader{static_cast<int>(last - blockIdx.x) + 1, w.s, w.head, w.k * kItemRows, w.q, 0};
        }
        w.next(a);
      }
      p.rec.headers[blockIdx.x] = header;
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    // Tile by tile in turn, P V of a step and S of the next together: one tile's
    // pair runs while the other's softmax works.  The whole warp walks along, all
    // it decides by being alike in its lanes (see umma_bf16_if).  A chunk of 2048
    // over 32k keys, us, calls back to back: 957 so; 1100 with one lane issuing; 1130 with an issuer for
    // each tile, whose pairs interleave (and the exponents of the two tiles taking
    // turns, which this order makes needless); 1357 when whatever is ready goes first.
    constexpr uint32_t f16_bits = (1u << 7) | (1u << 10);   // bf16 marks of A and B in the instruction descriptor
    constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false) & ~(E4M3 ? f16_bits : 0u);
    constexpr uint32_t id_o = idesc_bf16_f32(128, D, false, true) & ~(E4M3 ? f16_bits : 0u);   // V is MN-major
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0), go = elect_one();
    const uint64_t dq0 = sdesc_sw128(sQ(0), 16, 1024);
    const uint64_t dk0 = sdesc_sw128(sKv(0), 16, 1024);
    const uint64_t dv0 = sdesc_sw128(sKv(0), C::kHalf, 1024);
    int slot = 0, used = 0;
    uint32_t phase = 0, q0 = 0, q1 = 0, step0 = 0, step1 = 0, seq = 0;
    auto wait = [&](int i, uint32_t parity) { return __all_sync(0xFFFFFFFFu, mbar_wait(bar(i), parity, a.status)); };
    auto advance = [&]() {
      ++used;
      if (++slot == C::kRing) {
        slot = 0;
        phase ^= 1;
      }
    };
    auto issue_s = [&](int x, int at, int tile) {        // into score tile `tile`
      const uint64_t dq = dq0 + static_cast<uint64_t>(x * (C::kBytes >> 4));
      const uint64_t dk = dk0 + static_cast<uint64_t>(at * (C::kBytes >> 4));
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint64_t off = (k >> 2) * (C::kHalf >> 4) + 2 * (k & 3);
        umma_bf16_if(go, tm + tile * 128, dq + off, dk + off, id_s, k != 0);
      }
      umma_commit_if(go, bar(kBarSFull + tile));
    };
    auto issue_pv = [&](int x, int at, bool fresh, int tile) {
      const uint64_t dv = dv0 + static_cast<uint64_t>(at * (C::kBytes >> 4));
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        umma_bf16_ts_if(go, tm + C::kTmemO + x * D, tm + tile * 128 + k * 8, dv + 128 * k, id_o, !fresh | (k != 0));   // 16 rows = 2048 B
      umma_commit_if(go, bar(kBarPvDone + x));
    };
    // Place of a tile `ahead` of the next in the ring, and whether it has been filled.
    auto place = [&](int ahead) { return slot + ahead < C::kRing ? slot + ahead : slot + ahead - C::kRing; };
    auto there = [&](int ahead) {
      return wait(kBarKvFull + place(ahead), slot + ahead < C::kRing ? phase : phase ^ 1);
    };
    auto release = [&](int at) { umma_commit_if(go, bar(kBarKvEmpty + at)); };
    Job w;
    for (int n = 0; __all_sync(0xFFFFFFFFu, take(n, w)); ++n) {
      const bool both = __shfl_sync(0xFFFFFFFFu, w.q.c * a.group - w.rho0, 0) > kTile;
      const int count = __shfl_sync(0xFFFFFFFFu, w.end - w.b, 0);
      bool ok = true;
      if constexpr (C::kScores == 3) {
        // Products n = 0, 1, ... of the item, A's and B's in turn, use score tiles seq + n
        // mod 3: S of n + 3 follows P V of n, so that a softmax finds its next scores ready.
        const int products = both ? 2 * count : count;
        const uint32_t base = used;
        auto at = [&](int i) { return static_cast<int>((base + i) % C::kRing); };
        auto filled = [&](int i) { return wait(kBarKvFull + at(i), ((base + i) / C::kRing) & 1); };
        auto scores = [&](int n) {
          const int x = n & 1, i = both ? n & ~1 : 2 * n;       // the keys' place
          if (!filled(i)) return false;
          if (n < 2) {
            if (!wait(kBarQ + x, x == 0 ? q0 : q1)) return false;
            (x == 0 ? q0 : q1) ^= 1;
          }
          issue_s(x, at(i), (seq + n) % 3);
          if (!both || x == 1) release(at(i));
          return true;
        };
        for (int n = 0; ok && n < 3 && n < products; ++n) ok = scores(n);
        for (int n = 0; ok && n < products; ++n) {
          const int x = n & 1, i = (both ? n & ~1 : 2 * n) + 1;
          const uint32_t step = x == 0 ? step0++ : step1++;
          const int score = (seq + n) % 3;
          ok = filled(i) && wait(kBarPFull + score, ((seq + n) / 3) & 1);
          if (!ok) break;
          issue_pv(x, at(i), n < 2, score);
          if (!both || x == 1) {
            release(at(i));
            used = base + i + 1;
          }
          if (n + 3 < products) ok = wait(kBarPvDone + x, step & 1) && scores(n + 3);
        }
        seq += products;
      } else if (both) {
        if (!there(0) || !wait(kBarQ, q0)) break;
        issue_s(0, slot, 0);
        if (!wait(kBarQ + 1, q1)) break;
        issue_s(1, slot, 1);
        release(slot);
        q0 ^= 1;
        q1 ^= 1;
        advance();
        for (int b = 0; b < count; ++b) {
          const bool more = b + 1 < count;
          const int v_slot = slot;
          ok = there(0);
          advance();
          ok = ok && wait(kBarPFull, step0 & 1);
          if (!ok) break;
          issue_pv(0, v_slot, b == 0, 0);
          if (more) {
            // S_X overwrites P_X: its product must be complete.
            ok = there(0) && wait(kBarPvDone, step0 & 1);
            if (!ok) break;
            issue_s(0, slot, 0);
          }
          ++step0;
          ok = wait(kBarPFull + 1, step1 & 1);
          if (!ok) break;
          issue_pv(1, v_slot, b == 0, 1);
          release(v_slot);
          if (more) {
            ok = wait(kBarPvDone + 1, step1 & 1);
            if (!ok) break;
            issue_s(1, slot, 1);
            release(slot);
            advance();
          }
          ++step1;
        }
      } else {
        // Key tiles 0, 2, .. are tile A's, 1, 3, .. tile B's.  The ring holds K0 V0 K1
        // V1 ...; `slot` stays at the values of the step.
        if (!there(0) || !wait(kBarQ, q0)) break;
        q0 ^= 1;
        issue_s(0, slot, 0);
        release(slot);
        advance();
        if (C::kShare && count > 1) {
          if (!there(1) || !wait(kBarQ + 1, q1)) break;
          q1 ^= 1;
          issue_s(1, place(1), 1);
          release(place(1));
        }
        constexpr int kTurns = C::kShare ? 2 : 1;
        auto turn = [&](int x, uint32_t& step, int b) {
          if (!there(0) || !wait(kBarPFull + x, step & 1)) return false;
          issue_pv(x, slot, b < kTurns, x);
          release(slot);
          if (b + kTurns < count) {
            if (!there(2 * kTurns - 1) || !wait(kBarPvDone + x, step & 1)) return false;
            issue_s(x, place(2 * kTurns - 1), x);
            release(place(2 * kTurns - 1));
          }
          ++step;
          advance();
          if (b + 1 < count) advance();
          return true;
        };
        for (int b = 0; ok && b < count; ++b) ok = kTurns == 1 || (b & 1) == 0 ? turn(0, step0, b) : turn(1, step1, b);
      }
      if (!ok) break;
    }
    if (lane == 0) consumed = used;
    // All MMAs complete before TMEM is released.
    umma_commit_if(go, bar(kBarDrain));
    mbar_wait(bar(kBarDrain), 0, a.status);
  }
  } else if (E4M3 && warp >= kWarpConvert) {
    if constexpr (E4M3) registers_dec<40>();
    // ------------------------------------------------------------ e4m3 -> fp16
    // Four warps take the key tiles and four the value tiles (four for both were
    // what the rest waited for: 5500 cycles a step of 256 rows x 128 keys).
    const int part = (warp - kWarpConvert) / 4, wc = (warp - kWarpConvert) % 4;
    const int tid = 32 * wc + lane;
    // A thread takes 16-byte piece `piece` of rows r0, r0 + kStep, ...: their
    // places differ by constants (kStep is a multiple of the swizzle's 8 rows).
    constexpr int kPieces = D / 16, kStep = 128 / kPieces, kEach = 32 / kPieces;
    const int piece = tid % kPieces, r0 = tid / kPieces, second = (piece >> 2) & 1;
    const uint32_t raw_at = r0 * D + ((D == 128 ? piece ^ (r0 & 7) : piece ^ ((r0 >> 1) & 3)) << 4);
    const uint32_t tile_at0 = tile_piece<D, E4M3>(0, r0, 2 * piece + second);
    const uint32_t tile_at1 = tile_piece<D, E4M3>(0, r0, 2 * piece + 1 - second);
    int tile = 0;
    bool ok = true;
    Job w;
    for (int n = 0; ok && take(n, w); ++n) {
      const int p0 = w.q.kv - w.q.c + a.by_group(w.rho0);
      const int p1 = w.q.kv - w.q.c + a.by_group(min(w.rho0 + kItemRows, w.q.c * a.group) - 1);
      const int lo = window_start(a, p0);
      auto any = [&](int j) { return j <= p1 && (j >= lo || j < a.sinks); };
      for (int b = w.b; b < w.end; ++b, ++tile) {
        const int key0 = w.kb.at(b) << kTileShift;
        {
          const uint32_t count = 2 * static_cast<uint32_t>(tile) + part;     // tiles before this one
          const int raw = count % C::kRaw, slot = count % C::kRing;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(kBarRawFull + raw), (count / C::kRaw) & 1, a.status));
          if (!ok) break;
          const uint8_t* ex = smem + C::kOffExp + raw * kTile;
          // The largest and the least exponent among rows that some row sees (255 marks
          // a NaN row), and the factor of one of this warp's 32 rows: lane y has row
          // kStep (y / kEach) + kEach wc + y % kEach.
          int top = 0, least = 255;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int r = 32 * y + lane, e = ex[r];
            if (any(key0 + r) && e != 255) {
              top = max(top, e);
              least = min(least, e);
            }
          }
          top = __reduce_max_sync(0xFFFFFFFFu, top);
          least = __reduce_min_sync(0xFFFFFFFFu, least);
          const bool far = top - least > (part == 0 ? kSpanK : kSpanV);
          if (top == 0) top = 127;
          uint32_t factor;
          {
            const int r = kStep * (lane / kEach) + kEach * wc + lane % kEach;
            const int e = ex[r], down = far ? 0 : top - e;
            factor = e == 255 ? 0x3C00u : down <= 14 ? (15u - down) << 10 : down <= 24 ? 1u << (24 - down) : 0u;
            factor = any(key0 + r) ? factor | factor << 16 : 0xFFFFFFFFu;      // marks a row that nobody sees
          }
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(kBarKvEmpty + slot), ((count / C::kRing) & 1) ^ 1, a.status));
          if (!ok) break;
          if (tid == 0) tile_exp[8 * part + (tile & 7)] = far ? kFar : top - 127;
          const uint32_t from = sRaw(raw) + raw_at;
          const uint32_t to0 = sKv(slot) + tile_at0, to1 = sKv(slot) + tile_at1;
#pragma unroll
          for (int y = 0; y < 32 / kEach; ++y) {
            const uint4 v = lds128(from + y * kStep * D);
            const uint32_t f = __shfl_sync(0xFFFFFFFFu, factor, y * kEach + lane / kPieces);
            uint4 u0, u1;
            u0.x = mul_f16x2(e4m3x2_to_f16x2(v.x & 0xFFFFu), f), u0.y = mul_f16x2(e4m3x2_to_f16x2(v.x >> 16), f);
            u0.z = mul_f16x2(e4m3x2_to_f16x2(v.y & 0xFFFFu), f), u0.w = mul_f16x2(e4m3x2_to_f16x2(v.y >> 16), f);
            u1.x = mul_f16x2(e4m3x2_to_f16x2(v.z & 0xFFFFu), f), u1.y = mul_f16x2(e4m3x2_to_f16x2(v.z >> 16), f);
            u1.z = mul_f16x2(e4m3x2_to_f16x2(v.w & 0xFFFFu), f), u1.w = mul_f16x2(e4m3x2_to_f16x2(v.w >> 16), f);
            if (f == 0xFFFFFFFFu) u0 = u1 = make_uint4(0, 0, 0, 0);
            // Lanes of the two halves of the dims store their two pieces in opposite orders: no bank conflicts.
            sts128(to0 + y * kStep * 128, second ? u1 : u0);
            sts128(to1 + y * kStep * 128, second ? u0 : u1);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(kBarRawEmpty + raw));
            mbar_arrive(bar(kBarKvFull + slot));
          }
        }
      }
    }
  } else {
    if constexpr (E4M3) registers_inc<96>();
    // ------------------------------------------------------------ softmax (warps 0-15)
    const int x = warp >> 3;                 // query tile A (0) or B (1)
    const int row0 = (warp & 3) * 32 + ((warp >> 2) & 1) * 16;   // the warp's first row
    const int h = lane >> 4;                 // 64-key half of the score tile
    const int r = row0 + (lane & 15);        // row inside the tile == TMEM lane
    const uint32_t lane_sel = static_cast<uint32_t>(row0) << 16;
    uint32_t tS = tmem + x * 128 + lane_sel;
    const uint32_t tO = tmem + C::kTmemO + x * D + lane_sel;
    uint32_t step = 0, merges = 0, seq = 0;      // seq: as the MMA issuer's
    int tile = 0;
    bool ok = true;
    Job w;
    for (int n = 0; ok && take(n, w); ++n) {
      const int R = w.q.c * a.group, count = w.end - w.b;
      // Tile B without rows of its own takes A's rows and every other key tile.
      const bool shared = C::kShare && R - w.rho0 <= kTile;
      const int rho0 = shared ? w.rho0 : w.rho0 + x * kTile;   // first row of the tile
      const int stride = shared ? 2 : 1, b0 = shared ? w.b + x : w.b;
      const uint32_t seq0 = seq;
      seq += R - w.rho0 <= kTile ? count : 2 * count;
      if (rho0 >= R || b0 >= w.end) {
        tile += count;
        if constexpr (C::kScores == 3) {
          // Nothing for B here; it waits for A all the same.  Score tiles go round between
          // the two, and a wait of B's must not come before A's use of the tile is complete.
          mbar_arrive(bar(kBarOther));
          if (!mbar_wait(bar(kBarMerged), merges & 1, a.status)) {
            ok = false;
            break;
          }
          ++merges;
        }
        continue;
      }
      const int first = w.q.kv - w.q.c;
      // ---- the warp's 16 query rows: lane l takes piece l % kPieces of rows l / kPieces, + kEach, ...
      float c0 = a.scale_log2;
      {
        constexpr int kPieces = D / 8, kEach = 32 / kPieces;
        const int piece = lane % kPieces;
        uint4 v[16 / kEach];
#pragma unroll
        for (int y = 0; y < 16 / kEach; ++y) {
          const int rho = rho0 + row0 + y * kEach + lane / kPieces, i = a.by_group(rho);
          const bf16* src = a.q + (w.q.row0 + i) * a.q_stride + (w.head * a.group + rho - i * a.group) * D + piece * 8;
          v[y] = rho < R ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int y = 0; y < 16 / kEach; ++y) {
          if constexpr (E4M3) {
            uint32_t top = __vmaxu2(__vmaxu2(v[y].x & 0x7FFF7FFFu, v[y].y & 0x7FFF7FFFu),
                                    __vmaxu2(v[y].z & 0x7FFF7FFFu, v[y].w & 0x7FFF7FFFu));
            top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
            for (int o = kPieces / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            // The largest's exponent field E: times 2^(141 - E), in two steps of normal powers of two.
            const int E = max(static_cast<int>(top >> 7), 1), up = 141 - E, half = up / 2;
            const float f0 = __int_as_float((127 + half) << 23), f1 = __int_as_float((127 + up - half) << 23);
            auto to16 = [&](uint32_t two) { return pack_f16x2(bf16lo(two) * f0 * f1, bf16hi(two) * f0 * f1); };
            v[y] = make_uint4(to16(v[y].x), to16(v[y].y), to16(v[y].z), to16(v[y].w));
            // The row's own threads scale its scores back.
            const int mine = __shfl_sync(0xFFFFFFFFu, up, (lane % kEach) * kPieces);
            if ((lane & 15) / kEach == y)
              c0 = a.scale_log2 * __int_as_float((127 - mine / 2) << 23) * __int_as_float((127 - mine + mine / 2) << 23);
          }
          sts128(tile_piece<D, E4M3>(sQ(x), row0 + y * kEach + lane / kPieces, piece), v[y]);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(kBarQ + x));
      const int rho = rho0 + r;
      const int pos = rho < R ? first + a.by_group(rho) : -1;
      // Positions of the tile's first and last rows, for tiles without a mask.
      const int pa = first + a.by_group(rho0), pb = first + a.by_group(min(rho0 + kTile, R) - 1);
      const int lo = window_start(a, pos), lo_b = window_start(a, pb);

      float m = -INFINITY, d = 0.f, l = 0.f;      // d: e4m3, see Raise
      for (int b = b0; b < w.end; b += stride, ++step) {
        const int key0 = w.kb.at(b) << kTileShift, nth = tile + (b - w.b);     // the CTA's tiles before this one
        const bool open = key0 + kTile - 1 <= pa && (key0 >= lo_b || key0 + kTile <= a.sinks);
        int at = x;
        uint32_t use = step;
        if constexpr (C::kScores == 3) {
          const uint32_t n = seq0 + (shared ? b - w.b : 2 * (b - w.b) + x);
          at = n % 3, use = n / 3;
          tS = tmem + at * 128 + lane_sel;
        }
        if (!mbar_wait(bar(kBarSFull + at), use & 1, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float c = c0, ev = 0.f;
        int ek = 0, e = 0;
        if constexpr (E4M3) {
          // E(V) is known once the value tile is there (it stays until P V).
          const uint32_t nv = 2 * static_cast<uint32_t>(nth) + 1;
          if (!mbar_wait(bar(kBarKvFull + nv % C::kRing), (nv / C::kRing) & 1, a.status)) {
            ok = false;
            break;
          }
          ek = tile_exp[nth & 7], e = tile_exp[8 + (nth & 7)];
          // Not zero: a masked score of -inf stays -inf.
          if (ek != kFar) c = fmaxf(c * __int_as_float((ek + 127) << 23), 1e-35f);
          ev = static_cast<float>(e);
        }
        // Key y of this half is seen when y <= last and (y >= from or y < keep): one bit each.
        const int j0 = key0 + 64 * h;
        auto seen_keys = [&](int last, int from, int j) {
          return bits_below(last - j + 1) & (~bits_below(from - j) | bits_below(a.sinks - j));
        };
        // O_X times alpha.  With a score tile each, S_X waited for the product that wrote O_X last.
        // With three, a warp may come here before that product was even issued (others of
        // its tile being a step behind).  The item's last step waits for it in any case: a warp two
        // products ahead would mistake the parity of the last but two for the last one's
        // at the item's end and leave without both.
        auto rescale = [&](float alpha) {
          const bool change = __any_sync(0xFFFFFFFFu, alpha != 1.f);
          if (b == b0 || !(change || (C::kScores == 3 && b + stride >= w.end))) return;
          if (C::kScores == 3) {
            if (!mbar_wait(bar(kBarPvDone + x), (step - 1) & 1, a.status)) ok = false;
            tc_fence_after();
          }
          if (!change) return;
#pragma unroll
          for (int y = 0; y < D / 64; ++y) {
            uint32_t o[32];
            tmem_ld32_x2<D / 2>(tO + 32 * y, o);
            tmem_wait_ld();
#pragma unroll
            for (int z = 0; z < 32; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * alpha);
            tmem_st32_x2<D / 2>(tO + 32 * y, o);
          }
        };
        const bool far = E4M3 && (ek == kFar || e == kFar);
        if (far) {
          // A tile with factors by key.  The weights are added up here; for the products, the
          // scores give way to those of the contributions (score + e - the row's largest e).
          // Eight keys at a time, for few registers (out of line or all at once it took
          // from every tile: a tail chunk 116 and 138 us, 111 so, 108.5 without).  Such a
          // tile takes some five times as long as another (a tail chunk with a zero value row
          // in every 16 tokens, so that all are: 501 us).
          // Copies, so that nothing of this is computed ahead of the loop and kept.
          int seq_no = w.s, head = w.head, last = pos, from = lo, j1 = j0;
          asm volatile("" : "+r"(seq_no), "+r"(head), "+r"(last), "+r"(from), "+r"(j1));
          const uint64_t seen = seen_keys(last, from, j1);
          float s8[8], top = -INFINITY, largest = -INFINITY;
          auto load = [&](int g) {
            uint32_t r8[8];
            __syncwarp();
            tmem_ld8_x2<64>(tS + g, r8);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 8; ++y) s8[y] = tmem_after_wait(__uint_as_float(r8[y]));
          };
          auto store = [&](int g) {
            uint32_t r8[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) r8[y] = __float_as_uint(s8[y]);
            __syncwarp();
            tmem_st8_x2<64>(tS + g, r8);
          };
          // Exponent bytes of keys g .. g + 7, of which some are seen (they lie in a page then).
          auto bytes = [&](const uint8_t* exps, int g) {
            return (seen >> g) & 255u ? exponent_bytes(a, exps, seq_no, head, j1 + g) : make_uint2(0, 0);
          };
          auto value_exponent = [&](uint2 v, int y) {
            return e == kFar ? static_cast<float>(static_cast<int>(byte_of(v, y)) - 127) : static_cast<float>(e);
          };
#pragma unroll 1
          for (int g = 0; g < 64; g += 8) {
            const uint2 kb = bytes(a.c.k_exp, g), vb = bytes(a.c.v_exp, g);
            load(g);
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              const bool on = (seen >> (g + y)) & 1u;
              const float f = ek == kFar ? c0 * __uint_as_float(byte_of(kb, y) << 23) : c;
              s8[y] = on ? s8[y] * f : -INFINITY;
              top = fmaxf(top, s8[y]);
              if (on) largest = fmaxf(largest, value_exponent(vb, y));
            }
            store(g);
          }
          tmem_wait_st();
          largest = fmaxf(largest, __shfl_xor_sync(0xFFFFFFFFu, largest, 16));
          ev = fminf(fmaxf(largest, -127.f), 120.f);       // 128: a row of NaN
          const Raise up = raised(m, d, fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16)), -INFINITY);
          m = up.m, d = up.d, l *= up.l;
          rescale(up.o);
#pragma unroll 1
          for (int g = 0; g < 64; g += 8) {
            const uint2 vb = bytes(a.c.v_exp, g);
            load(g);
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              if (s8[y] == -INFINITY) continue;            // hidden, its value's exponent may be anything
              l += ex2_approx(s8[y] - m);
              s8[y] += value_exponent(vb, y) - ev;
            }
            store(g);
          }
          tmem_wait_st();
          c = 1.f;
        }
        uint32_t sr[64];
        float top = tmem_ld32_max_x2<64>(tS, sr), top2 = tmem_ld32_max_x2<64>(tS + 32, sr + 32);
        tmem_wait_ld();
        top = fmaxf(tmem_after_wait(top), tmem_after_wait(top2));
        if (!open) {
          const uint64_t seen = seen_keys(pos, lo, j0);
          const uint32_t s0 = static_cast<uint32_t>(seen), s1 = static_cast<uint32_t>(seen >> 32);
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int y = 0; y < 64; ++y) {
            if (!((y < 32 ? s0 : s1) & (1u << (y & 31)))) sr[y] = __float_as_uint(-INFINITY);
            mx[y & 3] = fmaxf(mx[y & 3], __uint_as_float(sr[y]));
          }
          top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        }
        // Both threads of the row derive the same reference.
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
        const float reach = top * c;
        float alpha = 1.f, off, unit = 1.f;  // alpha: of the outputs so far
        if constexpr (E4M3) {
          const Raise up = raised(m, d, reach, reach + ev);
          m = up.m, d = up.d, alpha = up.o, l *= up.l;
          // Operands 2^(z + x); their sum is scaled back by 2^-x.  Under -60 (a tile of
          // values far below the row's largest) they are zeros in fp16 all the same.
          const float x = fmaxf(ev - d, -60.f);
          off = m == -INFINITY ? 0.f : x - m;
          unit = far ? 0.f : __int_as_float(max(127 - static_cast<int>(x), 0) << 23);
        } else {
          if (reach > m + C::kLag16) {       // always true on the first visible key (m = -inf)
            alpha = ex2_approx(m - reach);
            m = reach;
          }
          off = m == -INFINITY ? 0.f : -m;
        }
        const uint64_t c2 = f2(c, c), nm2 = f2(off, off);
        uint64_t acc[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
        uint32_t pk[32];
#pragma unroll
        for (int y = 0; y < 32; ++y) {
          const uint64_t z = f2_fma(f2(__uint_as_float(sr[2 * y]), __uint_as_float(sr[2 * y + 1])), c2, nm2);
          float z0, z1;
          f2_split(z, z0, z1);
          z0 = ex2_approx(z0);
          z1 = ex2_approx(z1);
          acc[y & 3] = f2_add(acc[y & 3], f2(z0, z1));
          // The product's operand: weights in 16 bits (their sum stays in fp32).
          pk[y] = E4M3 ? pack_f16x2(z0, z1) : pack_bf16x2(z0, z1);
        }
        const uint64_t s2 = f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3]));
        float s0, s1;
        f2_split(s2, s0, s1);
        // This half's share of the row sum.
        l = E4M3 ? fmaf(s0 + s1, unit, l) : fmaf(l, alpha, s0 + s1);
        tmem_st32_x2<32>(tS, pk);
        rescale(alpha);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kBarPFull + at));
      }
      if (!ok || !mbar_wait(bar(kBarPvDone + x), (step - 1) & 1, a.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // ---- the item's end: finished here, or a record for the join.  The rows go
      // through their place in the Q tile (its products are complete), 16 bytes a
      // piece, and leave as whole rows.
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
      tile += count;
      float fa = 1.f, fb = 0.f;              // what the tiles' outputs are weighed by
      const bool two = shared && count > 1, paired = shared && (two || C::kScores == 3);
      if (paired) {
        if (x == 1) {
          if (h == 0) other[r] = make_float4(m, d, l, 0.f);
          tc_fence_before();
          mbar_arrive(bar(kBarOther));
          if (!mbar_wait(bar(kBarMerged), merges & 1, a.status)) {
            ok = false;
            break;
          }
          ++merges;
          tc_fence_after();
          continue;
        }
        if (!mbar_wait(bar(kBarOther), merges & 1, a.status)) {
          ok = false;
          break;
        }
        ++merges;
        tc_fence_after();
        if (two) {
          const float4 b = other[r];
          const float to_m = fmaxf(m, b.x), to_d = E4M3 ? shift_at(to_m, fmaxf(m + d, b.x + b.y)) : 0.f;
          fa = output_factor<E4M3>(m, d, to_m, to_d);
          fb = output_factor<E4M3>(b.x, b.y, to_m, to_d);
          l = l * sum_factor<E4M3>(m, to_m) + b.z * sum_factor<E4M3>(b.x, to_m);
          m = to_m, d = to_d;
        }
      }
      // Columns col .. of the row's output (kCols of each half of the dims).
      auto load_o = [&](auto cols, int col, uint32_t* o) {
        constexpr int kCols = decltype(cols)::value;
        if constexpr (kCols == 32)
          tmem_ld32_x2<D / 2>(tO + col, *reinterpret_cast<uint32_t(*)[32]>(o));
        else
          tmem_ld16_x2<D / 2>(tO + col, o);
        tmem_wait_ld();
        if (two) {
#pragma unroll
          for (int c1 = 0; c1 < kCols; c1 += 16) {
            uint32_t o2[16];
            tmem_ld16_x2<D / 2>(tO + D + col + c1, o2);
            tmem_wait_ld();
#pragma unroll
            for (int z = 0; z < 16; ++z)
              o[c1 + z] = __float_as_uint(fmaf(__uint_as_float(o[c1 + z]), fa, __uint_as_float(o2[z]) * fb));
          }
        }
      };
      if (w.whole == 1) {
        const float inv = 1.f / l, up = E4M3 ? shift_up(d) : 1.f;
        bool bad = false;
#pragma unroll 1
        for (int y = 0; y < D / 64; ++y) {
          uint32_t o[32];
          load_o(std::integral_constant<int, 32>{}, 32 * y, o);
#pragma unroll
          for (int z = 0; z < 16; ++z) {
            const float o0 = __uint_as_float(o[2 * z]) * inv * up, o1 = __uint_as_float(o[2 * z + 1]) * inv * up;
            bad |= not_finite(o0) || not_finite(o1);
            o[z] = pos < 0 ? 0u : pack_bf16x2(o0, o1);
          }
#pragma unroll
          for (int z = 0; z < 4; ++z)
            sts128(tile_piece<D, E4M3>(sQ(x), r, h * (D / 16) + 4 * y + z),
                   make_uint4(o[4 * z], o[4 * z + 1], o[4 * z + 2], o[4 * z + 3]));
        }
        __syncwarp();
        constexpr int kPieces = D / 8, kEach = 32 / kPieces;
#pragma unroll
        for (int y = 0; y < 16 / kEach; ++y) {
          const int rr = row0 + y * kEach + lane / kPieces, piece = lane % kPieces;
          const int i = a.by_group(rho0 + rr);
          const uint4 v = lds128(tile_piece<D, E4M3>(sQ(x), rr, piece));
          if (rho0 + rr < R)
            *reinterpret_cast<uint4*>(a.out + (w.q.row0 + i) * a.out_stride +
                                      (w.head * a.group + rho0 + rr - i * a.group) * D + piece * 8) = v;
        }
        if (w.q.c > 1 && bad && pos >= 0) marked = 1;      // a row that sees nothing has no sum
      } else {
        float* rec = p.rec.at(blockIdx.x, w.whole == 2 ? 0 : 1);
        if (h == 0) {
          p.rec.max_of(rec, D)[x * kTile + r] = m;
          p.rec.sum_of(rec, D)[x * kTile + r] = l;
          if constexpr (E4M3) p.rec.shift_of(rec, D)[x * kTile + r] = d;
        }
        // Passes of kCols columns of each half of the dims: a row's place holds both.
        constexpr int kCols = D / 4;
#pragma unroll 1
        for (int y = 0; y < D / 2; y += kCols) {
          uint32_t o[32];
          load_o(std::integral_constant<int, kCols>{}, y, o);
          __syncwarp();                      // the last pass has been read
#pragma unroll
          for (int z = 0; z < kCols / 4; ++z)
            sts128(tile_piece<D, E4M3>(sQ(x), r, h * (kCols / 4) + z),
                   make_uint4(o[4 * z], o[4 * z + 1], o[4 * z + 2], o[4 * z + 3]));
          __syncwarp();
          constexpr int kPieces = kCols / 2, kEach = 32 / kPieces;      // pieces of a row's place
#pragma unroll
          for (int z = 0; z < 16 / kEach; ++z) {
            const int rr = row0 + z * kEach + lane / kPieces, piece = lane % kPieces;
            const int d0 = (piece / (kPieces / 2)) * (D / 2) + y + 4 * (piece % (kPieces / 2));
            *reinterpret_cast<uint4*>(rec + static_cast<int64_t>(x * kTile + rr) * D + d0) =
                lds128(tile_piece<D, E4M3>(sQ(x), rr, piece));
          }
        }
      }
      tc_fence_before();
      if (paired) mbar_arrive(bar(kBarMerged));
      __syncwarp();                          // the rows' places are free for the next item's
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpTma && status_failed(a.status)) {
    // After an error: wait (bounded) for the loads that may still be in flight,
    // so no TMA write lands in shared memory after the CTA has exited.
    constexpr int kDepth = E4M3 ? C::kRaw : C::kRing;
    constexpr int kFull = E4M3 ? kBarRawFull : kBarKvFull;
    const int done = E4M3 ? max(0, issued - kDepth) : consumed;
    for (int j = done; j < issued; ++j)
      if (!mbar_wait(bar(kFull + j % kDepth), (j / kDepth) & 1, nullptr)) break;
  }
  __syncthreads();
  if (warp == kWarpTma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 32 * kWarpJobs) p.rec.headers[blockIdx.x].marked = marked;
}

// Adds up the records of the split items and writes their rows: all those rows in one
// list, dealt to the warps of one wave of blocks (51 and 115 rows, 32 query and 4 K/V heads,
// over 23 and 43 thousand tokens, 24 items in 152 parts: 8 us, eight parts
// of a row in flight instead of four 12; with blocks bound to
// items it took 16).  Where the rows are few, the warps of a block share a row's parts.
constexpr int kMaxCtas = 256;        // of the kernel above; a thread here looks at each
constexpr int kJoinBlocks = 4;       // per SM

// All rows of whole items that are not finite: computed again where they have to be.  A rare
// pass over the whole output, by all warps of the join; out of line, and looking up what
// belongs to a row, for the join's registers (walking the shares' items, 3 us a tail chunk).
template <int D, bool E4M3>
__device__ __noinline__ void mend_rows(const AttentionArgs& a, const SplitHeader* heads, int workers, int warp, int lane) {
  const int64_t total = static_cast<int64_t>(a.b.rows) * a.heads, step = static_cast<int64_t>(gridDim.x) * kJoinWarps;
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * kJoinWarps + warp; x < total; x += step) {
    const int r = static_cast<int>(x / a.heads), h = static_cast<int>(x - static_cast<int64_t>(r) * a.heads);
    if (!row_not_finite<D>(a, r, h, lane)) continue;
    const int s = find_seq(a.b, r, lane);
    if (s < 0) continue;
    const Seq q = load_seq(a.b, a.c.page_shift, s, nullptr);
    const int i = r - q.row0, head = h / a.group;
    if (i < 0 || i >= q.c || q.c <= 1) continue;
    const int k = (i * a.group + h - head * a.group) / kItemRows;
    bool split = false;                      // its rows are being joined: they are looked at there
    for (int w = lane; w < workers; w += 32)
      split |= heads[w].parts != 0 && heads[w].s == s && heads[w].head == head && heads[w].rho0 == k * kItemRows;
    if (__any_sync(0xFFFFFFFFu, split)) continue;
    int p0, p1;
    item_positions(a, q, k, p0, p1);
    mend_row<D, E4M3>(a, s, q.row0, q.kv - q.c + i, i, h, p0, p1, lane);
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kJoinWarps, kJoinBlocks)
    join_items_kernel(const __grid_constant__ AttentionArgs a, const Records rec, int workers) {
  static_assert(kMaxCtas == 32 * kJoinWarps, "a thread per worker");
  __shared__ SplitHeader heads[kMaxCtas];
  __shared__ int before[kMaxCtas];     // rows of the workers before each
  __shared__ int sums[kJoinWarps];
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < 2 * workers; i += 32 * kJoinWarps)
    reinterpret_cast<int4*>(heads)[i] = reinterpret_cast<const int4*>(rec.headers)[i];
  __syncthreads();
  int rows = 0;
  if (tid < workers && heads[tid].parts != 0)
    rows = min(heads[tid].q.c * a.group - heads[tid].rho0, kItemRows);
  int inc = rows;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sums[warp] = inc;
  const bool marks = __syncthreads_or(tid < workers && heads[tid].marked);
  int total = 0, ahead = 0;
#pragma unroll
  for (int y = 0; y < kJoinWarps; ++y) {
    if (y == warp) ahead = total;
    total += sums[y];
  }
  before[tid] = ahead + inc - rows;
  __syncthreads();
  const bool together = total <= 2 * static_cast<int>(gridDim.x);
  const int first = together ? blockIdx.x : warp * gridDim.x + blockIdx.x;
  const int step = together ? gridDim.x : kJoinWarps * gridDim.x;
  for (int r = first; r < total; r += step) {
    int w = 0;                         // the last worker with before[w] <= r
#pragma unroll
    for (int half = kMaxCtas / 2; half > 0; half >>= 1)
      if (before[w + half] <= r) w += half;
    const SplitHeader& hd = heads[w];
    const int row = r - before[w];
    Sum<D> sum;
    join_parts<D, E4M3, 4>(rec, w, hd.parts, row, together ? warp : 0, together ? kJoinWarps : 1, lane, sum);
    if (together) join_warps<D, E4M3>(warp, lane, sum);
    if (!together || warp == 0)
      join_finish<D, E4M3>(a, hd, hd.rho0 + row, sum, lane, [&](int& p0, int& p1) {
        item_positions(a, hd.q, hd.rho0 / kItemRows, p0, p1);
      });
  }
  if (marks) mend_rows<D, E4M3>(a, heads, workers, warp, lane);
}

template <int D, bool E4M3>
int launch(const AttentionArgs& a, void* ws, cudaStream_t stream) {
  using C = Cfg<D, E4M3>;
  CUtensorMap tk, tv;
  const uint64_t rows = static_cast<uint64_t>(a.c.n_pages) * a.c.kv_heads << a.c.page_shift;
  const uint64_t cols = E4M3 ? D / 2 : D;    // in 16-bit units
  const uint32_t box = 1u << a.c.page_shift;
  auto map = [&](CUtensorMap* m, const void* q) {
    return cols == 32 ? make_tmap_bf16_sw64(m, q, rows, cols, box) : make_tmap_bf16(m, q, rows, cols, box);
  };
  if (!map(&tk, a.c.k) || !map(&tv, a.c.v)) return DS_VIT_ECUDA;
  if (allow_smem(reinterpret_cast<const void*>(prefill_kernel<D, E4M3>), C::kSmem) != cudaSuccess) return DS_VIT_ECUDA;
  const int sms = num_sms(), grid = sms < kMaxCtas ? sms : kMaxCtas;
  const PrefillArgs p{a, records_in(ws, grid, kItemRows, D)};
  cudaError_t e = launch_pdl(prefill_kernel<D, E4M3>, dim3(grid), dim3(C::kThreads), C::kSmem, stream, tk, tv, p);
  if (e == cudaSuccess)
    e = launch_pdl(join_items_kernel<D, E4M3>, dim3(kJoinBlocks * sms), dim3(32 * kJoinWarps), 0, stream, a, p.rec, grid);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? DS_VIT_OK : DS_VIT_ECUDA;
}

}  // namespace

size_t cache_prefill_workspace(int head_dim) { return records_bytes(num_sms(), kItemRows, head_dim); }

int launch_cache_prefill(const AttentionArgs& a, int head_dim, bool e4m3, void* ws, cudaStream_t stream) {
  if (head_dim == 128) return e4m3 ? launch<128, true>(a, ws, stream) : launch<128, false>(a, ws, stream);
  return e4m3 ? launch<64, true>(a, ws, stream) : launch<64, false>(a, ws, stream);
}

}  // namespace dsvit
