// Pages of many sequences: resizing, releasing, forking and compacting on the device, and
// copying pages of a cache (include/dsvit.h).
//
// The four calls that change tables are chains of small steps over the list, the
// counts and the entries: bound by latency, a few round trips to L2 each (64 forks 10 us, 240 of 450 pages 17; ending
// those 20, of which the atomics of one cluster's SMs are half; 240 sequences giving up 446 pages each behind a window 16, 64
// of one page each 2.6; a pool of 3000 pages compacted 11).  One cluster of
// eight CTAs makes a whole call in one launch; the steps are separated by the cluster's
// hardware barrier, and sums over its stripes of the pool go from CTA to CTA
// through distributed shared memory.  Work per list entry is unequal (one sequence
// of a thousand pages, sixty of ten), so table entries are dealt to the warps in chunks of
// kChunk columns.  Fresh pages are taken in order: a CTA that knows how many free pages
// lie before its stripe gives the j-th free page to the sequence whose part of the
// running sum j falls in, with no list in between.  Counts change by integer atomics, whose order
// leaves no trace.  (Clusters of sixteen: 240 forks 46 -> 38 us with ending and copies, small calls 1 to 2 us
// slower, and a device may have no room for them.)
//
// cache_copy_kernel is bound by memory.
#include <algorithm>

#include "cache.cuh"

namespace dsvit {

namespace {

constexpr int kCtas = 8, kThreads = 1024, kWarps = kThreads / 32;
constexpr int kChunk = 128;      // table columns a warp takes at a time

struct PageArgs {
  int32_t* refs;
  int64_t n_pages;
  int page_shift;
  int32_t* table;
  int32_t* kv_len;
  int slots, cols;
  const int32_t *a, *b, *c;      // the list: up to three arrays of n
  int n;
  int32_t *from, *to, *count;
  int cap;
  int* status;
};

struct Shared {
  uint32_t seen[DS_VIT_MAX_SLOTS / 32], twice[DS_VIT_MAX_SLOTS / 32];   // bits of slots
  int a[DS_VIT_MAX_SEQS], b[DS_VIT_MAX_SEQS];      // the list's slots (and lengths)
  int len[DS_VIT_MAX_SEQS];                        // tokens of a[i] before the call; -1: the entry is left out
  int chunk[DS_VIT_MAX_SEQS + 1];                  // chunks of table entries before each
  int fresh[DS_VIT_MAX_SEQS + 1];                  // fresh pages taken before each
  int copies[DS_VIT_MAX_SEQS + 1];                 // of them, copies
  int64_t sums[2][kWarps];                         // of warps: one scan's, and the next one's
  int counts[3][kWarps];                           // of warps, in the first, second and third count
  int all[3][kCtas];                               // what the CTAs tell one another
};
static_assert(sizeof(Shared) <= 48 * 1024, "static shared memory");

__device__ __forceinline__ int64_t ceil_page(const PageArgs& a, int64_t tokens) {
  return (tokens + (int64_t{1} << a.page_shift) - 1) >> a.page_shift;
}
__device__ __forceinline__ bool length_there(const PageArgs& a, int len) {
  return len >= 0 && len <= static_cast<int64_t>(a.cols) << a.page_shift;
}
__device__ __forceinline__ bool slot_there(const PageArgs& a, int s) { return s >= 0 && s < a.slots; }

// Sum of v over the threads before this one, and over all; by all threads of the CTA, which
// take turns 0, 1, 0, ... from scan to scan (the other turn's sums may still be read).
template <typename T>
__device__ __forceinline__ T scan(Shared& sh, int turn, T v, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh.sums[turn][warp] = x;
  __syncthreads();
  T w = static_cast<T>(sh.sums[turn][lane]);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xFFFFFFFFu, w, 31);
  const T before = __shfl_sync(0xFFFFFFFFu, w, warp > 0 ? warp - 1 : 0);
  return x - v + (warp > 0 ? before : 0);
}

// Value v of this CTA (the same in its threads) to all CTAs' all[which]; they have it behind the
// cluster's next barrier, which also orders what the CTAs wrote to memory.
__device__ __forceinline__ void tell(Shared& sh, int which, int v) {
  if (threadIdx.x < kCtas) {
    const uint32_t to = mapa_shared(smem_u32(&sh.all[which][cluster_rank()]), threadIdx.x);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(v) : "memory");
  }
}
__device__ __forceinline__ int64_t told_before(const Shared& sh, int which) {
  int64_t x = 0;
  for (uint32_t r = 0; r < cluster_rank(); ++r) x += sh.all[which][r];
  return x;
}
__device__ __forceinline__ int64_t told(const Shared& sh, int which) {
  int64_t x = 0;
  for (int r = 0; r < kCtas; ++r) x += sh.all[which][r];
  return x;
}

// This CTA's stripe of the pool, a multiple of four pages but for the last one's end.
struct Stripe {
  int64_t begin, end;
};
__device__ __forceinline__ Stripe stripe(const PageArgs& a) {
  const int64_t each = ((a.n_pages + 4 * kCtas - 1) / (4 * kCtas)) * 4;
  const int64_t begin = cluster_rank() * each;
  return Stripe{min(begin, a.n_pages), min(begin + each, a.n_pages)};
}
// The counts of pages p .. p + 3 of a stripe that ends at `end`, past L1 (other CTAs change them); kBehind
// behind the end.  p is a multiple of four.
constexpr int kBehind = INT32_MIN;
__device__ __forceinline__ int4 counts_at(const PageArgs& a, int64_t p, int64_t end) {
  if (p + 4 <= end) return __ldcg(reinterpret_cast<const int4*>(a.refs + p));
  int4 v = make_int4(kBehind, kBehind, kBehind, kBehind);
  if (p < end) v.x = __ldcg(a.refs + p);
  if (p + 1 < end) v.y = __ldcg(a.refs + p + 1);
  if (p + 2 < end) v.z = __ldcg(a.refs + p + 2);
  return v;
}
// Those of this thread in the first round over its stripe.
__device__ __forceinline__ int4 first_counts(const PageArgs& a) {
  const Stripe st = stripe(a);
  return counts_at(a, st.begin + 4 * threadIdx.x, st.end);
}

// How many pages of the stripe satisfy f(page, count); `first` as of first_counts.
template <typename F>
__device__ __forceinline__ int count_pages(Shared& sh, const PageArgs& a, int which, int4& first, F&& f) {
  const Stripe st = stripe(a);
  int n = 0;
  int4 v = first;
  for (int64_t p = st.begin + 4 * threadIdx.x; p < st.end;) {
    n += f(p, v.x) + f(p + 1, v.y) + f(p + 2, v.z) + f(p + 3, v.w);
    if (p < st.begin + 4 * kThreads) first = v;
    p += 4 * kThreads;
    if (p < st.end) v = counts_at(a, p, st.end);
  }
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  if ((threadIdx.x & 31) == 0) sh.counts[which][threadIdx.x >> 5] = n;
  __syncthreads();
  return __reduce_add_sync(0xFFFFFFFFu, sh.counts[which][threadIdx.x & 31]);
}

// Calls g(j, page) for the pages of the stripe that satisfy f, j = `before` + their number in
// order, as long as j < limit.  Takes turns of scan from `turn` on.
template <typename F, typename G>
__device__ __forceinline__ void number_pages(Shared& sh, const PageArgs& a, int turn, int4 first, int64_t before,
                                             int64_t limit, F&& f, G&& g) {
  const Stripe st = stripe(a);
  int4 v = first;
  for (int64_t p0 = st.begin; p0 < st.end && before < limit; p0 += 4 * kThreads) {
    const int64_t p = p0 + 4 * threadIdx.x;
    if (p0 != st.begin) v = counts_at(a, p, st.end);
    const bool on[4] = {f(p, v.x), f(p + 1, v.y), f(p + 2, v.z), f(p + 3, v.w)};
    int total;
    int64_t j = before + scan<int>(sh, turn, on[0] + on[1] + on[2] + on[3], &total);
    turn ^= 1;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      if (on[y]) {
        if (j < limit) g(j, static_cast<int32_t>(p + y));
        ++j;
      }
    }
    before += total;
  }
}

// The last i < n with from[i] <= x (from[0] = 0 <= x < from[n]).
__device__ __forceinline__ int part_of(const int* from, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (from[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Fills part[i] (i <= n) with the sum of the v of the entries before i, at most 2^31 - 1; thread i has
// entry i's.  A barrier has to follow.
__device__ __forceinline__ void fill_parts(int* part, int n, int64_t before, int64_t total) {
  if (threadIdx.x < n) part[threadIdx.x] = static_cast<int>(min(before, int64_t{INT32_MAX}));
  if (threadIdx.x == 0) part[n] = static_cast<int>(min(total, int64_t{INT32_MAX}));
}

// Calls f(i, column) for columns begin(i) .. end(i) - 1 of every entry, warps of the whole cluster a chunk
// at a time; sh.chunk has the chunks of each.  f may use its own lane alone.
template <typename B, typename E, typename F>
__device__ __forceinline__ void each_column(const Shared& sh, const PageArgs& a, B&& begin, E&& end, F&& f) {
  const int lane = threadIdx.x & 31;
  for (int x = (threadIdx.x >> 5) * kCtas + cluster_rank(); x < sh.chunk[a.n]; x += kCtas * kWarps) {
    const int i = part_of(sh.chunk, a.n, x);
    const int64_t c0 = begin(i) + static_cast<int64_t>(x - sh.chunk[i]) * kChunk, c1 = min(end(i), c0 + kChunk);
#pragma unroll
    for (int y = 0; y < kChunk / 32; ++y) {
      const int64_t c = c0 + lane + 32 * y;
      if (c < c1) f(i, c);
    }
  }
}

// Takes a page out of one table entry (where nothing else tells that the table and the counts do not agree).
__device__ __forceinline__ void give_back(const PageArgs& a, int32_t page) {
  if (page < 0) return;
  if (page >= a.n_pages) {
    report_error(a.status, DS_VIT_ERANGE);
  } else if (atomicSub(a.refs + page, 1) <= 0) {      // the table and the counts do not agree
    atomicAdd(a.refs + page, 1);
    report_error(a.status, DS_VIT_EINVAL);
  }
}

__device__ __forceinline__ void clear_bits(Shared& sh, const PageArgs& a) {
  for (int w = threadIdx.x; w < (a.slots + 31) / 32; w += kThreads) sh.seen[w] = sh.twice[w] = 0;
  __syncthreads();
}
__device__ __forceinline__ void note_slot(Shared& sh, int s) {
  const uint32_t bit = 1u << (s & 31);
  if (atomicOr(&sh.seen[s >> 5], bit) & bit) atomicOr(&sh.twice[s >> 5], bit);
}
__device__ __forceinline__ bool has_bit(const uint32_t* bits, int s) { return bits[s >> 5] >> (s & 31) & 1; }

// The slots of a list that names none twice, by thread i: whether entry i may be served.
__device__ __forceinline__ bool one_of_its_own(Shared& sh, const PageArgs& a, int slot) {
  const bool mine = threadIdx.x < a.n, there = mine && slot_there(a, slot);
  if (there) note_slot(sh, slot);
  __syncthreads();
  if (mine && !there) report_error(a.status, DS_VIT_ERANGE);
  if (!there) return false;
  if (has_bit(sh.twice, slot)) {
    report_error(a.status, DS_VIT_EINVAL);
    return false;
  }
  return true;
}

__device__ __forceinline__ int32_t& entry(const PageArgs& a, int slot, int64_t col) {
  return a.table[static_cast<int64_t>(slot) * a.cols + col];
}

__device__ __forceinline__ bool is_free(int64_t, int count) { return count == 0; }

__global__ void __launch_bounds__(kThreads) pages_resize_kernel(const __grid_constant__ PageArgs a) {
  __shared__ Shared sh;
  grid_dep_launch();
  clear_bits(sh, a);
  grid_dep_wait();
  const int i = threadIdx.x;
  const int slot = i < a.n ? __ldg(a.a + i) : -1, to = i < a.n ? __ldg(a.b + i) : 0;
  bool on = one_of_its_own(sh, a, slot);
  int len = -1;
  if (on) {
    len = __ldcg(a.kv_len + slot);
    if (!length_there(a, len) || !length_there(a, to)) {
      report_error(a.status, DS_VIT_ERANGE);
      on = false;
    }
  }
  if (i < a.n) {
    sh.a[i] = slot;
    sh.b[i] = to;
    sh.len[i] = on ? len : -1;
  }
  const int64_t had = on ? ceil_page(a, len) : 0, gets = on ? ceil_page(a, to) : 0;
  int chunks;
  const int chunks_before = scan<int>(sh, 0, on && gets < had ? static_cast<int>((had - gets + kChunk - 1) / kChunk) : 0, &chunks);
  fill_parts(sh.chunk, a.n, chunks_before, chunks);
  __syncthreads();
  each_column(
      sh, a, [&](int x) { return ceil_page(a, sh.b[x]); }, [&](int x) { return ceil_page(a, sh.len[x]); },
      [&](int x, int64_t c) {
        int32_t& e = entry(a, sh.a[x], c);
        if (page_there(e, a.n_pages))
          atomicSub(a.refs + e, 1);     // below 0 is found when they are counted
        else if (e >= 0)
          report_error(a.status, DS_VIT_ERANGE);
        e = -1;
      });
  cluster_sync();                       // the counts without what was given back; and all CTAs have begun
  int4 v = first_counts(a);
  // What grows: fresh pages, and a copy of the last one where another sequence names it too.
  bool copy = false;
  int32_t last = -1;
  if (on && to > len && (len & ((1 << a.page_shift) - 1)) != 0) {
    last = __ldcg(&entry(a, slot, had - 1));
    if (!page_there(last, a.n_pages)) {
      report_error(a.status, DS_VIT_ERANGE);
      on = false;
      sh.len[i] = -1;
    } else {
      copy = __ldcg(a.refs + last) > 1;
    }
  }
  const bool grows = on && to > len;
  // Both sums in one: at most 1024 copies, 11 bits.
  int64_t both;
  const int64_t before = scan<int64_t>(sh, 1, (grows ? gets - had + copy : 0) << 11 | copy, &both);
  const int64_t want = both >> 11, n_copies = both & 2047;
  fill_parts(sh.fresh, a.n, before >> 11, want);
  fill_parts(sh.copies, a.n, before & 2047, n_copies);
  tell(sh, 0, count_pages(sh, a, 0, v, [&](int64_t p, int& count) {
         if (count < 0 && count != kBehind) {      // the tables and the counts did not agree
           report_error(a.status, DS_VIT_EINVAL);
           a.refs[p] = count = 0;
         }
         return count == 0;
       }));
  cluster_sync();
  const bool served = want <= told(sh, 0) && n_copies <= a.cap;
  if (served) {
    // (Counts below 0 of a further round have been put right in memory.)
    number_pages(
        sh, a, 0, v, told_before(sh, 0), want, is_free,
        [&](int64_t j, int32_t page) {
          const int x = part_of(sh.fresh, a.n, static_cast<int>(j));
          const int64_t col = ceil_page(a, sh.len[x]);
          const int y = static_cast<int>(j) - sh.fresh[x], copied = sh.copies[x + 1] - sh.copies[x];
          if (copied && y == 0) {
            int32_t& e = entry(a, sh.a[x], col - 1);
            a.from[sh.copies[x]] = e;
            a.to[sh.copies[x]] = page;
            e = page;
          } else {
            entry(a, sh.a[x], col + y - copied) = page;
          }
          a.refs[page] = 1;
        });
  } else if (i == 0 && cluster_rank() == 0) {
    report_error(a.status, DS_VIT_ECAP);
  }
  cluster_sync();                       // every stripe has been numbered: counts may fall again
  if (cluster_rank() != 0) return;
  if (copy && served) atomicSub(a.refs + last, 1);
  if (on && (to < len || (grows && served))) a.kv_len[slot] = to;
  if (i == 0) *a.count = served ? static_cast<int>(n_copies) : 0;
}

__global__ void __launch_bounds__(kThreads) pages_release_kernel(const __grid_constant__ PageArgs a) {
  __shared__ Shared sh;
  grid_dep_launch();
  grid_dep_wait();
  const int i = threadIdx.x;
  int64_t first = 0, last = 0;
  if (i < a.n) {
    const int slot = __ldg(a.a + i), begin = __ldg(a.b + i), end = __ldg(a.c + i);
    const int len = slot_there(a, slot) ? a.kv_len[slot] : -1;
    if (!length_there(a, len) || begin < 0) {
      report_error(a.status, DS_VIT_ERANGE);
    } else if (end < begin) {
      report_error(a.status, DS_VIT_EINVAL);
    } else {
      first = ceil_page(a, begin);
      last = max(first, static_cast<int64_t>(min(end, len)) >> a.page_shift);
    }
    sh.a[i] = slot;
    sh.b[i] = static_cast<int>(first);
    sh.len[i] = static_cast<int>(last);
  }
  int chunks;
  const int before = scan<int>(sh, 0, static_cast<int>((last - first + kChunk - 1) / kChunk), &chunks);
  fill_parts(sh.chunk, a.n, before, chunks);
  __syncthreads();
  // A slot may be in the list more than once: whoever takes the page out of the entry gives it back.
  each_column(
      sh, a, [&](int x) { return static_cast<int64_t>(sh.b[x]); }, [&](int x) { return static_cast<int64_t>(sh.len[x]); },
      [&](int x, int64_t c) { give_back(a, atomicExch(&entry(a, sh.a[x], c), -1)); });
}

__global__ void __launch_bounds__(kThreads) pages_fork_kernel(const __grid_constant__ PageArgs a) {
  __shared__ Shared sh;
  grid_dep_launch();
  clear_bits(sh, a);
  cluster_arrive();
  grid_dep_wait();
  int4 v = first_counts(a);
  const int i = threadIdx.x;
  const int src = i < a.n ? __ldg(a.a + i) : -1, dst = i < a.n ? __ldg(a.b + i) : -1;
  bool on = one_of_its_own(sh, a, dst);
  int len = 0;
  int32_t last = -1;
  if (on) {
    if (!slot_there(a, src)) {
      report_error(a.status, DS_VIT_ERANGE);
      on = false;
    } else if (has_bit(sh.seen, src) || a.kv_len[dst] != 0) {
      report_error(a.status, DS_VIT_EINVAL);
      on = false;
    } else if (len = a.kv_len[src]; !length_there(a, len)) {
      report_error(a.status, DS_VIT_ERANGE);
      on = false;
    } else if ((len & ((1 << a.page_shift) - 1)) != 0) {
      last = entry(a, src, len >> a.page_shift);
      if (last >= a.n_pages) report_error(a.status, DS_VIT_ERANGE);
    }
  }
  const bool copy = on && page_there(last, a.n_pages);
  if (i < a.n) {
    sh.a[i] = src;
    sh.b[i] = dst;
    sh.len[i] = on ? len : -1;
  }
  const int64_t full = on ? len >> a.page_shift : 0;
  int64_t both;
  const int64_t before = scan<int64_t>(sh, 0, (full + kChunk - 1) / kChunk << 32 | copy, &both);
  const int want = static_cast<int>(both);
  fill_parts(sh.chunk, a.n, before >> 32, both >> 32);
  fill_parts(sh.fresh, a.n, static_cast<int>(before), want);
  const int free_pages = count_pages(sh, a, 0, v, is_free);
  cluster_wait();                       // all CTAs have begun: their shared memory is there
  tell(sh, 0, free_pages);
  cluster_sync();
  if (want > told(sh, 0) || want > a.cap) {
    if (i == 0 && cluster_rank() == 0) {
      report_error(a.status, DS_VIT_ECAP);
      *a.count = 0;
    }
    return;
  }
  number_pages(
      sh, a, 1, v, told_before(sh, 0), want, is_free,
      [&](int64_t j, int32_t page) {
        const int x = part_of(sh.fresh, a.n, static_cast<int>(j));
        const int64_t col = sh.len[x] >> a.page_shift;
        a.from[j] = entry(a, sh.a[x], col);
        a.to[j] = page;
        entry(a, sh.b[x], col) = page;
        a.refs[page] = 1;
      });
  // Counts rise from 1 at least, so the numbering of free pages elsewhere does not see it.
  each_column(
      sh, a, [](int) { return int64_t{0}; }, [&](int x) { return static_cast<int64_t>(sh.len[x] >> a.page_shift); },
      [&](int x, int64_t c) {
        const int32_t page = entry(a, sh.a[x], c);
        const bool there = page_there(page, a.n_pages);
        if (there) atomicAdd(a.refs + page, 1);
        if (page >= a.n_pages) report_error(a.status, DS_VIT_ERANGE);
        entry(a, sh.b[x], c) = there ? page : -1;
      });
  if (cluster_rank() != 0) return;
  if (on) {
    if ((len & ((1 << a.page_shift) - 1)) != 0 && !copy) entry(a, dst, full) = -1;
    a.kv_len[dst] = len;
  }
  if (i == 0) *a.count = want;
}

__global__ void __launch_bounds__(kThreads) pages_compact_kernel(const __grid_constant__ PageArgs a) {
  __shared__ Shared sh;
  grid_dep_launch();
  grid_dep_wait();
  cluster_sync();
  const int64_t lane = threadIdx.x + static_cast<int64_t>(cluster_rank()) * kThreads, lanes = kCtas * kThreads;
  int4 v = first_counts(a);
  bool below = false;                   // a count under 0: the table entries that name its page could not be told from moved ones
  const int here = count_pages(sh, a, 0, v, [&](int64_t p, int count) {
    below |= count < 0 && p < a.n_pages;
    return count > 0;
  });
  below = __syncthreads_or(below);
  tell(sh, 0, below ? -1 - here : here);
  cluster_sync();
  for (int r = 0; r < kCtas; ++r) below |= sh.all[0][r] < 0;
  if (below) {
    if (lane == 0) {
      report_error(a.status, DS_VIT_EINVAL);
      *a.count = 0;
    }
    return;
  }
  const int64_t used = told(sh, 0);
  const auto hole = [&](int64_t p, int count) { return count == 0 && p < used; };
  const auto mover = [&](int64_t p, int count) { return count > 0 && p >= used; };
  tell(sh, 1, count_pages(sh, a, 1, v, hole));
  tell(sh, 2, count_pages(sh, a, 2, v, mover));
  cluster_sync();
  // As many holes as movers.
  const int64_t moved = min(min(told(sh, 1), told(sh, 2)), static_cast<int64_t>(a.cap));
  number_pages(sh, a, 0, v, told_before(sh, 1), moved, hole, [&](int64_t j, int32_t page) { a.to[j] = page; });
  __syncthreads();                      // the last scan's sums have been read
  number_pages(sh, a, 0, v, told_before(sh, 2), moved, mover, [&](int64_t j, int32_t page) { a.from[j] = page; });
  cluster_sync();
  // The counts move along; in the place of the old one stands where the page went.
  for (int64_t j = lane; j < moved; j += lanes) {
    const int32_t from = __ldcg(a.from + j), to = __ldcg(a.to + j);
    a.refs[to] = __ldcg(a.refs + from);
    a.refs[from] = -1 - to;
  }
  cluster_sync();
  if (moved > 0) {
    for (int s = (threadIdx.x >> 5) * kCtas + cluster_rank(); s < a.slots; s += kCtas * kWarps) {
      const int len = a.kv_len[s];
      if (!length_there(a, len)) {
        report_error(a.status, DS_VIT_ERANGE);
        continue;
      }
      const int64_t cols = ceil_page(a, len);
      for (int64_t c = threadIdx.x & 31; c < cols; c += 32) {
        const int32_t page = entry(a, s, c);
        if (page < used) continue;
        if (page >= a.n_pages) {
          report_error(a.status, DS_VIT_ERANGE);
          continue;
        }
        const int went = __ldcg(a.refs + page);
        if (went < 0) entry(a, s, c) = -1 - went;
      }
    }
  }
  cluster_sync();
  for (int64_t j = lane; j < moved; j += lanes) a.refs[__ldcg(a.from + j)] = 0;
  if (lane == 0) *a.count = static_cast<int>(moved);
}

// ------------------------------------------------------------------ contents

struct CopyArgs {
  uint4* held[2];          // keys, values, in 16-byte words
  int64_t held_words;      // of either, a page's
  uint4* small[3];         // their exponents, bounds (nullptr: none)
  int small_words[3];
  uint8_t* bound_exp;
  int heads;
  int64_t n_pages;
  const int32_t *from, *to, *count;
  int cap;
  int held_tiles;          // CTAs in x: these for the keys, as many for the values, one for the rest
  int* status;
};

constexpr int kCopyThreads = 256, kCopyWords = 4;    // words a thread has in flight

// CTA (x, y) copies its part x of pages y, y + gridDim.y, ...: what it has to look up is one pair of
// page numbers.  690 pages of 2 x 131 KB: 53 us, the rate of a plain copy; 65 with eight CTAs an SM, whose 32 registers
// do not hold the words in flight, 75 with the parts of all pages dealt out in one row, which takes a division and
// a search for the part.
__global__ void __launch_bounds__(kCopyThreads, 5) cache_copy_kernel(const __grid_constant__ CopyArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const int n = __ldg(a.count);
  if (n < 0 || n > a.cap) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) report_error(a.status, DS_VIT_EINVAL);
    return;
  }
  const int x = static_cast<int>(blockIdx.x);
  const int64_t first = static_cast<int64_t>(x % a.held_tiles) * (kCopyThreads * kCopyWords) + threadIdx.x;
  uint4* const base = a.held[x >= a.held_tiles && x < 2 * a.held_tiles];
  for (int i = static_cast<int>(blockIdx.y); i < n; i += static_cast<int>(gridDim.y)) {
    const int from = __ldg(a.from + i), to = __ldg(a.to + i);
    if (!page_there(from, a.n_pages) || !page_there(to, a.n_pages)) {
      if (threadIdx.x == 0) report_error(a.status, DS_VIT_ERANGE);
      continue;
    }
    if (x < 2 * a.held_tiles) {
      const uint4* const get = base + from * a.held_words + first;
      uint4* const put = base + to * a.held_words + first;
      uint4 v[kCopyWords];
#pragma unroll
      for (int y = 0; y < kCopyWords; ++y)
        if (first + y * kCopyThreads < a.held_words) v[y] = __ldcs(get + y * kCopyThreads);
#pragma unroll
      for (int y = 0; y < kCopyWords; ++y)
        if (first + y * kCopyThreads < a.held_words) __stcs(put + y * kCopyThreads, v[y]);
      continue;
    }
#pragma unroll
    for (int y = 0; y < 3; ++y)
      for (int w = threadIdx.x; w < a.small_words[y]; w += kCopyThreads)
        a.small[y][to * static_cast<int64_t>(a.small_words[y]) + w] = a.small[y][from * static_cast<int64_t>(a.small_words[y]) + w];
    if (a.bound_exp != nullptr)
      for (int h = threadIdx.x; h < a.heads; h += kCopyThreads)
        a.bound_exp[static_cast<int64_t>(to) * a.heads + h] = a.bound_exp[static_cast<int64_t>(from) * a.heads + h];
  }
}

int page_shift_of(int page) {
  for (int s = 4; s < 8; ++s)
    if (page == 1 << s) return s;
  return -1;
}

bool bad_ints(const void* p) { return !p || !aligned(p, 4); }

bool bad_copies(const ds_vit_page_copies* c) {
  return !c || bad_ints(c->from) || bad_ints(c->to) || bad_ints(c->count) || c->cap < 1;
}

int check_pages(const ds_vit_page_pool* pool, const ds_vit_page_tables* t, int32_t* status, PageArgs* a) {
  if (!pool || !t || !pool->refs || !aligned(pool->refs, 16) || pool->n_pages < 1 || bad_ints(t->table) ||
      bad_ints(t->kv_len) || bad_ints(status) || t->slots < 1 || t->slots > DS_VIT_MAX_SLOTS || t->table_cols < 1 ||
      page_shift_of(pool->page) < 0)
    return DS_VIT_EINVAL;
  if (pool->n_pages > INT32_MAX - 65535 || t->table_cols > (INT32_MAX - 255) / pool->page) return DS_VIT_ERANGE;
  a->refs = pool->refs;
  a->n_pages = pool->n_pages;
  a->page_shift = page_shift_of(pool->page);
  a->table = t->table;
  a->kv_len = t->kv_len;
  a->slots = t->slots;
  a->cols = t->table_cols;
  a->status = reinterpret_cast<int*>(status);
  return DS_VIT_OK;
}

bool bad_list(PageArgs* a, const int32_t* x, const int32_t* y, const int32_t* z, int n) {
  a->a = x;
  a->b = y;
  a->c = z;
  a->n = n;
  return bad_ints(x) || bad_ints(y) || bad_ints(z) || n < 1 || n > DS_VIT_MAX_SEQS;
}

void take_copies(PageArgs* a, const ds_vit_page_copies* c) {
  a->from = c->from;
  a->to = c->to;
  a->count = c->count;
  a->cap = c->cap;
}

int launch_pages(void (*kernel)(PageArgs), const PageArgs& a, void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return launched(cudaLaunchKernelEx(&cfg, kernel, a));
}

}  // namespace

}  // namespace dsvit

using namespace dsvit;

extern "C" {

int ds_vit_pages_resize(const ds_vit_page_pool* pool, const ds_vit_page_tables* tables, const int32_t* slot,
                        const int32_t* length, int32_t n, const ds_vit_page_copies* copies, int32_t* status,
                        void* stream) {
  PageArgs a{};
  if (const int rc = check_pages(pool, tables, status, &a)) return rc;
  if (bad_list(&a, slot, length, slot, n) || bad_copies(copies)) return DS_VIT_EINVAL;
  take_copies(&a, copies);
  return launch_pages(pages_resize_kernel, a, stream);
}

int ds_vit_pages_release(const ds_vit_page_pool* pool, const ds_vit_page_tables* tables, const int32_t* slot,
                         const int32_t* begin, const int32_t* end, int32_t n, int32_t* status, void* stream) {
  PageArgs a{};
  if (const int rc = check_pages(pool, tables, status, &a)) return rc;
  if (bad_list(&a, slot, begin, end, n)) return DS_VIT_EINVAL;
  return launch_pages(pages_release_kernel, a, stream);
}

int ds_vit_pages_fork(const ds_vit_page_pool* pool, const ds_vit_page_tables* tables, const int32_t* src,
                      const int32_t* dst, int32_t n, const ds_vit_page_copies* copies, int32_t* status,
                      void* stream) {
  PageArgs a{};
  if (const int rc = check_pages(pool, tables, status, &a)) return rc;
  if (bad_list(&a, src, dst, src, n) || bad_copies(copies)) return DS_VIT_EINVAL;
  take_copies(&a, copies);
  return launch_pages(pages_fork_kernel, a, stream);
}

int ds_vit_pages_compact(const ds_vit_page_pool* pool, const ds_vit_page_tables* tables,
                         const ds_vit_page_copies* copies, int32_t* status, void* stream) {
  PageArgs a{};
  if (const int rc = check_pages(pool, tables, status, &a)) return rc;
  if (bad_copies(copies)) return DS_VIT_EINVAL;
  take_copies(&a, copies);
  return launch_pages(pages_compact_kernel, a, stream);
}

int ds_vit_cache_copy(const ds_vit_cache* cache, const ds_vit_key_bounds* bounds, const ds_vit_page_copies* copies,
                      int32_t* status, void* stream) {
  CacheView c;
  if (const int rc = check_pages_of(cache, &c)) return rc;
  if (bad_copies(copies) || bad_ints(status) ||
      (bounds && (!bounds->hi_lo || !aligned(bounds->hi_lo, 16) || !bounds->exp)))
    return DS_VIT_EINVAL;
  const bool e4m3 = cache->kind == DS_VIT_CACHE_E4M3;
  const int64_t rows = static_cast<int64_t>(c.kv_heads) * cache->page;      // of a page
  CopyArgs a{};
  a.held[0] = reinterpret_cast<uint4*>(c.k), a.held[1] = reinterpret_cast<uint4*>(c.v);
  a.held_words = rows * cache->head_dim * (e4m3 ? 1 : 2) / 16;
  if (e4m3) {
    a.small[0] = reinterpret_cast<uint4*>(c.k_exp), a.small[1] = reinterpret_cast<uint4*>(c.v_exp);
    a.small_words[0] = a.small_words[1] = static_cast<int>(rows / 16);
  }
  if (bounds) {
    a.small[2] = reinterpret_cast<uint4*>(bounds->hi_lo);
    a.small_words[2] = 2 * c.kv_heads * cache->head_dim / 16;
    a.bound_exp = bounds->exp;
  }
  a.heads = c.kv_heads;
  a.n_pages = c.n_pages;
  a.from = copies->from;
  a.to = copies->to;
  a.count = copies->count;
  a.cap = copies->cap;
  a.held_tiles = static_cast<int>((a.held_words + kCopyThreads * kCopyWords - 1) / (kCopyThreads * kCopyWords));
  a.status = reinterpret_cast<int*>(status);
  const int parts = 2 * a.held_tiles + (e4m3 || bounds);
  const dim3 grid(static_cast<unsigned>(parts), static_cast<unsigned>(std::min(copies->cap, (10 * num_sms() + parts - 1) / parts)));
  return launched(launch_pdl(cache_copy_kernel, grid, dim3(kCopyThreads), 0, static_cast<cudaStream_t>(stream), a));
}

}  // extern "C"
