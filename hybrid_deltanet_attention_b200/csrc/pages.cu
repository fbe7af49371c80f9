// Pages of a paged KV cache: resizing and freeing sequences, forking, compacting, copying.
//
// Every call but the plain copy is two steps. A planning kernel of one CTA reads lengths, table and use
// counts, decides, and writes them back together with a list of page copies; it is a few
// microseconds of dependent loads, block scans and shared counters, bound by latency, and one
// CTA needs no grid-wide barrier between its phases. A copy kernel then moves the listed pages
// with 16-byte loads and stores over the whole GPU, bound by HBM.
//
// Measured: a plan for 61 sequences in 16384 pages about 7 us (dependent loads 4000 clocks, counts into shared memory
// 1000, releases 2000, free list 4000, table 3000), for a fork of eight 1001-position sequences 6; the copies of
// a 357 MB compaction 58 us, 6.2 TB/s.
//
// All decisions are order-free: releases and counts are integer atomics, pages are taken by
// rank (lowest free id first, in the order of the call's sequences), so results never depend
// on scheduling.
#include <algorithm>
#include <string>

#include "dev.cuh"
#include "mk_internal.h"
#include "mk_model.h"
#include "paged.h"

namespace mk {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// Scratch of a cache (int32 entries, mk_pages_work_ints of them):
//   [0] number of page copies, [1] pages in use (compact), [2], [3] unused
//   src, dst, rows [n_pages] each: the copies (rows = slots of the page to copy)
//   list [n_pages]: free pages by rank (resize, fork); new id of a moved page (compact)
//   mark, need [n_seqs] each
struct Work {
  int *count, *src, *dst, *rows, *list, *mark, *need;
};
__host__ __device__ inline Work work_of(const mk_paged_cache& c) {
  int* p = c.work + 4;
  const long long np = c.n_pages, ns = c.n_seqs;
  return Work{c.work, p, p + np, p + 2 * np, p + 3 * np, p + 4 * np, p + 4 * np + ns};
}

__device__ __forceinline__ int pages_of(int n, int ps) { return (n + ps - 1) / ps; }

// Exclusive scan of one value per thread over the block; total in every thread.
template <typename T>
__device__ T block_scan(T v, T* total, T* red) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // the previous scan's totals have been read
  if (lane == 31) red[w] = x;
  __syncthreads();
  const T t = red[lane];   // kPlanWarps == 32
  T s = t;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += y;
  }
  const T base = __shfl_sync(0xFFFFFFFFu, s - t, w);
  *total = __shfl_sync(0xFFFFFFFFu, s, 31);
  return base + x - v;
}

// The use counts and the list of free pages while a plan works on them: copies in shared memory for up
// to kRefCached / kListCached pages (scattered counts, and entries that are read right after they were
// written, each cost an L2 round trip otherwise), the arrays themselves beyond that. Changes go to the copy and,
// without waiting, to the array, so nothing is written back at the end.
constexpr int kRefCached = 48 * 1024, kListCached = 24 * 1024;
struct Counts {
  int* p;          // to read from
  int* all;        // the cache's counts
  int n;
  bool cached;
  __device__ int at(long long i) const { return cached ? p[i] : __ldcg(p + i); }
  __device__ void add(int i, int by) const {
    if (cached) atomicAdd(p + i, by);
    atomicAdd(all + i, by);
  }
  __device__ void take(int i) const {   // a free page
    if (cached) p[i] = 1;
    all[i] = 1;
  }
};
// Asynchronous: cp_async_wait and a barrier before the first use.
__device__ Counts open_counts(const mk_paged_cache& c, int* cache) {
  if (c.n_pages > kRefCached) return Counts{c.ref, c.ref, c.n_pages, false};
  const bool wide = (reinterpret_cast<uintptr_t>(c.ref) & 15) == 0;
  const int quads = wide ? c.n_pages / 4 : 0;
  for (int i = threadIdx.x; i < quads; i += kPlanThreads) cp_async16(cache + 4 * i, c.ref + 4 * i, 16);
  for (int i = 4 * quads + threadIdx.x; i < c.n_pages; i += kPlanThreads) cp_async4(cache + i, c.ref + i, 4);
  cp_async_commit();
  return Counts{cache, c.ref, c.n_pages, true};
}

// Ranks the free pages in ascending order into list until `want` are found; returns how many
// there are (at most about want + one chunk are looked at). A lane looks at four consecutive counts, the block at
// 4096: most calls find their few pages in the first chunk.
template <bool kCachedCounts>
__device__ int list_free(const Counts& ref, int want, int* list, int* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned below = (1u << lane) - 1u;
  const bool wide = kCachedCounts || (reinterpret_cast<uintptr_t>(ref.p) & 15) == 0;
  int found = 0;
  for (long long base = 0; base < ref.n && found < want; base += kPlanThreads * 4) {
    const long long p = base + 4 * threadIdx.x;
    int4 v = make_int4(1, 1, 1, 1);
    if (wide && p + 4 <= ref.n) {
      v = kCachedCounts ? *reinterpret_cast<const int4*>(ref.p + p) : __ldcg(reinterpret_cast<const int4*>(ref.p + p));
    } else {
      if (p < ref.n) v.x = ref.at(p);
      if (p + 1 < ref.n) v.y = ref.at(p + 1);
      if (p + 2 < ref.n) v.z = ref.at(p + 2);
      if (p + 3 < ref.n) v.w = ref.at(p + 3);
    }
    const unsigned mine = (v.x == 0) | (v.y == 0) << 1 | (v.z == 0) << 2 | (v.w == 0) << 3;
    unsigned before = 0, all = 0;                // free pages of the warp's lanes below, and of the warp
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned b = __ballot_sync(0xFFFFFFFFu, mine >> j & 1);
      before += __popc(b & below);
      all += __popc(b);
    }
    __syncthreads();   // the totals of the chunk before have been read
    if (lane == 0) red[warp] = all;
    __syncthreads();
    const int t = red[lane];   // kPlanWarps == 32
    int at = found + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? t : 0) + before;
    found += __reduce_add_sync(0xFFFFFFFFu, t);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (mine >> j & 1) {
        if (at < want) list[at] = static_cast<int>(p) + j;
        ++at;
      }
  }
  __syncthreads();
  return found;
}

// Scan of need[0 .. n) in place (exclusive); returns the sum, which may be far above what an
// offset can be (offsets are only used when the sum is at most n_pages).
template <typename T>
__device__ long long scan_need(int* need, int n, T* red) {
  long long sum = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    T total;
    const long long off = sum + block_scan<T>(i < n ? need[i] : 0, &total, red);
    if (i < n) need[i] = static_cast<int>(min(off, 0x7fffffffll));
    sum += total;
  }
  __syncthreads();
  return sum;
}

__device__ __forceinline__ bool len_ok(const mk_paged_cache& c, int n) { return n >= 0 && n <= c.max_pages * c.page_size; }

// What a plan keeps of each of its sequences: in shared memory for up to kCached of them,
// beyond that it reads the arrays again (and keeps need and own in the scratch).
constexpr int kCached = 1024;
struct Plan {
  int a[kCached], from[kCached], to[kCached], from_pages[kCached], to_pages[kCached], need[kCached], own[kCached];
  int red[32];
  long long red64[32];
};

// f(j, p) for the entries p of table columns first .. last - 1 of a row, by one warp; four loads in flight.
template <typename F>
__device__ __forceinline__ void for_row(const int* row, int first, int last, F&& f) {
  for (int j0 = first + (threadIdx.x & 31); j0 < last; j0 += 128) {
    int p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = j0 + 32 * k < last ? row[j0 + 32 * k] : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (j0 + 32 * k < last) f(j0 + 32 * k, p[k]);
  }
}

// Adds `by` to the counts of the pages in columns first .. last - 1; true where an entry names no page.
__device__ __forceinline__ bool count_row(const mk_paged_cache& c, const Counts& ref, int s, int first, int last, int by) {
  bool bad = false;
  for_row(c.table + static_cast<long long>(s) * c.max_pages, first, last, [&](int, int p) {
    if (p >= 0 && p < c.n_pages)
      ref.add(p, by);
    else
      bad = true;
  });
  return bad;
}

// Each sequence at most once: the last writer's index stands in mark, every other one finds it.
__device__ __forceinline__ bool named_twice(const Work& w, int s, int i) { return __ldcg(&w.mark[s]) != i; }

// mk_pages_resize. Phases, a block barrier between them: check ids and lengths; give back the
// pages past each new end; count what each sequence takes (a shared partly filled page that stays
// is replaced: its count is read after every release and before any replacement); rank the
// free pages; write table, counts and lengths. A bad entry or too few pages take the releases back.
__global__ void __launch_bounds__(kPlanThreads, 1) plan_resize(mk_paged_cache c, const int* seqs, const int* lens, int n) {
  __shared__ Plan sm;
  extern __shared__ __align__(16) int counts[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the copy kernel comes up meanwhile
  const Work w = work_of(c);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ps = c.page_size;
  const bool small = n <= kCached;
  int* need = small ? sm.need : w.need;
  int* own = small ? sm.own : w.mark;
  auto get = [&](int i, int& s, int& op, int& np) {   // pages before and after
    if (small) {
      s = sm.a[i], op = sm.from_pages[i], np = sm.to_pages[i];
    } else {
      s = seqs[i], op = pages_of(c.len[s], ps), np = pages_of(lens ? lens[i] : 0, ps);
    }
  };
  const Counts ref = open_counts(c, counts);
  int* list = c.n_pages <= kListCached ? counts + ((c.n_pages + 3) & ~3) : w.list;
  if (tid == 0) w.count[0] = 0;
  int bad = 0;
  for (int i = tid; i < n; i += kPlanThreads) {
    const int s = seqs[i], now = lens ? lens[i] : 0;
    const bool there = s >= 0 && s < c.n_seqs;
    const int old = there ? c.len[s] : 0;
    bad |= !there || !len_ok(c, old) || !len_ok(c, now);
    if (there) w.mark[s] = i;
    if (small) sm.a[i] = s, sm.from[i] = old, sm.to[i] = now, sm.from_pages[i] = pages_of(old, ps), sm.to_pages[i] = pages_of(now, ps);
  }
  cp_async_wait<0>();
  if (!__syncthreads_or(bad)) {
    for (int i = tid; i < n; i += kPlanThreads) bad |= named_twice(w, small ? sm.a[i] : seqs[i], i);
    bad = __syncthreads_or(bad);
  } else {
    bad = 1;
  }
  if (bad) {
    if (tid == 0) atomicOr(c.err, MK_DEVERR_BAD_PAGE);
    return;
  }
  // a sequence is one warp's
  for (int i = warp; i < n; i += kPlanWarps) {
    int s, op, np;
    get(i, s, op, np);
    bad |= count_row(c, ref, s, np, op, -1);
  }
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const int s = small ? sm.a[i] : seqs[i];
    const int old = small ? sm.from[i] : c.len[s], now = small ? sm.to[i] : lens ? lens[i] : 0;
    const int low = min(old, now);
    int mine = 0;
    if (low % ps) {
      const int p = c.table[static_cast<long long>(s) * c.max_pages + low / ps];
      if (p < 0 || p >= c.n_pages)
        bad = 1;
      else
        mine = ref.at(p) > 1;
    }
    own[i] = mine;
    need[i] = max(0, pages_of(now, ps) - pages_of(low, ps)) + mine;
  }
  bad = __syncthreads_or(bad);
  // 1024 of these fit 32 bits in any table of less than 2^21 columns
  const long long total = bad ? 0 : c.max_pages < (1 << 20) ? scan_need(need, n, sm.red) : scan_need(need, n, sm.red64);
  const int want = static_cast<int>(min(total, static_cast<long long>(c.n_pages) + 1));
  if (bad || (ref.cached ? list_free<true>(ref, want, list, sm.red) : list_free<false>(ref, want, list, sm.red)) < total) {   // nothing changes: take the releases back
    for (int i = warp; i < n; i += kPlanWarps) {
      int s, op, np;
      get(i, s, op, np);
      count_row(c, ref, s, np, op, 1);
    }
    if (tid == 0) atomicOr(c.err, bad ? MK_DEVERR_BAD_PAGE : MK_DEVERR_NO_PAGES);
    return;
  }
  for (int i = warp; i < n; i += kPlanWarps) {
    int s, op, np;
    get(i, s, op, np);
    const int mine = own[i], have = min(op, np);
    int* row = c.table + static_cast<long long>(s) * c.max_pages;
    const int* take = list + need[i];
    if (mine && lane == 0) {
      const int low = min(c.len[s], lens ? lens[i] : 0);
      const int e = low / ps, was = row[e], page = take[0], at = atomicAdd(&w.count[0], 1);
      w.src[at] = was;
      w.dst[at] = page;
      w.rows[at] = low % ps;
      ref.add(was, -1);
      ref.take(page);
      row[e] = page;
    }
    for_row(take + mine - have, have, np, [&](int j, int p) {
      row[j] = p;
      ref.take(p);
    });
    for (int j = np + lane; j < op; j += 32) row[j] = -1;
    __syncwarp();
    if (lane == 0) c.len[s] = lens ? lens[i] : 0;
  }
}

// mk_pages_fork, the same phases: give back what the destinations hold, count the partly
// filled pages, rank free ones, share and write.
__global__ void __launch_bounds__(kPlanThreads, 1) plan_fork(mk_paged_cache c, const int* src, const int* dst, int n) {
  __shared__ Plan sm;
  extern __shared__ __align__(16) int counts[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the copy kernel comes up meanwhile
  const Work w = work_of(c);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ps = c.page_size;
  const bool small = n <= kCached;
  int* need = small ? sm.need : w.need;
  auto get = [&](int i, int& a, int& b, int& len, int& had) {
    if (small) {
      a = sm.a[i], b = sm.own[i], len = sm.from[i], had = sm.to[i];
    } else {
      a = src[i], b = dst[i], len = c.len[a], had = c.len[b];
    }
  };
  const Counts ref = open_counts(c, counts);
  int* list = c.n_pages <= kListCached ? counts + ((c.n_pages + 3) & ~3) : w.list;
  if (tid == 0) w.count[0] = 0;
  int bad = 0;
  for (int i = tid; i < n; i += kPlanThreads) {
    const int a = src[i], b = dst[i];
    const bool there = a >= 0 && a < c.n_seqs && b >= 0 && b < c.n_seqs;
    const int len = there ? c.len[a] : 0, had = there ? c.len[b] : 0;
    bad |= !there || !len_ok(c, len) || !len_ok(c, had);
    if (there) w.mark[b] = i;
    if (small) sm.a[i] = a, sm.own[i] = b, sm.from[i] = len, sm.to[i] = had;
    need[i] = len % ps ? 1 : 0;
  }
  cp_async_wait<0>();
  if (!__syncthreads_or(bad)) {
    for (int i = tid; i < n; i += kPlanThreads) {
      int a, b, len, had;
      get(i, a, b, len, had);
      // a source that is also a destination: its mark (which may be an old one) names a destination that is it
      const int m = __ldcg(&w.mark[a]);
      bad |= named_twice(w, b, i) || (m >= 0 && m < n && dst[m] == a);
    }
    bad = __syncthreads_or(bad);
  } else {
    bad = 1;
  }
  if (bad) {
    if (tid == 0) atomicOr(c.err, MK_DEVERR_BAD_PAGE);
    return;
  }
  for (int i = warp; i < n; i += kPlanWarps) {
    int a, b, len, had;
    get(i, a, b, len, had);
    bad |= count_row(c, ref, b, 0, pages_of(had, ps), -1);
    for_row(c.table + static_cast<long long>(a) * c.max_pages, 0, pages_of(len, ps),
            [&](int, int p) { bad |= p < 0 || p >= c.n_pages; });
  }
  bad = __syncthreads_or(bad);
  const int total = bad ? 0 : static_cast<int>(scan_need(need, n, sm.red));
  if (bad || (ref.cached ? list_free<true>(ref, total, list, sm.red) : list_free<false>(ref, total, list, sm.red)) < total) {
    for (int i = warp; i < n; i += kPlanWarps) {
      int a, b, len, had;
      get(i, a, b, len, had);
      count_row(c, ref, b, 0, pages_of(had, ps), 1);
    }
    if (tid == 0) atomicOr(c.err, bad ? MK_DEVERR_BAD_PAGE : MK_DEVERR_NO_PAGES);
    return;
  }
  for (int i = warp; i < n; i += kPlanWarps) {
    int a, b, len, had;
    get(i, a, b, len, had);
    const int np = pages_of(len, ps);
    int* rb = c.table + static_cast<long long>(b) * c.max_pages;
    for_row(c.table + static_cast<long long>(a) * c.max_pages, 0, np, [&](int j, int p) {
      if (j < len / ps) {
        ref.add(p, 1);
      } else {
        const int page = list[need[i]], at = atomicAdd(&w.count[0], 1);
        w.src[at] = p;
        w.dst[at] = page;
        w.rows[at] = len % ps;
        ref.take(page);
        p = page;
      }
      rb[j] = p;
    });
    for (int j = np + lane; j < pages_of(had, ps); j += 32) rb[j] = -1;
    __syncwarp();
    if (lane == 0) c.len[b] = len;
  }
}

// mk_pages_compact, counts and copies: pages in use, then the r-th used page with an id past
// them paired with the r-th free id below (there are equally many). list[p] is the new id of
// page p >= live, -1 where it has no count; the table follows in the copy kernel. Four counts a thread and step.
__global__ void __launch_bounds__(kPlanThreads, 1) plan_compact(mk_paged_cache c) {
  __shared__ int red[32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Work w = work_of(c);
  const int tid = threadIdx.x;
  const bool wide = (reinterpret_cast<uintptr_t>(c.ref) & 15) == 0;
  auto four = [&](long long p) {               // counts of pages p .. p + 3, 0 past the last one
    if (wide && p + 4 <= c.n_pages) return *reinterpret_cast<const int4*>(c.ref + p);
    int4 v = make_int4(0, 0, 0, 0);
    if (p < c.n_pages) v.x = c.ref[p];
    if (p + 1 < c.n_pages) v.y = c.ref[p + 1];
    if (p + 2 < c.n_pages) v.z = c.ref[p + 2];
    if (p + 3 < c.n_pages) v.w = c.ref[p + 3];
    return v;
  };
  int used = 0;
#pragma unroll 4
  for (long long p = 4ll * tid; p < c.n_pages; p += 4 * kPlanThreads) {
    const int4 v = four(p);
    used += (v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0);
  }
  int live;
  block_scan(used, &live, red);
  int holes = 0, movers = 0;
  for (long long base = 0; base < c.n_pages; base += 4 * kPlanThreads) {
    const long long p = base + 4 * tid;
    const int4 v = four(p);
    const int r[4] = {v.x, v.y, v.z, v.w};
    unsigned hole = 0, mover = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (p + k >= c.n_pages) continue;
      hole |= (p + k < live && r[k] <= 0) << k;
      mover |= (p + k >= live && r[k] > 0) << k;
      if (p + k >= live && r[k] <= 0) w.list[p + k] = -1;   // (what an earlier call left there is not this one's)
    }
    int total;   // both counts in one scan: holes in the low half, movers in the high half
    const int s = block_scan(static_cast<int>(__popc(hole) | __popc(mover) << 16), &total, red);
    int h = holes + (s & 0xFFFF), m = movers + (s >> 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (hole >> k & 1) w.dst[h++] = static_cast<int>(p) + k;
      if (mover >> k & 1) {
        w.src[m] = static_cast<int>(p) + k;
        w.rows[m++] = c.page_size;
      }
    }
    holes += total & 0xFFFF;
    movers += total >> 16;
  }
  __syncthreads();
  for (int i = tid; i < movers; i += kPlanThreads) {
    const int a = w.src[i], b = w.dst[i];
    w.list[a] = b;
    c.ref[b] = c.ref[a];
    c.ref[a] = 0;
  }
  if (tid == 0) {
    w.count[0] = movers;
    w.count[1] = live;
  }
}

// The table entries of moved pages, by the whole grid of the copy kernel.
__device__ void remap_table(const mk_paged_cache& c) {
  const Work w = work_of(c);
  const int live = w.count[1];
  const unsigned total = static_cast<unsigned>(c.n_seqs) * c.max_pages;   // below 2^31 (checked by the host)
  for (unsigned i = blockIdx.x * blockDim.x + threadIdx.x; i < total; i += gridDim.x * blockDim.x) {
    const int s = i / c.max_pages, j = i - s * c.max_pages, p = c.table[i];
    if (static_cast<long long>(j) * c.page_size >= c.len[s] || p < live || p >= c.n_pages) continue;
    const int to = w.list[p];
    if (to >= 0) c.table[i] = to;   // a page that is named but not counted in ref stays where it is
  }
}

// Page copies. A warp's task is up to 256 16-byte vectors of one (page pair, layer, K or V, head), 8 in flight a
// lane: the two divisions that find it are paid once, inside it an address is a shift and a product whatever the
// strides (divisions for every vector made the copy bound by instructions: 70 % of the issue slots), and a few
// pages still reach every SM.
struct CopyArgs {
  mk_paged_cache from, to;
  const int *src, *dst, *rows;   // rows null: whole pages
  const int* count;              // null: n
  int n;
  int remap;                     // compaction: the table follows the pages
  int* err;
};
constexpr int kCopyThreads = 128, kCopyWarps = kCopyThreads / 32, kCopyVec = 256, kCopyPer = 8;

__global__ void __launch_bounds__(kCopyThreads) copy_pages(const __grid_constant__ CopyArgs a) {
  if (a.count) asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while its plan still runs
  const mk_paged_cache& f = a.from;
  const mk_paged_cache& t = a.to;
  const int count = a.count ? *a.count : a.n;
  if (a.remap && count > 0) remap_table(f);
  const int dv = f.head_dim / 8, sh = __ffs(dv) - 1, lane = threadIdx.x & 31;   // vectors of a row (a power of two)
  const unsigned triples = static_cast<unsigned>(f.n_layers) * 2u * f.kv_heads;
  const unsigned chunks = (static_cast<unsigned>(f.page_size) * dv + kCopyVec - 1) / kCopyVec;   // of a triple's page
  const unsigned page_tasks = triples * chunks;   // below 2^31 (checked by the host)
  for (unsigned long long task = blockIdx.x * static_cast<unsigned long long>(kCopyWarps) + (threadIdx.x >> 5);
       task < static_cast<unsigned long long>(page_tasks) * count; task += static_cast<unsigned long long>(gridDim.x) * kCopyWarps) {
    const int pair = static_cast<int>(task / page_tasks);
    const unsigned in = static_cast<unsigned>(task - static_cast<unsigned long long>(pair) * page_tasks);
    const int ps = a.src[pair], pd = a.dst[pair];
    const unsigned total = static_cast<unsigned>(a.rows ? a.rows[pair] : f.page_size) * dv;   // vectors of a triple
    if (ps < 0 || ps >= f.n_pages || pd < 0 || pd >= t.n_pages) {
      if (lane == 0) atomicOr(a.err, MK_DEVERR_BAD_PAGE);
      continue;
    }
    const unsigned triple = in / chunks, v0 = (in - triple * chunks) * kCopyVec, lk = triple / f.kv_heads;
    const int h = static_cast<int>(triple - lk * f.kv_heads), layer = static_cast<int>(lk >> 1);
    const bool val = lk & 1;
    const uint16_t* s = static_cast<const uint16_t*>(val ? f.v : f.k) + layer * f.layer_stride + ps * f.page_stride + h * f.head_stride;
    uint16_t* d = static_cast<uint16_t*>(val ? t.v : t.k) + layer * t.layer_stride + pd * t.page_stride + h * t.head_stride;
    for (unsigned v = v0 + lane; v < min(total, v0 + kCopyVec); v += 32 * kCopyPer) {
      uint4 x[kCopyPer];
#pragma unroll
      for (int j = 0; j < kCopyPer; ++j) {
        const unsigned w = v + 32 * j;
        if (w < total) x[j] = *reinterpret_cast<const uint4*>(s + (w >> sh) * f.slot_stride + (w & (dv - 1)) * 8);
      }
#pragma unroll
      for (int j = 0; j < kCopyPer; ++j) {
        const unsigned w = v + 32 * j;
        if (w < total) *reinterpret_cast<uint4*>(d + (w >> sh) * t.slot_stride + (w & (dv - 1)) * 8) = x[j];
      }
    }
  }
}

// Grid for at most `pairs` copies of whole pages, and at most `most` blocks an SM over the launch. Blocks beyond
// what an SM holds even out the end of a large copy (357 MB: a call 70 us with 64 of them, 80 with 4), but a call that usually
// copies nothing should not pay for them.
cudaError_t launch_copy(const CopyArgs& a, long long pairs, int most, cudaStream_t s) {
  const long long chunks = (static_cast<long long>(a.from.page_size) * (a.from.head_dim / 8) + kCopyVec - 1) / kCopyVec;
  const long long tasks = (2ll * a.from.n_layers * a.from.kv_heads * chunks + kCopyWarps - 1) / kCopyWarps, cap = 148ll * most;
  const long long grid = tasks > cap / std::max(1ll, pairs) ? cap : tasks * pairs;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(std::max(1ll, grid)));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = a.count ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, copy_pages, a);
}

// The copies number the 16-byte vectors of a page in 32 bits.
bool page_too_large(const mk_paged_cache* c) {
  const double vec = 2.0 * c->n_layers * c->kv_heads * c->page_size * (c->head_dim / 8);
  return vec > 2147000000.0;
}
constexpr const char* kTooLarge = "a page of all layers must be smaller than 32 GB";

int refuse(const char* who, const char* why) {
  mk_set_last_error(std::string(who) + ": " + why);
  return MK_ERR_ARG;
}
int done(const char* who, cudaError_t e) {
  if (e == cudaSuccess) return MK_OK;
  mk_set_last_error(std::string(who) + ": " + cudaGetErrorString(e));
  return MK_ERR_CUDA;
}

using PlanKernel = void (*)(mk_paged_cache, const int*, const int*, int);
cudaError_t launch_plan(PlanKernel kernel, const mk_paged_cache& c, const int* a, const int* b, int n, cudaStream_t s) {
  static std::atomic<uint64_t> attr_set{0};   // per device, both kernels
  const cudaError_t e = once_per_device(attr_set, [] {
    const int bytes = kRefCached * static_cast<int>(sizeof(int));
    const cudaError_t e1 = cudaFuncSetAttribute(plan_resize, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return e1 != cudaSuccess ? e1 : cudaFuncSetAttribute(plan_fork, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
  if (e != cudaSuccess) return e;
  const size_t counts = (static_cast<size_t>(c.n_pages) * sizeof(int) + 15) & ~size_t(15);
  const size_t bytes = c.n_pages > kRefCached ? 0 : c.n_pages > kListCached ? counts : 2 * counts;
  kernel<<<1, kPlanThreads, bytes, s>>>(c, a, b, n);
  return cudaGetLastError();
}

cudaError_t copy_planned(const mk_paged_cache& c, long long pairs, int most, int remap, cudaStream_t s) {
  const Work w = work_of(c);
  return launch_copy(CopyArgs{c, c, w.src, w.dst, w.rows, w.count, 0, remap, c.err}, pairs, most, s);
}

}  // namespace
}  // namespace mk

// ---------------------------------------------------------------- C ABI
extern "C" int64_t mk_pages_work_ints(const mk_paged_cache* c) {
  if (!c || c->n_pages < 1 || c->n_seqs < 1) return 0;
  return 4 + 4ll * c->n_pages + 2ll * c->n_seqs;
}

extern "C" int mk_pages_resize(const mk_paged_cache* c, const int32_t* d_seqs, const int32_t* d_lens, int32_t n, void* stream) {
  const char* who = "mk_pages_resize";
  if (const char* why = mk::paged_cache_problem(c)) return mk::refuse(who, why);
  if (mk::page_too_large(c)) return mk::refuse(who, mk::kTooLarge);
  if (n < 0 || n > c->n_seqs) return mk::refuse(who, "n must lie in 0 .. n_seqs");
  if (n == 0) return MK_OK;
  if (!d_seqs) return mk::refuse(who, "NULL sequence ids");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = mk::launch_plan(mk::plan_resize, *c, d_seqs, d_lens, n, s);
  if (e == cudaSuccess && d_lens) e = mk::copy_planned(*c, n, 2, 0, s);   // freeing replaces no page
  return mk::done(who, e);
}

extern "C" int mk_pages_fork(const mk_paged_cache* c, const int32_t* d_src, const int32_t* d_dst, int32_t n, void* stream) {
  const char* who = "mk_pages_fork";
  if (const char* why = mk::paged_cache_problem(c)) return mk::refuse(who, why);
  if (mk::page_too_large(c)) return mk::refuse(who, mk::kTooLarge);
  if (n < 0 || n > c->n_seqs) return mk::refuse(who, "n must lie in 0 .. n_seqs");
  if (n == 0) return MK_OK;
  if (!d_src || !d_dst) return mk::refuse(who, "NULL sequence ids");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = mk::launch_plan(mk::plan_fork, *c, d_src, d_dst, n, s);
  if (e == cudaSuccess) e = mk::copy_planned(*c, n, 128, 0, s);
  return mk::done(who, e);
}

extern "C" int mk_pages_compact(const mk_paged_cache* c, void* stream) {
  const char* who = "mk_pages_compact";
  if (const char* why = mk::paged_cache_problem(c)) return mk::refuse(who, why);
  if (mk::page_too_large(c)) return mk::refuse(who, mk::kTooLarge);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  mk::plan_compact<<<1, mk::kPlanThreads, 0, s>>>(*c);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = mk::copy_planned(*c, c->n_pages / 2 + 1, 64, 1, s);
  return mk::done(who, e);
}

extern "C" int mk_pages_copy(const mk_paged_cache* from, const mk_paged_cache* to, const int32_t* d_src,
                             const int32_t* d_dst, int32_t n, void* stream) {
  const char* who = "mk_pages_copy";
  if (const char* why = mk::paged_cache_problem(from)) return mk::refuse(who, why);
  if (const char* why = mk::paged_cache_problem(to)) return mk::refuse(who, why);
  if (from->n_layers != to->n_layers || from->kv_heads != to->kv_heads || from->page_size != to->page_size ||
      from->head_dim != to->head_dim)
    return mk::refuse(who, "the caches must agree in n_layers, kv_heads, page_size and head_dim");
  if (mk::page_too_large(from)) return mk::refuse(who, mk::kTooLarge);
  if (n < 0) return mk::refuse(who, "negative count");
  if (n == 0) return MK_OK;
  if (!d_src || !d_dst) return mk::refuse(who, "NULL page ids");
  return mk::done(who, mk::launch_copy(mk::CopyArgs{*from, *to, d_src, d_dst, nullptr, nullptr, n, 0, to->err}, n, 128,
                                       static_cast<cudaStream_t>(stream)));
}
