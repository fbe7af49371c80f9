// Pages of a paged KV cache: resizing and freeing sequences, forking, compacting, copying.
//
// Every call but the plain copy is two steps. A planning kernel of one CTA reads lengths, table and use
// counts, decides, and writes them back together with a list of page copies; it is a few
// microseconds of dependent loads, block scans and shared counters, bound by latency, and one
// CTA needs no grid-wide barrier between its phases. A copy kernel then moves the listed pages
// with 16-byte loads and stores over the whole GPU, bound by HBM.
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

// Ranks the free pages below n_pages in ascending order into list until `want` are found;
// returns how many there are (at most about want + one chunk are looked at).
__device__ int list_free(const mk_paged_cache& c, int want, int* list, int* red) {
  constexpr int kPer = 8;
  int found = 0;
  for (long long base = 0; base < c.n_pages && found < want; base += kPlanThreads * kPer) {
    const long long p0 = base + threadIdx.x * kPer;
    unsigned free = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (p0 + j < c.n_pages && c.ref[p0 + j] == 0) free |= 1u << j;
    int total;
    int r = found + block_scan(__popc(free), &total, red);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (free >> j & 1) {
        if (r < want) list[r] = static_cast<int>(p0 + j);
        ++r;
      }
    found += total;
  }
  __syncthreads();
  return found;
}

// Scan of need[0 .. n) in place (exclusive); returns the sum, which may be far above what an
// offset can be (offsets are only used when the sum is at most n_pages).
__device__ long long scan_need(int* need, int n, long long* red) {
  long long sum = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    long long total;
    const long long off = sum + block_scan<long long>(i < n ? need[i] : 0, &total, red);
    if (i < n) need[i] = static_cast<int>(min(off, 0x7fffffffll));
    sum += total;
  }
  __syncthreads();
  return sum;
}

__device__ __forceinline__ bool len_ok(const mk_paged_cache& c, int n) { return n >= 0 && n <= c.max_pages * c.page_size; }

// mk_pages_resize. Phases, a block barrier between them: check everything; give back the
// pages past each new end; count what each sequence takes (a shared partly filled page that stays
// is replaced: its count is read after every release and before any replacement); rank the
// free pages, or undo; write table, counts and lengths.
__global__ void __launch_bounds__(kPlanThreads) plan_resize(mk_paged_cache c, const int* seqs, const int* lens, int n) {
  __shared__ int red[32];
  __shared__ long long red64[32];
  const Work w = work_of(c);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ps = c.page_size;
  if (tid == 0) w.count[0] = 0;
  for (int i = tid; i < c.n_seqs; i += kPlanThreads) w.mark[i] = 0;
  __syncthreads();
  int bad = 0;
  for (int i = tid; i < n; i += kPlanThreads) {
    const int s = seqs[i];
    if (s < 0 || s >= c.n_seqs || atomicAdd(&w.mark[s], 1) || !len_ok(c, c.len[s]) || (lens && !len_ok(c, lens[i]))) bad = 1;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(c.err, MK_DEVERR_BAD_PAGE);
    return;
  }
  // a sequence is one warp's: columns [first, last) are the entries the call touches
  for (int i = warp; i < n; i += kPlanWarps) {
    const int s = seqs[i], old = c.len[s], now = lens ? lens[i] : 0;
    const int* row = c.table + static_cast<long long>(s) * c.max_pages;
    for (int j = min(old, now) / ps + lane; j < pages_of(old, ps); j += 32)
      if (row[j] < 0 || row[j] >= c.n_pages) bad = 1;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(c.err, MK_DEVERR_BAD_PAGE);
    return;
  }
  for (int i = warp; i < n; i += kPlanWarps) {
    const int s = seqs[i], old = c.len[s], now = lens ? lens[i] : 0;
    const int* row = c.table + static_cast<long long>(s) * c.max_pages;
    for (int j = pages_of(now, ps) + lane; j < pages_of(old, ps); j += 32) atomicSub(&c.ref[row[j]], 1);
  }
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const int s = seqs[i], now = lens ? lens[i] : 0, low = min(c.len[s], now);
    int need = max(0, pages_of(now, ps) - pages_of(low, ps));
    const bool own = low % ps && c.ref[c.table[static_cast<long long>(s) * c.max_pages + low / ps]] > 1;
    w.mark[s] = own;
    w.need[i] = need + own;
  }
  __syncthreads();
  const long long total = scan_need(w.need, n, red64);
  const int want = static_cast<int>(min(total, static_cast<long long>(c.n_pages) + 1));
  if (list_free(c, want, w.list, red) < total) {   // nothing changes: take the releases back
    for (int i = warp; i < n; i += kPlanWarps) {
      const int s = seqs[i], old = c.len[s], now = lens ? lens[i] : 0;
      const int* row = c.table + static_cast<long long>(s) * c.max_pages;
      for (int j = pages_of(now, ps) + lane; j < pages_of(old, ps); j += 32) atomicAdd(&c.ref[row[j]], 1);
    }
    if (tid == 0) atomicOr(c.err, MK_DEVERR_NO_PAGES);
    return;
  }
  for (int i = warp; i < n; i += kPlanWarps) {
    const int s = seqs[i], old = c.len[s], now = lens ? lens[i] : 0, low = min(old, now);
    int* row = c.table + static_cast<long long>(s) * c.max_pages;
    const int own = w.mark[s], have = pages_of(low, ps), np = pages_of(now, ps);
    const int* take = w.list + w.need[i];
    if (own && lane == 0) {
      const int e = low / ps, was = row[e], now_p = take[0], at = atomicAdd(&w.count[0], 1);
      w.src[at] = was;
      w.dst[at] = now_p;
      w.rows[at] = low % ps;
      atomicSub(&c.ref[was], 1);
      c.ref[now_p] = 1;
      row[e] = now_p;
    }
    for (int j = have + lane; j < max(np, pages_of(old, ps)); j += 32) {
      const int p = j < np ? take[own + j - have] : -1;
      row[j] = p;
      if (p >= 0) c.ref[p] = 1;
    }
    __syncwarp();
    if (lane == 0) c.len[s] = now;
  }
}

// mk_pages_fork, the same phases: give back what the destinations hold, count the partly
// filled pages, rank free ones, share and write.
__global__ void __launch_bounds__(kPlanThreads) plan_fork(mk_paged_cache c, const int* src, const int* dst, int n) {
  __shared__ int red[32];
  __shared__ long long red64[32];
  const Work w = work_of(c);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ps = c.page_size;
  if (tid == 0) w.count[0] = 0;
  for (int i = tid; i < c.n_seqs; i += kPlanThreads) w.mark[i] = 0;
  __syncthreads();
  int bad = 0;
  for (int i = tid; i < n; i += kPlanThreads) {
    const int a = src[i], b = dst[i];
    if (a < 0 || a >= c.n_seqs || b < 0 || b >= c.n_seqs || atomicAdd(&w.mark[b], 1) || !len_ok(c, c.len[a]) ||
        !len_ok(c, c.len[b]))
      bad = 1;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(c.err, MK_DEVERR_BAD_PAGE);
    return;
  }
  for (int i = warp; i < n; i += kPlanWarps) {
    const int a = src[i], b = dst[i];
    if (w.mark[a]) bad = 1;   // a source that is also a destination
    const int* ra = c.table + static_cast<long long>(a) * c.max_pages;
    const int* rb = c.table + static_cast<long long>(b) * c.max_pages;
    for (int j = lane; j < pages_of(c.len[a], ps); j += 32)
      if (ra[j] < 0 || ra[j] >= c.n_pages) bad = 1;
    for (int j = lane; j < pages_of(c.len[b], ps); j += 32)
      if (rb[j] < 0 || rb[j] >= c.n_pages) bad = 1;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(c.err, MK_DEVERR_BAD_PAGE);
    return;
  }
  for (int i = warp; i < n; i += kPlanWarps) {
    const int b = dst[i];
    const int* rb = c.table + static_cast<long long>(b) * c.max_pages;
    for (int j = lane; j < pages_of(c.len[b], ps); j += 32) atomicSub(&c.ref[rb[j]], 1);
  }
  for (int i = tid; i < n; i += kPlanThreads) w.need[i] = c.len[src[i]] % ps ? 1 : 0;
  __syncthreads();
  const int total = static_cast<int>(scan_need(w.need, n, red64));
  if (list_free(c, total, w.list, red) < total) {
    for (int i = warp; i < n; i += kPlanWarps) {
      const int b = dst[i];
      const int* rb = c.table + static_cast<long long>(b) * c.max_pages;
      for (int j = lane; j < pages_of(c.len[b], ps); j += 32) atomicAdd(&c.ref[rb[j]], 1);
    }
    if (tid == 0) atomicOr(c.err, MK_DEVERR_NO_PAGES);
    return;
  }
  for (int i = warp; i < n; i += kPlanWarps) {
    const int a = src[i], b = dst[i], len = c.len[a], had = c.len[b], np = pages_of(len, ps);
    const int* ra = c.table + static_cast<long long>(a) * c.max_pages;
    int* rb = c.table + static_cast<long long>(b) * c.max_pages;
    for (int j = lane; j < max(np, pages_of(had, ps)); j += 32) {
      int p = -1;
      if (j < len / ps) {
        p = ra[j];
        atomicAdd(&c.ref[p], 1);
      } else if (j < np) {
        p = w.list[w.need[i]];
        const int at = atomicAdd(&w.count[0], 1);
        w.src[at] = ra[j];
        w.dst[at] = p;
        w.rows[at] = len % ps;
        c.ref[p] = 1;
      }
      rb[j] = p;
    }
    __syncwarp();
    if (lane == 0) c.len[b] = len;
  }
}

// mk_pages_compact, counts and copies: pages in use, then the r-th used page with an id past
// them paired with the r-th free id below (there are equally many). list[p] is the new id of
// a moved page p; the table follows in remap_table.
__global__ void __launch_bounds__(kPlanThreads) plan_compact(mk_paged_cache c) {
  __shared__ int red[32];
  const Work w = work_of(c);
  const int tid = threadIdx.x;
  int used = 0;
  for (int p = tid; p < c.n_pages; p += kPlanThreads) used += c.ref[p] > 0;
  int total;
  block_scan(used, &total, red);
  const int live = total;
  int holes = 0, movers = 0;
  for (long long base = 0; base < c.n_pages; base += kPlanThreads) {
    const long long p = base + tid;
    const bool in = p < c.n_pages;
    const int r = in ? c.ref[p] : 0;
    const bool hole = in && p < live && r <= 0, mover = in && p >= live && r > 0;
    // both counts in one scan: holes in the low half, movers in the high half
    const int s = block_scan(static_cast<int>(hole) | static_cast<int>(mover) << 16, &total, red);
    if (hole) w.dst[holes + (s & 0xFFFF)] = static_cast<int>(p);
    if (mover) {
      w.src[movers + (s >> 16)] = static_cast<int>(p);
      w.rows[movers + (s >> 16)] = c.page_size;
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

__global__ void remap_table(mk_paged_cache c) {
  const Work w = work_of(c);
  const int live = w.count[1];
  if (w.count[0] == 0) return;
  const long long total = static_cast<long long>(c.n_seqs) * c.max_pages;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int s = static_cast<int>(i / c.max_pages), j = static_cast<int>(i % c.max_pages);
    const int len = c.len[s], p = c.table[i];
    if (static_cast<long long>(j) * c.page_size >= len || p < live || p >= c.n_pages) continue;
    // a page that is named but not counted in ref stays where it is
    const int to = w.list[p];
    if (to >= 0 && to < live) c.table[i] = to;
  }
}

// Page copies. A task is 2048 16-byte vectors of one page pair (8 in flight per thread); the
// vectors of a pair are numbered over (layer, K or V, head, slot, entry), entries innermost, so
// a warp reads consecutive addresses whatever the strides.
struct CopyArgs {
  mk_paged_cache from, to;
  const int *src, *dst, *rows;   // rows null: whole pages
  const int* count;              // null: n
  int n;
  int* err;
};
constexpr int kCopyThreads = 256, kCopyPer = 8;

__global__ void __launch_bounds__(kCopyThreads) copy_pages(CopyArgs a) {
  const mk_paged_cache& f = a.from;
  const mk_paged_cache& t = a.to;
  const int count = a.count ? *a.count : a.n;
  const int dv = f.head_dim / 8, sh = __ffs(dv) - 1;   // vectors of a row (a power of two)
  const unsigned per_max = static_cast<unsigned>(f.n_layers) * 2u * f.kv_heads;   // (layer, K or V, head) triples
  const unsigned page_tasks = (per_max * f.page_size * dv + kCopyThreads * kCopyPer - 1) / (kCopyThreads * kCopyPer);
  for (unsigned long long task = blockIdx.x; task < static_cast<unsigned long long>(page_tasks) * count; task += gridDim.x) {
    const int pair = static_cast<int>(task / page_tasks);
    const int ps = a.src[pair], pd = a.dst[pair];
    const unsigned rows = a.rows ? a.rows[pair] : f.page_size;
    const unsigned total = per_max * rows * dv;   // below 2^31 (checked by the host)
    const unsigned v0 = static_cast<unsigned>(task - static_cast<unsigned long long>(pair) * page_tasks) * (kCopyThreads * kCopyPer) +
                        threadIdx.x;
    if (ps < 0 || ps >= f.n_pages || pd < 0 || pd >= t.n_pages) {
      if (threadIdx.x == 0) atomicOr(a.err, MK_DEVERR_BAD_PAGE);
      continue;
    }
    uint4 x[kCopyPer];
    uint4* to[kCopyPer];
#pragma unroll
    for (int j = 0; j < kCopyPer; ++j) {
      const unsigned v = v0 + j * kCopyThreads;
      to[j] = nullptr;
      if (v < total) {
        const unsigned row = v >> sh, triple = row / rows, lk = triple / f.kv_heads;
        const int e = static_cast<int>(v & (dv - 1)) * 8;
        const int slot = static_cast<int>(row - triple * rows);
        const int h = static_cast<int>(triple - lk * f.kv_heads);
        const int layer = static_cast<int>(lk >> 1);
        const bool val = lk & 1;
        const uint16_t* s = static_cast<const uint16_t*>(val ? f.v : f.k) + layer * f.layer_stride + ps * f.page_stride +
                            h * f.head_stride + slot * f.slot_stride + e;
        uint16_t* d = static_cast<uint16_t*>(val ? t.v : t.k) + layer * t.layer_stride + pd * t.page_stride +
                      h * t.head_stride + slot * t.slot_stride + e;
        x[j] = *reinterpret_cast<const uint4*>(s);
        to[j] = reinterpret_cast<uint4*>(d);
      }
    }
#pragma unroll
    for (int j = 0; j < kCopyPer; ++j)
      if (to[j]) *to[j] = x[j];
  }
}

// Grid for at most `pairs` copies of whole pages.
cudaError_t launch_copy(const CopyArgs& a, long long pairs, cudaStream_t s) {
  const long long vec = 2ll * a.from.n_layers * a.from.kv_heads * a.from.page_size * (a.from.head_dim / 8);
  const long long tasks = (vec + kCopyThreads * kCopyPer - 1) / (kCopyThreads * kCopyPer);
  const long long grid = std::min<long long>(148 * 4, tasks > (148 * 4) / std::max(1ll, pairs) ? 148 * 4 : tasks * pairs);
  copy_pages<<<static_cast<int>(std::max(1ll, grid)), kCopyThreads, 0, s>>>(a);
  return cudaGetLastError();
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

cudaError_t copy_planned(const mk_paged_cache& c, long long pairs, cudaStream_t s) {
  const Work w = work_of(c);
  return launch_copy(CopyArgs{c, c, w.src, w.dst, w.rows, w.count, 0, c.err}, pairs, s);
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
  mk::plan_resize<<<1, mk::kPlanThreads, 0, s>>>(*c, d_seqs, d_lens, n);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && d_lens) e = mk::copy_planned(*c, n, s);   // freeing replaces no page
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
  mk::plan_fork<<<1, mk::kPlanThreads, 0, s>>>(*c, d_src, d_dst, n);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = mk::copy_planned(*c, n, s);
  return mk::done(who, e);
}

extern "C" int mk_pages_compact(const mk_paged_cache* c, void* stream) {
  const char* who = "mk_pages_compact";
  if (const char* why = mk::paged_cache_problem(c)) return mk::refuse(who, why);
  if (mk::page_too_large(c)) return mk::refuse(who, mk::kTooLarge);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  mk::plan_compact<<<1, mk::kPlanThreads, 0, s>>>(*c);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) {
    const long long entries = static_cast<long long>(c->n_seqs) * c->max_pages;
    mk::remap_table<<<static_cast<int>(std::min<long long>((entries + 255) / 256, 148 * 8)), 256, 0, s>>>(*c);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = mk::copy_planned(*c, c->n_pages / 2 + 1, s);
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
  return mk::done(who, mk::launch_copy(mk::CopyArgs{*from, *to, d_src, d_dst, nullptr, nullptr, n, to->err}, n,
                                       static_cast<cudaStream_t>(stream)));
}
