// Host-side checks shared by the paged-cache entry points, and the row -> (sequence,
// position) lookup of their kernels.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mk.h"

namespace mk {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

// Reason why a cache description is refused, or null.
inline const char* paged_cache_problem(const mk_paged_cache* c) {
  if (!c) return "NULL cache";
  if (!c->k || !c->v || !c->table || !c->len || !c->ref || !c->work || !c->err) return "NULL pointer in the cache";
  if (!aligned16(c->k) || !aligned16(c->v)) return "k and v must be 16-byte aligned";
  if (!head_dim_ok(c->head_dim)) return "head_dim must be 64, 128 or 256";
  if (c->page_size < 8 || c->page_size % 8 || c->page_size > 65536) return "page_size must be a multiple of 8, 8 .. 65536";
  if (c->n_layers < 1 || c->n_pages < 1 || c->kv_heads < 1 || c->n_seqs < 1 || c->max_pages < 1)
    return "n_layers, n_pages, kv_heads, n_seqs and max_pages must be positive";
  if (static_cast<int64_t>(c->max_pages) * c->page_size > (1ll << 30)) return "max_pages * page_size must be at most 2^30";
  if (static_cast<int64_t>(c->n_seqs) * c->max_pages > 0x7fffffffll) return "the table must have fewer than 2^31 entries";
  if (c->layer_stride < 0 || c->layer_stride % 8 || c->page_stride <= 0 || c->page_stride % 8 || c->head_stride <= 0 ||
      c->head_stride % 8 || c->slot_stride < c->head_dim || c->slot_stride % 8)
    return "strides must be positive multiples of 8, slot_stride at least head_dim";
  return nullptr;
}

// New rows of n sequences: rows start[i] .. start[i + 1) belong to sequence seqs[i] (or i).
struct NewRows {
  const int* start;
  const int* seqs;
  int n;
};

// The sequence whose rows contain r (start ascending, start[0] <= r < start[n]): the last i
// with start[i] <= r. One warp, all lanes with the same r: 32 probes a step, so two steps
// find one of 1024 sequences.
__device__ __forceinline__ int find_rows(const NewRows& w, int r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = w.n;   // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int off = lane * step;
    const bool le = off < n && w.start[lo + off] <= r;
    const int k = 31 - __clz(__ballot_sync(0xFFFFFFFFu, le) | 1u);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

}  // namespace mk
