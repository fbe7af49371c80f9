// Causal attention of new tokens over the pages of a KV cache, on the sm_100a tensor cores.
//
// The query heads that share a kv head are packed: row rr of a sequence and kv head is token
// rr / group, head kv_head * group + rr % group, so one pass over the keys serves the whole group. A tile
// is 128 such rows against 128 keys, and a work unit is one (row tile, key tile). All units of a call,
// in the order sequence, kv head, row tile, key tile, are cut into one equal run per CTA (one CTA
// per SM), so a single long sequence spreads over the whole GPU and ragged ones balance; a row
// tile whose key range is cut leaves partial results (O, m, l), which a second kernel joins.
//
// Per key tile, with the scores in log2 units (c = scale log2 e):
//   S = Q K^T                         tcgen05, M = 128, N = 128, K = D, into TMEM
//   m = max(m, rowmax(c S));  P = 2^(c S - m), masked above the diagonal;  l += rowsum(P)
//   O = O + P V                       tcgen05, P (bf16) read from TMEM over the columns of S
// m is only raised (and O, l rescaled) when a tile's maximum passes it by more than 2^8, so
// weights are at most 2^8 and the result O / l is the same softmax. m, l, S, O and the partial results
// are fp32; a weight is rounded to bf16 once, as an operand, and the result once, at the end.
//
// Roles of the 12 warps: 0-7 softmax (two warps per 32 rows, each half of the tile's keys) and
// epilogue, 8 TMA producer, 9 MMA issuer, 10 scheduler. Keys and values go through a ring of
// shared-memory slots (128 keys x min(D, 128) entries), filled by TMA boxes that follow the page table (a
// box is the largest power of two of slots that divides the page size, at most 128); the order
// K0 K1 V0 K2 V1 ... is the order of use, and it runs on across row tiles, so memory stays busy through
// softmax and epilogue. Values are taken as they lie in the page (transposed by the MMA descriptor).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cuda.h>
#include <string>

#include "dev.cuh"
#include "mk_internal.h"
#include "mk_model.h"
#include "paged.h"
#include "tc.cuh"

namespace mk {
namespace {

constexpr int kM = 128, kN = 128;        // rows and keys of a tile
constexpr int kSoftWarps = 8;
constexpr int kThreads_ = 384;
constexpr int kSegs = 4;                 // segments the scheduler runs ahead
constexpr float kRaise = 8.0f;           // log2 units
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kPanel = 128 * 128;        // 64 bf16 entries of 128 rows: 16 KB
constexpr int kBarBytes = 3072;

template <int D>
struct Lay {
  static constexpr int kCW = D < 128 ? D : 128;       // entries of a ring slot's rows
  static constexpr int kCh = D / kCW;                 // slots of a key (or value) tile
  static constexpr int kSlot = kCW / 64 * kPanel;
  static constexpr int kQ = D / 64 * kPanel;
  static constexpr int kSlots = D == 256 ? 5 : D == 128 ? 6 : 8;
  static constexpr int kOffBars = kQ + kSlots * kSlot;
  static constexpr int kSmem = kOffBars + kBarBytes;
  // TMEM columns: O [0, D), then two score buffers of 128, whose first 64 columns take P
  static constexpr uint32_t kColS = D;
};
static_assert(Lay<256>::kSmem <= 232448 && Lay<128>::kSmem <= 232448, "fits the SM");

struct AttnArgs {
  mk_paged_cache c;
  int layer, rows, hq, group, box;
  const uint16_t* q;
  long long ldq;
  uint16_t* o;
  long long ldo;
  float c2;                // |scale| log2 e
  int negative;            // the sign of scale
  NewRows w;
  float* part;             // [2 * grid][max_rows][D]
  float2* ml;              // [2 * grid][max_rows] (m, l)
  int* meta;               // [2 * grid][kMeta]
  int max_rows;
};
// Partial results of one slot: first / last flags (kPart*), rows, first packed row, kv head, the
// sequence's first row.
constexpr int kMeta = 8;
constexpr int kPartUsed = 1, kPartFirst = 2, kPartLast = 4;

// One stretch of key tiles of one row tile.
struct Segment {
  int end;                 // no more segments
  int row0, new_rows;      // the sequence's first row and its rows
  int pos0;                // position of row0
  int len;                 // positions of the sequence
  int seq;                 // row of the page table
  int kvh, tile;           // kv head, row tile
  int t0, t1;              // key tiles
  int part;                // slot of the partial results, or -1
  int flags;
};

struct Bars {
  uint64_t full[8], empty[8], s_full[2], p_full[2], o_done[2], q_full, pair[4], seg_full[kSegs], seg_empty[kSegs];
  uint32_t tmem;
  int abort;
  Segment seg[kSegs];
  float mx[2][2][kM];      // [tile parity][half][row]; also takes l at the end of a row tile
};
static_assert(sizeof(Bars) <= kBarBytes, "barriers fit their slot");

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// D (TMEM) += A (TMEM, bf16 pairs in 32-bit columns) * B (shared memory).
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Values as they lie in a slot: entries of a position contiguous (MN-major), 128-byte swizzle: panels of 64
// entries kPanel bytes apart (leading offset), groups of 8 positions 1024 bytes apart (stride).
__device__ __forceinline__ uint64_t desc_mnmajor_sw128(const void* p) {
  const uint32_t a = smem_u32(p);
  return static_cast<uint64_t>((a >> 4) & 0x3FFF) | static_cast<uint64_t>(kPanel >> 4) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
constexpr uint32_t kBMajorMN = 1u << 16;   // instruction descriptor: B is MN-major

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ bool wait_bar(Bars* b, uint64_t* bar, uint32_t parity, int* err) {
  if (mbar_wait(bar, parity, &b->abort, kWaitNs)) return true;
  if (!b->abort) atomicOr(err, MK_DEVERR_PIPE_TIMEOUT);
  b->abort = 1;
  return false;
}
__device__ __forceinline__ bool warp_wait(Bars* b, uint64_t* bar, uint32_t parity, int* err) {
  const bool ok = wait_bar(b, bar, parity, err);
  return __all_sync(0xFFFFFFFFu, ok);
}

// Meeting point of the two warps that share 32 rows (bounded, unlike a named barrier); n counts their meetings.
__device__ __forceinline__ bool pair_sync(Bars* b, int quarter, uint32_t& n, int* err) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&b->pair[quarter]);
  return warp_wait(b, &b->pair[quarter], n++ & 1, err);
}

// What one sequence of the call asks for. A sequence that does not exist, or a length the table cannot
// hold, counts as one without positions: its rows become zeros.
struct SeqWork {
  int row0, rows, pos0, len, seq, row_tiles;
};
__device__ __forceinline__ SeqWork seq_work(const AttnArgs& a, int i, int* bad) {
  SeqWork w{};
  if (i >= a.w.n) return w;
  const int b = a.w.start[i], e = a.w.start[i + 1], s = a.w.seqs ? a.w.seqs[i] : i;
  w.row0 = max(b, 0);
  w.rows = max(0, min(e, a.rows) - w.row0);
  const bool there = s >= 0 && s < a.c.n_seqs;
  const int len = there ? a.c.len[s] : -1;
  const bool ok = len >= 0 && len <= a.c.max_pages * a.c.page_size;
  *bad |= !ok && w.rows > 0;
  w.seq = there ? s : 0;
  w.len = ok ? len : 0;
  w.pos0 = w.len - (e - w.row0);
  w.row_tiles = (w.rows * a.group + kM - 1) / kM;   // below 2^30 (checked by the host)
  return w;
}
// Key tiles of row tile j: up to the position of its last row; one (empty) where it sees nothing.
__device__ __forceinline__ int key_tiles(const AttnArgs& a, const SeqWork& w, int j) {
  const int last = min((j + 1) * kM, w.rows * a.group) - 1;
  const int keys = w.pos0 + last / a.group + 1;
  return max(1, (keys + kN - 1) / kN);
}
__device__ __forceinline__ SeqWork shfl_work(const SeqWork& w, int src) {
  return SeqWork{__shfl_sync(0xFFFFFFFFu, w.row0, src), __shfl_sync(0xFFFFFFFFu, w.rows, src), __shfl_sync(0xFFFFFFFFu, w.pos0, src),
                 __shfl_sync(0xFFFFFFFFu, w.len, src),  __shfl_sync(0xFFFFFFFFu, w.seq, src),  __shfl_sync(0xFFFFFFFFu, w.row_tiles, src)};
}
// Units of one kv head of each lane's sequence: short ones by their lane, long ones by the warp.
__device__ long long head_units(const AttnArgs& a, const SeqWork& w) {
  const int lane = threadIdx.x & 31;
  long long u = 0;
  if (w.row_tiles <= 4)
    for (int j = 0; j < w.row_tiles; ++j) u += key_tiles(a, w, j);
  for (unsigned big = __ballot_sync(0xFFFFFFFFu, w.row_tiles > 4); big; big &= big - 1) {
    const int src = __ffs(big) - 1;
    const SeqWork x = shfl_work(w, src);
    int sum = 0;
    for (int j = lane; j < x.row_tiles; j += 32) sum += key_tiles(a, x, j);
    const int t = __reduce_add_sync(0xFFFFFFFFu, sum);
    if (lane == src) u = t;
  }
  return u;
}
__device__ __forceinline__ long long warp_sum64(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ long long warp_scan64(long long v) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) >= o) v += y;
  }
  return v;
}

template <int D>
__global__ void __launch_bounds__(kThreads_, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const __grid_constant__ AttnArgs a) {
  using L = Lay<D>;
  extern __shared__ __align__(1024) uint8_t smem[];   // swizzled tiles need 1024-byte alignment
  uint8_t* ring = smem + L::kQ;
  Bars* b = reinterpret_cast<Bars*>(smem + L::kOffBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* err = a.c.err;
  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) atomicOr(err, MK_DEVERR_PIPE_TIMEOUT);
    return;
  }

  if (threadIdx.x == 0) {
    b->abort = 0;
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(&b->full[i], 1);
      mbar_init(&b->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b->s_full[i], 1);
      mbar_init(&b->p_full[i], kSoftWarps);
      mbar_init(&b->o_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&b->pair[i], 2);
    mbar_init(&b->q_full, kSoftWarps);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&b->seg_full[i], 1);
      mbar_init(&b->seg_empty[i], kSoftWarps + 2);
    }
    fence_barrier_init();
  }
  if (warp == 8) {
    if (lane == 0) {
      tc::prefetch_tensormap(&tk);
      tc::prefetch_tensormap(&tv);
    }
    tc::tmem_alloc(&b->tmem, 512);
    tc::tmem_relinquish();
  }
  // units of every group of 32 sequences, one warp per group (in the ring's memory, before its first use)
  long long* groups = reinterpret_cast<long long*>(ring);
  const int n_groups = (a.w.n + 31) / 32;
  for (int g = warp; g < n_groups; g += kThreads_ / 32) {
    int bad = 0;
    const SeqWork w = seq_work(a, g * 32 + lane, &bad);
    const long long u = warp_sum64(head_units(a, w)) * a.c.kv_heads;
    if (lane == 0) groups[g] = u;
    if (bad && blockIdx.x == 0) atomicOr(err, MK_DEVERR_BAD_PAGE);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  long long total = 0, before = 0, u0 = 0, u1 = 0;   // scheduler: all units, units before its group, its range
  int g = 0;
  if (warp == 10) {
    for (int i = lane; i < n_groups; i += 32) total += groups[i];
    total = warp_sum64(total);
    const long long ctas = min(static_cast<long long>(gridDim.x), total);   // each with work, the first ones
    if (blockIdx.x < ctas) {
      u0 = total * blockIdx.x / ctas;
      u1 = total * (blockIdx.x + 1) / ctas;
    }
    for (; g + 1 < n_groups && before + groups[g] <= u0; ++g) before += groups[g];
  }
  tc::fence_proxy_async_smem();
  __syncthreads();   // the ring is the producer's from here
  const uint32_t tmem = b->tmem;

  if (warp == 10) {
    // ---- scheduler: cut [u0, u1) into segments
    int emitted = 0, made = 0;
    bool ok = true;
    auto emit = [&](const Segment& s) {
      const int k = emitted % kSegs;
      if (emitted >= kSegs) ok = warp_wait(b, &b->seg_empty[k], (emitted / kSegs - 1) & 1, err);
      if (!ok) return;
      if (lane == 0) {
        b->seg[k] = s;
        mbar_arrive(&b->seg_full[k]);
      }
      ++emitted;
    };
    for (int k = lane; k < 2 * kMeta; k += 32) a.meta[blockIdx.x * 2 * kMeta + k] = 0;
    __syncwarp();
    long long u = u0;
    for (; u < u1 && ok && g < n_groups; ++g) {
      int bad = 0;
      const SeqWork mine = seq_work(a, g * 32 + lane, &bad);
      const long long hu = head_units(a, mine), units = hu * a.c.kv_heads;
      const long long incl = before + warp_scan64(units);
      while (ok && u < u1) {
        const unsigned past = __ballot_sync(0xFFFFFFFFu, incl > u);
        if (!past) break;
        const int src = __ffs(past) - 1;
        const SeqWork w = shfl_work(mine, src);
        const long long h = __shfl_sync(0xFFFFFFFFu, hu, src);
        const long long rel = u - __shfl_sync(0xFFFFFFFFu, incl - units, src);
        Segment s{};
        s.row0 = w.row0, s.new_rows = w.rows, s.pos0 = w.pos0, s.len = w.len, s.seq = w.seq;
        s.kvh = static_cast<int>(rel / h);
        int rem = static_cast<int>(rel - s.kvh * h), tiles = 0;
        for (int j0 = 0;; j0 += 32) {              // the row tile that holds unit rem of this head
          const int t = j0 + lane < w.row_tiles ? key_tiles(a, w, j0 + lane) : 0;
          const int inc = static_cast<int>(warp_scan64(t));
          const unsigned hit = __ballot_sync(0xFFFFFFFFu, inc > rem);
          if (hit) {
            const int k = __ffs(hit) - 1;
            s.tile = j0 + k;
            tiles = __shfl_sync(0xFFFFFFFFu, t, k);
            rem -= __shfl_sync(0xFFFFFFFFu, inc, k) - tiles;
            break;
          }
          rem -= __shfl_sync(0xFFFFFFFFu, inc, 31);
        }
        s.t0 = rem;
        s.t1 = static_cast<int>(min(static_cast<long long>(tiles), rem + (u1 - u)));
        const bool whole = s.t0 == 0 && s.t1 == tiles;
        s.part = whole ? -1 : static_cast<int>(blockIdx.x) * 2 + (made ? 1 : 0);
        u += s.t1 - s.t0;
        ++made;
        if (!whole && lane == 0) {
          int* m = a.meta + static_cast<long long>(s.part) * kMeta;
          m[0] = kPartUsed | (s.t0 == 0 ? kPartFirst : 0) | (s.t1 == tiles ? kPartLast : 0);
          m[1] = min(kM, w.rows * a.group - s.tile * kM);
          m[2] = s.tile;
          m[3] = s.kvh;
          m[4] = s.row0;
        }
        emit(s);
      }
      before = __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    Segment stop{};
    stop.end = 1;
    if (ok) emit(stop);
  } else if (warp == 8) {
    // ---- TMA producer
    uint32_t slot = 0;   // slots filled so far
    bool ok = true;
    const int per_tile = kN / a.box;
    auto load = [&](const Segment& s, const CUtensorMap* map, int tile, int page) {
      // lane i < per_tile holds the page of box i of the tile (-1: past the sequence's end)
      const int valid = min(per_tile, (s.len - tile * kN + a.box - 1) / a.box);
      for (int c = 0; c < L::kCh; ++c, ++slot) {
        const uint32_t k = slot % L::kSlots;
        if (slot >= L::kSlots) ok = ok && warp_wait(b, &b->empty[k], (slot / L::kSlots - 1) & 1, err);
        if (!ok) return;
        if (lane == 0) mbar_arrive_expect_tx(&b->full[k], valid * a.box * L::kCW * 2);
        __syncwarp();
        if (lane < valid) {
          const int at = (tile * kN + lane * a.box) % a.c.page_size;
          for (int p = 0; p < L::kCW / 64; ++p)
            tma_load_4d(ring + k * L::kSlot + p * kPanel + lane * a.box * 128, map, c * L::kCW + p * 64, at, s.kvh, page, &b->full[k]);
        }
      }
    };
    for (int i = 0; ok; ++i) {
      if (!warp_wait(b, &b->seg_full[i % kSegs], (i / kSegs) & 1, err)) break;
      const Segment s = b->seg[i % kSegs];
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->seg_empty[i % kSegs]);
      if (s.end) break;
      const int* row = a.c.table + static_cast<long long>(s.seq) * a.c.max_pages;
      auto page_of = [&](int tile) {
        const int p = tile * kN + lane * a.box;
        if (tile >= s.t1 || lane >= per_tile || p >= s.len) return -1;
        const int page = row[p / a.c.page_size];
        if (page >= 0 && page < a.c.n_pages) return page;
        atomicOr(err, MK_DEVERR_BAD_PAGE);
        return a.c.n_pages;                        // outside the tensor map: reads as zeros
      };
      if (s.len == 0) continue;                    // nothing to read
      // page ids one tile ahead of the loads that use them
      int now = page_of(s.t0), next = page_of(s.t0 + 1);
      load(s, &tk, s.t0, now);
      for (int t = s.t0; t < s.t1 && ok; ++t) {
        const int after = page_of(t + 2);
        if (t + 1 < s.t1) load(s, &tk, t + 1, next);
        if (ok) load(s, &tv, t, now);
        now = next;
        next = after;
      }
    }
    if (!ok && lane == 0) {                        // copies in flight land before the CTA ends (bounded)
      int never = 0;
      for (uint32_t k = slot < L::kSlots ? 0u : slot - L::kSlots; k < slot; ++k)
        mbar_wait(&b->full[k % L::kSlots], (k / L::kSlots) & 1, &never, kWaitNs / 10);
    }
  } else if (warp == 9) {
    if (lane == 0) {
      // ---- MMA issuer
      constexpr uint32_t id_s = tc::idesc_bf16_f32(kM, kN), id_o = tc::idesc_bf16_f32(kM, L::kCW) | kBMajorMN;
      uint32_t slot = 0, it = 0, nq = 0;
      bool ok = true;
      auto take = [&](uint32_t& k) {               // the next slot in order, filled
        k = slot % L::kSlots;
        ok = ok && wait_bar(b, &b->full[k], (slot / L::kSlots) & 1, err);
        ++slot;
        tc::fence_after_sync();
        return ok;
      };
      auto scores = [&](uint32_t n) {             // S buffer n & 1; its P was consumed by the product before
        const uint32_t d = tmem + L::kColS + (n & 1) * kN;
        for (int c = 0; c < L::kCh; ++c) {
          uint32_t k;
          if (!take(k)) return;
          for (int p = 0; p < L::kCW / 64; ++p)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc::mma_bf16(d, tc::desc_kmajor_sw128(smem + (c * (L::kCW / 64) + p) * kPanel + kk * 32),
                           tc::desc_kmajor_sw128(ring + k * L::kSlot + p * kPanel + kk * 32), id_s, (c | p | kk) ? 1u : 0u);
          tc::mma_commit(&b->empty[k]);
        }
        tc::mma_commit(&b->s_full[n & 1]);
      };
      for (int i = 0; ok; ++i) {
        if (!wait_bar(b, &b->seg_full[i % kSegs], (i / kSegs) & 1, err)) break;
        const Segment s = b->seg[i % kSegs];
        mbar_arrive(&b->seg_empty[i % kSegs]);
        if (s.end) break;
        if (s.len == 0) continue;
        if (!(ok = wait_bar(b, &b->q_full, nq++ & 1, err))) break;
        tc::fence_after_sync();
        scores(it);
        for (int t = s.t0; t < s.t1 && ok; ++t, ++it) {
          if (t + 1 < s.t1) scores(it + 1);
          if (!ok || !(ok = wait_bar(b, &b->p_full[it & 1], (it >> 1) & 1, err))) break;
          const uint32_t pa = tmem + L::kColS + (it & 1) * kN;
          for (int c = 0; c < L::kCh; ++c) {
            uint32_t k;
            if (!take(k)) break;
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)
              mma_bf16_ts(tmem + c * L::kCW, pa + kk * 8, desc_mnmajor_sw128(ring + k * L::kSlot + kk * 2048), id_o,
                          (t > s.t0 || kk) ? 1u : 0u);
            tc::mma_commit(&b->empty[k]);
          }
          if (ok) tc::mma_commit(&b->o_done[it & 1]);
        }
      }
    }
    __syncwarp();
  } else if (warp < kSoftWarps) {
    // ---- softmax and epilogue: row r of the tile, keys half * 64 .. + 63 of each key tile
    const int quarter = warp & 3, half = warp >> 2, r = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t it = 0, slot = 0, meets = 0;
    Segment s;
    // the next segment, and its row tile's queries on their way into the swizzled layout (whose last
    // reader, the row tile before, has computed its scores)
    auto fetch = [&](int i) {
      if (!warp_wait(b, &b->seg_full[i % kSegs], (i / kSegs) & 1, err)) return false;
      s = b->seg[i % kSegs];
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->seg_empty[i % kSegs]);
      if (s.end || s.len == 0) return true;
      constexpr int kLanes = D / 8, kAtOnce = kSoftWarps * 32 / kLanes;   // lanes of a row, rows at once
      const int rows = min(kM, s.new_rows * a.group - s.tile * kM), e = threadIdx.x % kLanes;
      for (int row = threadIdx.x / kLanes; row < rows; row += kAtOnce) {
        const int rr = s.tile * kM + row, tok = rr / a.group, h = s.kvh * a.group + rr - tok * a.group;
        cp_async16(smem + (e >> 3) * kPanel + row * 128 + (((e & 7) ^ (row & 7)) << 4),
                   a.q + static_cast<long long>(s.row0 + tok) * a.ldq + h * D + e * 8, 16);
      }
      cp_async_commit();
      return true;
    };
    auto queries_in = [&] {
      if (s.end || s.len == 0) return;
      cp_async_wait<0>();
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->q_full);
    };
    bool ok = fetch(0);
    if (ok) queries_in();
    for (int i = 0; ok && !s.end;) {
      const int rr0 = s.tile * kM, rows = min(kM, s.new_rows * a.group - rr0);
      const bool live = quarter * 32 < rows;       // the warp has rows of the tile
      const int tok = (rr0 + min(r, rows - 1)) / a.group, pos = s.pos0 + tok;
      const int pos_first = s.pos0 + (rr0 + quarter * 32) / a.group;   // the warp's lowest
      float m = -INFINITY, l = 0.f;                // m in log2 units
      const int n = s.len == 0 ? 0 : s.t1 - s.t0;
      for (int j = 0; j < n; ++j, ++it) {
        const int t = s.t0 + j, buf = it & 1;
        if (!(ok = warp_wait(b, &b->s_full[buf], (it >> 1) & 1, err))) break;
        // long done (it was issued before these scores), but a parity wait must not skip a phase
        if (it >= 2 && !(ok = warp_wait(b, &b->o_done[buf], ((it >> 1) - 1) & 1, err))) break;
        if (live) {
          tc::fence_after_sync();
          const uint32_t sb = tmem + lanes + L::kColS + buf * kN;
          float x[64];
          tmem_ld32(sb + half * 64, x);
          tmem_ld32(sb + half * 64 + 32, x + 32);
          tmem_wait_ld();
          if (a.negative) {
#pragma unroll
            for (int c = 0; c < 64; ++c) x[c] = -x[c];
          }
          const int key0 = t * kN + half * 64;
          if (key0 + 63 > pos_first) {
#pragma unroll
            for (int c = 0; c < 64; ++c) x[c] = key0 + c <= pos ? x[c] : -INFINITY;
          }
          float m0 = x[0], m1 = x[1], m2 = x[2], m3 = x[3];
#pragma unroll
          for (int c = 4; c < 64; c += 4) {
            m0 = fmaxf(m0, x[c]), m1 = fmaxf(m1, x[c + 1]);
            m2 = fmaxf(m2, x[c + 2]), m3 = fmaxf(m3, x[c + 3]);
          }
          m0 = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
          b->mx[buf][half][r] = m0;
          tc::fence_before_sync();
          if (!(ok = pair_sync(b, quarter, meets, err))) break;   // both halves of the scores are in registers
          tc::fence_after_sync();
          const float top = fmaxf(m0, b->mx[buf][half ^ 1][r]) * a.c2;   // -inf where the row sees none
          const bool raise = r < rows && top > m + kRaise;
          if (j == 0) {
            m = top;
          } else if (__any_sync(0xFFFFFFFFu, raise)) {
            // O and l of the rows that raise are rescaled (factor 1 for the others); O is up to
            // date once the product before has completed
            if (!(ok = warp_wait(b, &b->o_done[(it - 1) & 1], ((it - 1) >> 1) & 1, err))) break;
            tc::fence_after_sync();
            const float f = raise ? ex2(m - top) : 1.f;
            l *= f;
            if (raise) m = top;
            for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
              float o[32];
              tmem_ld32(tmem + lanes + c, o);
              tmem_wait_ld();
              uint32_t u[32];
#pragma unroll
              for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(o[k] * f);
              tmem_st32(tmem + lanes + c, u);
            }
          }
          const float sub = m == -INFINITY ? 0.f : -m;
          uint32_t p[32];
          float l0 = 0.f, l1 = 0.f;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float p0 = ex2(fmaf(x[2 * c], a.c2, sub)), p1 = ex2(fmaf(x[2 * c + 1], a.c2, sub));
            l0 += p0, l1 += p1;
            p[c] = pack_bf16(p0, p1);
          }
          l += l0 + l1;
          tmem_st32(sb + half * 32, p);
        }
        if ((t + 1) * kN > s.len) {
          // positions from len on: whatever lies there must not meet a weight of zero as NaN
          const uint32_t at = slot + L::kCh * (j < n - 1 ? 2 * j + 2 : 2 * n - 1);
          for (int c = 0; c < L::kCh && ok; ++c) {
            const uint32_t k = (at + c) % L::kSlots;
            ok = warp_wait(b, &b->full[k], ((at + c) / L::kSlots) & 1, err);
            if (!ok) break;
            const int first = s.len - t * kN;
            for (int v = threadIdx.x; v < (kN - first) * (L::kCW / 8); v += kSoftWarps * 32) {
              const int row = first + v / (L::kCW / 8), e = v % (L::kCW / 8);
              *reinterpret_cast<uint4*>(ring + k * L::kSlot + (e >> 3) * kPanel + row * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
          }
          if (!ok) break;
          tc::fence_proxy_async_smem();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->p_full[buf]);   // two barriers: a warp may be a tile ahead of another
      }
      if (!ok) break;
      slot += 2u * L::kCh * n;
      // row tile, output rows and partial slot of this segment; then the next one's queries, so that
      // its first scores are computed during this epilogue
      const int part = s.part;
      const int h = s.kvh * a.group + rr0 + min(r, rows - 1) - tok * a.group;
      uint16_t* out = a.o + static_cast<long long>(s.row0 + tok) * a.ldo + static_cast<long long>(h) * D;
      if (!(ok = fetch(++i))) break;
      if (n > 0) {
        if (!(ok = warp_wait(b, &b->o_done[(it - 1) & 1], ((it - 1) >> 1) & 1, err))) break;
        tc::fence_after_sync();
      }
      queries_in();
      if (live) {
        // the halves' sums, in the buffer that the last tile did not use
        b->mx[it & 1][half][r] = l;
        if (!(ok = pair_sync(b, quarter, meets, err))) break;
        l += b->mx[it & 1][half ^ 1][r];
        if (!(ok = pair_sync(b, quarter, meets, err))) break;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
          float o[32];
          if (n > 0) {
            tmem_ld32(tmem + lanes + c, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0.f;
          }
          if (r < rows) {
            if (part < 0) {
#pragma unroll
              for (int k = 0; k < 32; k += 8) {
                // a row that saw nothing has l = 0 and takes exact zeros
                *reinterpret_cast<uint4*>(out + c + k) =
                    make_uint4(pack_bf16(o[k] * inv, o[k + 1] * inv), pack_bf16(o[k + 2] * inv, o[k + 3] * inv),
                               pack_bf16(o[k + 4] * inv, o[k + 5] * inv), pack_bf16(o[k + 6] * inv, o[k + 7] * inv));
              }
            } else {
              float4* dst = reinterpret_cast<float4*>(a.part + (static_cast<long long>(part) * a.max_rows + r) * D + c);
#pragma unroll
              for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            }
          }
        }
        if (part >= 0 && half == 0 && r < rows) a.ml[static_cast<long long>(part) * a.max_rows + r] = make_float2(m, l);
        tc::fence_before_sync();
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 8) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Joins the partial results of the row tiles whose keys were cut: with M the largest m of the
// contributors, o = sum 2^(m - M) O / sum 2^(m - M) l. Contributors of a row tile are consecutive CTAs; the
// slot of the first one leads. A block takes the rows y, y + gridDim.y, ... of one leading slot; its 8 warps share the
// contributors of a row, or several rows where there are fewer, and are joined in a fixed order.
constexpr int kJoinY = 16;
template <int D>
__global__ void __launch_bounds__(256) join_parts(const __grid_constant__ AttnArgs a, int slots) {
  constexpr int E = D / 32;
  __shared__ float so[8][D];
  __shared__ float2 sm[8];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lead = blockIdx.x;
  const int* meta = a.meta + static_cast<long long>(lead) * kMeta;
  if ((meta[0] & (kPartUsed | kPartFirst)) != (kPartUsed | kPartFirst)) return;
  const int rows = meta[1], tile = meta[2], kvh = meta[3], row0 = meta[4];
  // contributor k > 0 is slot 2 (lead / 2 + k); the last one is marked
  const int cta = lead / 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n = 0;
  for (int base = 1;; base += 32) {
    const int k = base + lane, slot = 2 * (cta + k);
    const bool last = slot >= slots || (a.meta[static_cast<long long>(slot) * kMeta] & kPartLast);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, last);
    if (hit) {
      n = min(base + __ffs(hit), slots / 2 - cta);
      break;
    }
  }
  int per_row = 1;                                 // warps that share a row
  while (per_row < 8 && per_row * 2 <= n) per_row *= 2;
  const int at_once = 8 / per_row, sub = warp % per_row;
  for (int first = blockIdx.y * at_once; first < rows; first += gridDim.y * at_once) {
    const int r = first + warp / per_row;
    float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    if (r < rows) {
#pragma unroll 4
      for (int k = sub; k < n; k += per_row) {
        const long long at = static_cast<long long>(k ? 2 * (cta + k) : lead) * a.max_rows + r;
        const float2 ml = a.ml[at];
        const float* src = a.part + at * D + lane * E;
        const float top = fmaxf(m, ml.x), f = top == -INFINITY ? 0.f : ex2(m - top), w = top == -INFINITY ? 0.f : ex2(ml.x - top);
        l = l * f + ml.y * w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + src[e] * w;
        m = top;
      }
    }
    if (lane == 0) sm[warp] = make_float2(m, l);
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
    __syncthreads();
    if (sub == 0 && r < rows) {
      float top = m;
      for (int k = 1; k < per_row; ++k) top = fmaxf(top, sm[warp + k].x);
      float f = top == -INFINITY ? 0.f : ex2(m - top);
      l *= f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f;
      for (int k = 1; k < per_row; ++k) {
        f = top == -INFINITY ? 0.f : ex2(sm[warp + k].x - top);
        l += sm[warp + k].y * f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += so[warp + k][lane * E + e] * f;
      }
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int rr = tile * kM + r, tok = rr / a.group, h = kvh * a.group + rr - tok * a.group;
      uint32_t* out = reinterpret_cast<uint32_t*>(a.o + static_cast<long long>(row0 + tok) * a.ldo + static_cast<long long>(h) * D + lane * E);
#pragma unroll
      for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16(o[e] * inv, o[e + 1] * inv);
    }
    __syncthreads();
  }
}

template <int D>
cudaError_t launch_attn(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, int grid, cudaStream_t s) {
  static std::atomic<uint64_t> attr_set{0};   // per device
  cudaError_t e = once_per_device(attr_set, [] {
    return cudaFuncSetAttribute(paged_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kSmem);
  });
  if (e != cudaSuccess) return e;
  paged_attn_kernel<D><<<grid, kThreads_, Lay<D>::kSmem, s>>>(tk, tv, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * grid, std::min(kJoinY, a.max_rows));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;   // launched while the first kernel drains
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_parts<D>, a, 2 * grid);
}

// Key or value pages of a layer as a 4-D tensor: entries, slots, kv heads, pages; a box is 64 entries of `box` slots.
bool page_map(CUtensorMap* map, const mk_paged_cache& c, const void* base, int layer, int box) {
  const uint64_t dims[4] = {static_cast<uint64_t>(c.head_dim), static_cast<uint64_t>(c.page_size), static_cast<uint64_t>(c.kv_heads),
                            static_cast<uint64_t>(c.n_pages)};
  const uint64_t strides[3] = {2ull * c.slot_stride, 2ull * c.head_stride, 2ull * c.page_stride};
  const uint32_t boxes[4] = {64, static_cast<uint32_t>(box), 1, 1};
  return tensor_map_bf16_nd(map, static_cast<const uint16_t*>(base) + layer * c.layer_stride, 4, dims, strides, boxes);
}

int refuse(const std::string& why) {
  mk_set_last_error("mk_paged_attention: " + why);
  return MK_ERR_ARG;
}

struct Scratch {
  size_t part, ml, meta, total;
};
Scratch scratch_of(int grid, int max_rows, int d) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  Scratch s{};
  const size_t rows = 2ull * grid * max_rows;
  s.ml = up(rows * d * sizeof(float));
  s.meta = s.ml + up(rows * sizeof(float2));
  s.total = s.meta + up(2ull * grid * kMeta * sizeof(int));
  return s;
}
int max_rows_of(const mk_paged_cache* c, int rows, int q_heads) {
  return static_cast<int>(std::min<long long>(kM, static_cast<long long>(rows) * (q_heads / c->kv_heads)));
}
int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms;
}

}  // namespace
}  // namespace mk

// ---------------------------------------------------------------- C ABI
extern "C" size_t mk_paged_attention_scratch(const mk_paged_cache* c, int32_t rows, int32_t q_heads) {
  if (mk::paged_cache_problem(c) || rows < 0 || q_heads < 1 || q_heads % c->kv_heads) return 0;
  return mk::scratch_of(mk::sm_count(), mk::max_rows_of(c, rows, q_heads), c->head_dim).total;
}

extern "C" int mk_paged_attention(const mk_paged_cache* c, int32_t layer, const void* d_q, int64_t ldq, int32_t rows,
                                  int32_t q_heads, const int32_t* d_seq_start, const int32_t* d_seqs, int32_t n, float scale,
                                  void* d_out, int64_t ldo, void* d_scratch, size_t scratch_bytes, void* stream) {
  using mk::refuse;
  if (const char* why = mk::paged_cache_problem(c)) return refuse(why);
  if (layer < 0 || layer >= c->n_layers) return refuse("layer out of range");
  if (rows < 0 || n < 0 || n > 65536) return refuse("rows must not be negative, n must lie in 0 .. 65536");
  if (q_heads < 1 || q_heads % c->kv_heads) return refuse("q_heads must be a positive multiple of kv_heads");
  if (!(scale > -INFINITY && scale < INFINITY)) return refuse("scale must be finite");
  if (static_cast<int64_t>(rows) * (q_heads / c->kv_heads) > (1 << 30)) return refuse("rows * group must be at most 2^30");
  if (rows == 0 || n == 0) return MK_OK;
  const int64_t dq = static_cast<int64_t>(q_heads) * c->head_dim;
  if (!d_q || !d_out || !d_seq_start || !d_scratch) return refuse("NULL pointer");
  if (ldq < dq || ldo < dq || ldq % 8 || ldo % 8) return refuse("row pitches must be multiples of 8 that hold the heads");
  if (!mk::aligned16(d_q) || !mk::aligned16(d_out) || !mk::aligned16(d_scratch)) return refuse("pointers must be 16-byte aligned");
  const int max_rows = mk::max_rows_of(c, rows, q_heads);
  const size_t least = mk::scratch_of(1, max_rows, c->head_dim).total;
  if (scratch_bytes < least) return refuse("scratch too small");
  const int grid = mk::sm_count();
  cudaError_t e = grid > 0 ? cudaSuccess : cudaGetLastError();
  if (e == cudaSuccess) {
    const mk::Scratch sc = mk::scratch_of(grid, max_rows, c->head_dim);
    if (scratch_bytes < sc.total) return refuse("scratch too small");
    uint8_t* ws = static_cast<uint8_t*>(d_scratch);
    const int box = std::min(128, c->page_size & -c->page_size);
    // a scale of zero (the mean of the values) keeps a factor that is lost beside any score, so that a
    // masked score stays minus infinity
    const float c2 = std::max(std::fabs(scale) * 1.4426950408889634f, 1e-30f);
    const mk::AttnArgs a{*c, layer, rows, q_heads, q_heads / c->kv_heads, box, static_cast<const uint16_t*>(d_q), ldq,
                         static_cast<uint16_t*>(d_out), ldo, c2, scale < 0 ? 1 : 0,
                         mk::NewRows{d_seq_start, d_seqs, n}, reinterpret_cast<float*>(ws), reinterpret_cast<float2*>(ws + sc.ml),
                         reinterpret_cast<int*>(ws + sc.meta), max_rows};
    CUtensorMap tk, tv;
    if (!mk::page_map(&tk, *c, c->k, layer, box) || !mk::page_map(&tv, *c, c->v, layer, box))
      return refuse("the cache's strides cannot be described to the copy engine");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    e = c->head_dim == 256   ? mk::launch_attn<256>(tk, tv, a, grid, s)
        : c->head_dim == 128 ? mk::launch_attn<128>(tk, tv, a, grid, s)
                             : mk::launch_attn<64>(tk, tv, a, grid, s);
  }
  if (e == cudaSuccess) return MK_OK;
  mk_set_last_error(std::string("mk_paged_attention: ") + cudaGetErrorString(e));
  return MK_ERR_CUDA;
}
