// Causal attention of new tokens over the pages of a KV cache, on the sm_100a tensor cores.
//
// The query heads that share a kv head are packed: a row tile is 128 / group tokens times the group's
// heads (row r: token r / group, head kv_head * group + r % group), so one pass over the keys serves the whole
// group. A work unit is one row tile against one key tile of 128 keys. All units of a call,
// in the order sequence, kv head, row tile, key tile, are cut into one equal run per CTA (one CTA
// per SM), so a single long sequence spreads over the whole GPU and ragged ones balance; a row
// tile whose key range is cut leaves partial results (O, m, l), which a second kernel joins.
//
// Per key tile, with the scores in log2 units (c = |scale| log2 e, Q negated where the scale is):
//   S = Q K^T                         tcgen05, M = 128, N = 128, K = D, into TMEM
//   m = max(m, rowmax(c S));  P = 2^(c S - m), masked above the diagonal;  l += rowsum(P)
//   O = O + P V                       tcgen05, P (bf16) read from TMEM
// m is only raised (and O, l rescaled) when a tile's maximum passes it by more than 2^8, so
// weights are at most 2^8 and the result O / l is the same softmax. m, l, S, O and the partial results
// are fp32; a weight is rounded to bf16 once, as an operand, and the result once, at the end.
//
// Roles of the 12 warps: 0-7 softmax (two warps per 32 rows, each half of the tile's keys) and
// epilogue, 8 and 11 TMA producers (keys, values), 9 MMA issuer, 10 scheduler. Keys and values go through a ring of
// shared-memory slots (128 keys x min(D, 128) entries), filled by TMA boxes that follow the page table (a
// box is the largest power of two of slots that divides the page size, at most 128); the order
// K0 K1 V0 K2 V1 ... is the order of use, and it runs on across row tiles, so memory stays busy through
// softmax and epilogue. Values are taken as they lie in the page (transposed by the MMA descriptor).
//
// Measured on several B200s, per call: one token of each of 64 sequences (1.27 GB of keys and values) 203-222 us, 87-95 %
// of the measured copy bandwidth; a 4096-token prompt (8/2 heads of 256) 68-75 us, 920-1010 TFLOP/s of causal work, where
// shared memory bounds a tile (128 x 128 tiles at 256 entries move 320 KB through it, 2560 clocks; measured 3400);
// ragged chunks of 128-wide heads 72-78 us, bound by the chain of a group's softmax (about 3000 clocks a
// tile, two groups at work); one token over 32769 positions 25 us, of which the stream of 67 MB is half.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cuda.h>
#include <limits>
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
constexpr int kSoftRegs = 208, kOtherRegs = 88;
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
  // TMEM columns: O [0, D), then the score buffers of 128, whose first 64 columns take P. With three of
  // them (head dims up to 128) the scores run two tiles ahead of the products, so a softmax group finds
  // its next tile ready; 256 columns of O leave room for two. (P in columns of its own, so that scores could follow as
  // soon as the last ones are in registers, was slower: its writers wait for the product two tiles before.)
  static constexpr uint32_t kColS = D;
  static constexpr int kBufs = D == 256 ? 2 : 3, kAhead = kBufs - 1;
  // Places of the n key and value tiles of a segment in the ring: the scores of kAhead + 1 tiles, the
  // first product, and so on in turn, the last kAhead products at the end.
  __device__ static int k_place(int j, int) { return j <= kAhead ? j : 2 * j - kAhead; }
  __device__ static int v_place(int j, int n) { return j < n - kAhead ? 2 * j + kAhead + 1 : n + j; }
};
static_assert(Lay<256>::kSmem <= 232448 && Lay<128>::kSmem <= 232448, "fits the SM");

struct AttnArgs {
  mk_paged_cache c;
  int layer, rows, hq, group, box;
  const uint16_t* q;
  long long ldq;
  uint16_t* o;
  long long ldo;
  int tokens, few;         // of a row tile: 128 / group; of the smaller box of queries
  int over;                // key tiles that a full row tile's queries and results cost, beside one
  float c2;                // |scale| log2 e
  int negative;            // the sign of scale
  int deal;                // row tiles may stay whole (at most 32 sequences then)
  NewRows w;
  float* part;             // [2 * grid][max_rows][D]
  float2* ml;              // [2 * grid][max_rows] (m, l)
  int4* lead;              // [2 * grid]: what each CTA leads, see below
  int max_rows;
};
// The row tile whose first keys a CTA has and whose others it leaves to the next ones (its last segment, so one
// at most): {slot of its partial results, contributors (0: none), rows, row tile}, {kv head, the sequence's first
// row}. The other contributors are the next CTAs, each with its first slot.

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
};

struct Bars {
  uint64_t full[8], empty[8], s_full[3], p_full[3], o_done[2], mma_end, q_full, q_free, pair[4], m_full[2][4], seg_full[kSegs], seg_empty[kSegs];
  uint32_t tmem;
  int abort;
  Segment seg[kSegs];
  float m[2][kM], l[2][kM];   // [softmax group][row]
  int pages[2][2][16];        // [keys, values][tile parity][box]: page of each box of a tile
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
// Wait for the loads issued so far; v are the registers of one of them, used after the wait only.
__device__ __forceinline__ void tmem_wait_ld(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]),
                 "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]),
                 "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The MMAs are issued by a whole warp that stays converged, the instruction itself by its elected lane, so
// that descriptors live in uniform registers (one lane branching off costs more issue slots per
// MMA than the MMA takes). A descriptor is a constant high word and the address in the low one.
__device__ __forceinline__ bool elect_lane() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;   // groups of 8 rows 1024 bytes apart, version, 128-byte swizzle
constexpr uint32_t kLoK = 1u << 16;                   // K-major: leading offset unused
constexpr uint32_t kLoMN = (kPanel >> 4) << 16;       // MN-major: panels of 64 entries kPanel bytes apart
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate, uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(issue), "r"(kDescHi)
      : "memory");
}
// A from TMEM, bf16 pairs in 32-bit columns.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate, uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 b, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(issue), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t issue) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(issue)
      : "memory");
}
constexpr uint32_t kBMajorMN = 1u << 16, kNegateA = 1u << 13;   // instruction descriptor: B is MN-major; A negated

// One box of a 4-D tensor map.
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_box3(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// 32 bytes to a 32-byte aligned address in one store (a whole sector), or to a 16-byte aligned one in two.
__device__ __forceinline__ void store32(void* p, const uint32_t* u) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]),
                 "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    static_cast<uint4*>(p)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// a * b + c and a + b in both halves (packed fp32 instructions of sm_100).
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
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
// Wait for a phase; gives up after kWaitNs or when another role did. try_wait suspends the thread in
// hardware for a while by itself; the timer (a slow read) is looked at once in 64 attempts.
__device__ __forceinline__ bool wait_bar(Bars* b, uint64_t* bar, uint32_t parity, int* err) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !mbar_test(bar, parity); ++i) {
    if (i & 63) continue;
    const uint64_t t = global_ns();
    if (t0 == 0) t0 = t;
    const bool gone = *static_cast<volatile int*>(&b->abort);
    if (gone || t - t0 > kWaitNs) {
      if (!gone) atomicOr(err, MK_DEVERR_PIPE_TIMEOUT);
      *static_cast<volatile int*>(&b->abort) = 1;
      return false;
    }
  }
  return true;
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
  w.row_tiles = (w.rows + a.tokens - 1) / a.tokens;
  return w;
}
// Key tiles of row tile j: up to the position of its last row; one (empty) where it sees nothing.
__device__ __forceinline__ int key_tiles(const AttnArgs& a, const SeqWork& w, int j) {
  const int keys = w.pos0 + min((j + 1) * a.tokens, w.rows);
  return max(1, (keys + kN - 1) / kN);
}
// What row tile j costs beside its key tiles, in units of them (a.over + 1 for 128 rows, 1 for a few). Measured, cut, 256
// entries: a 4096-token prompt 79 us with 3 units, 81 with 2 and 80 with 4; 128 entries, ragged chunks: 68 us with 4, 69 with 3
// and 5.
__device__ __forceinline__ int extra_units(const AttnArgs& a, const SeqWork& w, int j) {
  return 1 + min(a.tokens, w.rows - j * a.tokens) * a.group * a.over / kM;
}
__device__ __forceinline__ SeqWork shfl_work(const SeqWork& w, int src) {
  return SeqWork{__shfl_sync(0xFFFFFFFFu, w.row0, src), __shfl_sync(0xFFFFFFFFu, w.rows, src), __shfl_sync(0xFFFFFFFFu, w.pos0, src),
                 __shfl_sync(0xFFFFFFFFu, w.len, src),  __shfl_sync(0xFFFFFFFFu, w.seq, src),  __shfl_sync(0xFFFFFFFFu, w.row_tiles, src)};
}
__device__ __forceinline__ long long warp_sum64(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// Units of one kv head of each lane's sequence: short ones by their lane, long ones by the warp.
__device__ long long head_units(const AttnArgs& a, const SeqWork& w) {
  const int lane = threadIdx.x & 31;
  long long u = 0;
  if (w.row_tiles <= 4)
    for (int j = 0; j < w.row_tiles; ++j) u += extra_units(a, w, j) + key_tiles(a, w, j);
  for (unsigned big = __ballot_sync(0xFFFFFFFFu, w.row_tiles > 4); big; big &= big - 1) {
    const int src = __ffs(big) - 1;
    const SeqWork x = shfl_work(w, src);
    long long sum = 0;
    for (int j = lane; j < x.row_tiles; j += 32) sum += extra_units(a, x, j) + key_tiles(a, x, j);
    sum = warp_sum64(sum);
    if (lane == src) u = sum;
  }
  return u;
}
__device__ __forceinline__ long long warp_scan64(long long v) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) >= o) v += y;
  }
  return v;
}

// Row tiles that stay whole. An even cut of the units costs each CTA about one more segment, two partial
// results and their join; where the row tiles themselves fill the CTAs evenly enough it is left out: the
// row tiles are put in the order of their key tiles and dealt to the CTAs there and back (CTA c takes ranks c,
// 2 ctas - 1 - c, 2 ctas + c, ...). Nothing is sorted: the key tiles of a sequence's row tiles do not fall, so
// how many of them have x or more is a formula, and a table of these sums finds the row tile of any rank.
// Taken where the longest share is at most kSlack units above the even one. Measured over prompts of 1 to 12
// sequences: with 2 to 5 units more 8 to 33 % faster (4096-token prompt, 8 heads of 256, 79 -> 66 us; three of 400
// tokens, 16 heads, 31 -> 25), with 6 and 7 more 0 to 13 %, with 8 and 9 more the same, 9 % slower for heads of 64, with
// 11 and more 3 to 17 % slower. Not looked at where it would cost more than it gives: row tiles of more than kMost
// key tiles, more than kRounds of them a CTA (the cuts weigh little), more than 32 sequences, and sequences of
// fewer than kM packed rows on average, whose partial results are small (decode of 32 sequences of 250
// positions 14 us cut, 18 whole).
constexpr int kMaxSeqs = 65536, kRounds = 8, kMost = 1024, kSlack = 7;
struct Whole {
  int4 seq[32][2];                               // pos0, rows, row tiles, row0; len, sequence
  int load, limit, most, tiles, maybe;
  Segment list[kRounds];
  int count[kMost];                              // row tiles with more than i key tiles
};
// Row tiles of one kv head of a sequence with x key tiles or more: its last ones.
__device__ __forceinline__ int tiles_from(int4 s, int tokens, int x) {
  const int y = (x - 1) * kN - s.x;              // the first y rows see fewer
  return x <= 1 || y < 0 ? s.z : y >= s.y ? 0 : s.z - y / tokens;
}
// Called by the whole CTA: its row tiles, in o->list, or -1 where the even cut is better. Not inlined: with its
// code inside, ragged chunks that do not take it were 2 us of 70 slower.
__device__ __noinline__ int plan_whole(const AttnArgs& a, Whole* o) {
  const int ctas = gridDim.x, tiles = o->tiles, most = o->most;
  for (int x = threadIdx.x; x < most; x += kThreads_) {
    int count = 0;
#pragma unroll 1
    for (int i = 0; i < a.w.n; ++i) count += tiles_from(o->seq[i][0], a.tokens, x + 1);
    o->count[x] = count * a.c.kv_heads;
  }
  __syncthreads();
  auto rank_of = [&](int k, int c) { return k * ctas + (k & 1 ? ctas - 1 - c : c); };
  auto size = [&](int rank) {                    // key tiles of the row tile of this rank
    int lo = 1, hi = most;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (o->count[mid - 1] > rank) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  int load = 0;
  for (int c = threadIdx.x; c < ctas; c += kThreads_) {
    int mine = 0;
#pragma unroll 1
    for (int k = 0; k * ctas < tiles; ++k)
      if (rank_of(k, c) < tiles) mine += size(rank_of(k, c)) + 1 + a.over;
    load = max(load, mine);
  }
  load = __reduce_max_sync(0xFFFFFFFFu, load);
  if ((threadIdx.x & 31) == 0) atomicMax(&o->load, load);
  __syncthreads();
  if (o->load > o->limit) return -1;
  int n = 0;
  const int k = static_cast<int>(threadIdx.x) - 10 * 32;   // the scheduler's lane, which reads the list
  while (n < kRounds && rank_of(n, blockIdx.x) < tiles) ++n;
  if (k >= 0 && k < n) {
    const int rank = rank_of(k, blockIdx.x), x = size(rank);
    int rel = rank - (x < most ? o->count[x] : 0);
#pragma unroll 1
    for (int i = 0; i < a.w.n; ++i) {
      const int4 q = o->seq[i][0], r = o->seq[i][1];
      const int above = tiles_from(q, a.tokens, x + 1), same = tiles_from(q, a.tokens, x) - above;
      if (rel < same * a.c.kv_heads) {
        o->list[k] = Segment{0, q.w, q.y, q.x, r.x, r.y, rel / same, q.z - above - 1 - rel % same, 0, x, -1};
        break;
      }
      rel -= same * a.c.kv_heads;
    }
  }
  return n;
}

template <int D>
__global__ void __launch_bounds__(kThreads_, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tq1, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                      const __grid_constant__ AttnArgs a) {
  using L = Lay<D>;
  extern __shared__ __align__(1024) uint8_t smem[];   // swizzled tiles need 1024-byte alignment
  uint8_t* ring = smem + L::kQ;
  Bars* b = reinterpret_cast<Bars*>(smem + L::kOffBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* err = a.c.err;
  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      a.lead[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
      atomicOr(err, MK_DEVERR_PIPE_TIMEOUT);
    }
    return;
  }

  if (threadIdx.x == 0) {
    b->abort = 0;
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(&b->full[i], 1);
      mbar_init(&b->empty[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&b->s_full[i], 1);
      mbar_init(&b->p_full[i], kSoftWarps / 2);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&b->o_done[i], 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&b->pair[i], 2);
      mbar_init(&b->m_full[0][i], 1);
      mbar_init(&b->m_full[1][i], 1);
    }
    mbar_init(&b->mma_end, 1);
    mbar_init(&b->q_full, 1);
    mbar_init(&b->q_free, 1);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&b->seg_full[i], 1);
      mbar_init(&b->seg_empty[i], kSoftWarps + 3);
    }
    fence_barrier_init();
  }
  if (warp == 8) {   // (TMEM may still be the kernel's before on this SM: then this waits for its end)
    if (lane == 0) {
      tc::prefetch_tensormap(&tq);
      tc::prefetch_tensormap(&tq1);
      tc::prefetch_tensormap(&tk);
      tc::prefetch_tensormap(&tv);
    }
    tc::tmem_alloc(&b->tmem, 512);
    tc::tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // what came before in the stream is complete
  // units of every group of 32 sequences, one warp per group (in the ring's memory, before its first use)
  long long* groups = reinterpret_cast<long long*>(ring);
  const int n_groups = (a.w.n + 31) / 32;
  SeqWork first{};           // the scheduler's warp keeps the first group
  long long first_units = 0;
  constexpr int kGroupBytes = kMaxSeqs / 32 * sizeof(long long);
  static_assert(kGroupBytes + sizeof(Whole) <= L::kSlots * L::kSlot, "fits the ring");
  Whole* order = reinterpret_cast<Whole*>(ring + kGroupBytes);
  for (int g = (warp + kThreads_ / 32 - 10) % (kThreads_ / 32); g < n_groups; g += kThreads_ / 32) {
    int bad = 0;
    const SeqWork w = seq_work(a, g * 32 + lane, &bad);
    const long long hu = head_units(a, w), u = warp_sum64(hu) * a.c.kv_heads;
    if (lane == 0) groups[g] = u;
    if (g == 0) first = w, first_units = hu;
    if (a.deal) {                                // one group
      const int tiles = static_cast<int>(min(warp_sum64(w.row_tiles) * a.c.kv_heads, 1ll << 30));
      const int mean = static_cast<int>(min(u, 1ll << 30)) / static_cast<int>(gridDim.x);
      const int most = __reduce_max_sync(0xFFFFFFFFu, w.row_tiles > 0 ? key_tiles(a, w, w.row_tiles - 1) : 0);
      order->seq[lane][0] = make_int4(w.pos0, w.rows, w.row_tiles, w.row0);
      order->seq[lane][1] = make_int4(w.len, w.seq, 0, 0);
      if (lane == 0) {
        order->load = 0, order->most = most, order->tiles = tiles, order->limit = mean + kSlack;
        order->maybe = tiles <= kRounds * static_cast<int>(gridDim.x) && most <= kMost &&
                       most + 1 + a.over <= mean + kSlack;
      }
    }
    if (bad && blockIdx.x == 0) atomicOr(err, MK_DEVERR_BAD_PAGE);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  int whole = -1;                                // row tiles of this CTA where all stay whole
  if (a.deal && order->maybe) whole = plan_whole(a, order);
  Segment planned{};                             // the scheduler's lane k: the k-th of them
  long long total = 0, before = 0, u0 = 0, u1 = 0;   // scheduler: all units, units before its group, its range
  int g = 0;
  if (warp == 10) {
    __syncwarp();
    if (lane < whole) planned = order->list[lane];
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
  __syncthreads();   // the ring is the producers' from here
  const uint32_t tmem = b->tmem;
  // registers: 256 x 208 + 128 x 88 = 384 x 168, what the CTA was launched with (checked by the host)
  if (warp >= kSoftWarps) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == 10) {
    // ---- scheduler: cut [u0, u1) into segments
    int emitted = 0, made = 0, with_queries = 0;
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
      if (s.end || s.len == 0) return;
      // its queries, once the last scores of the row tile before are computed: boxes of 64 entries x group heads x
      // tokens, which is the packed order (rows past the sequence are another's, or zeros, and are not used)
      if (with_queries && !(ok = warp_wait(b, &b->q_free, (with_queries - 1) & 1, err))) return;
      ++with_queries;
      if (elect_lane()) {
        // the smaller box where it holds all (decode): the whole one would be mostly other rows
        const bool few = s.new_rows - s.tile * a.tokens <= a.few;
        mbar_arrive_expect_tx(&b->q_full, (few ? a.few : a.tokens) * a.group * D * 2);
#pragma unroll
        for (int p = 0; p < D / 64; ++p)
          tma_box3(smem + p * kPanel, few ? &tq1 : &tq, p * 64, s.kvh * a.group, s.row0 + s.tile * a.tokens, &b->q_full);
      }
      __syncwarp();
    };
    if (lane == 0) a.lead[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    __syncwarp();
    long long u = u0;
    int taken = 0;
    if (whole >= 0) u = 0, u1 = 1, g = 0;          // one pass over the only group
    for (; u < u1 && ok && g < n_groups; ++g) {
      int bad = 0;
      const SeqWork mine = g ? seq_work(a, g * 32 + lane, &bad) : first;
      const long long hu = g ? head_units(a, mine) : first_units, units = hu * a.c.kv_heads;
      const long long incl = before + warp_scan64(units);
      while (ok && u < u1) {
        Segment s{};
        if (whole >= 0) {
          if (taken == whole) break;
          s.row0 = __shfl_sync(0xFFFFFFFFu, planned.row0, taken), s.new_rows = __shfl_sync(0xFFFFFFFFu, planned.new_rows, taken);
          s.pos0 = __shfl_sync(0xFFFFFFFFu, planned.pos0, taken), s.len = __shfl_sync(0xFFFFFFFFu, planned.len, taken);
          s.seq = __shfl_sync(0xFFFFFFFFu, planned.seq, taken), s.kvh = __shfl_sync(0xFFFFFFFFu, planned.kvh, taken);
          s.tile = __shfl_sync(0xFFFFFFFFu, planned.tile, taken), s.t1 = __shfl_sync(0xFFFFFFFFu, planned.t1, taken);
          s.part = -1;
          ++taken;
        } else {
          const unsigned past = __ballot_sync(0xFFFFFFFFu, incl > u);
          if (!past) break;
          const int src = __ffs(past) - 1;
          const SeqWork w = shfl_work(mine, src);
          const long long h = __shfl_sync(0xFFFFFFFFu, hu, src);
          const long long rel = u - __shfl_sync(0xFFFFFFFFu, incl - units, src);
          s.row0 = w.row0, s.new_rows = w.rows, s.pos0 = w.pos0, s.len = w.len, s.seq = w.seq;
          s.kvh = static_cast<int>(rel / h);
          long long rem = rel - s.kvh * h;           // units into this head
          int tiles = 0;
          for (int j0 = 0;; j0 += 32) {              // the row tile that holds unit rem of this head
            const int t = j0 + lane < w.row_tiles ? extra_units(a, w, j0 + lane) + key_tiles(a, w, j0 + lane) : 0;
            const long long inc = warp_scan64(t);
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
          // tiles counts the extra units and then the key tiles; a run that ends in the former leaves the
          // row tile to the next CTA
          const int over = extra_units(a, w, s.tile);
          const int upto = static_cast<int>(min(static_cast<long long>(tiles), rem + (u1 - u)));
          u += upto - rem;
          s.t0 = max(0, static_cast<int>(rem) - over);
          s.t1 = upto - over;
          if (s.t1 <= s.t0) continue;
          tiles -= over;
          const bool whole = s.t0 == 0 && s.t1 == tiles;
          s.part = whole ? -1 : static_cast<int>(blockIdx.x) * 2 + (made ? 1 : 0);
          ++made;
          if (!whole && s.t0 == 0 && lane == 0) {
            // the CTA whose run holds the row tile's last unit: the largest c with total c / ctas <= that unit
            const long long end = u + (tiles - s.t1), ctas = min(static_cast<long long>(gridDim.x), total);
            const int last = static_cast<int>((end * ctas + total - 1) / total) - 1;
            a.lead[2 * blockIdx.x] = make_int4(s.part, last - static_cast<int>(blockIdx.x) + 1,
                                               min(a.tokens, w.rows - s.tile * a.tokens) * a.group, s.tile);
            a.lead[2 * blockIdx.x + 1] = make_int4(s.kvh, s.row0, 0, 0);
          }
        }
        emit(s);
      }
      before = __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    Segment stop{};
    stop.end = 1;
    if (ok) emit(stop);
    if (!ok && with_queries && lane == 0) {        // queries in flight land before the CTA ends (bounded)
      int never = 0;
      mbar_wait(&b->q_full, (with_queries - 1) & 1, &never, kWaitNs / 10);
    }
    __syncwarp();
  } else if (warp == 8 || warp == 11) {
    // ---- TMA producers, of the keys and of the values. Lane i reads the page of box i of a tile two tiles
    // ahead of its use; one elected lane issues the loads (a load issued by each lane in turn cost
    // about 110 clocks a box).
    const bool is_v = warp == 11;
    const CUtensorMap* map = is_v ? &tv : &tk;
    const int per_tile = kN / a.box;
    uint32_t base = 0, last = 0;                   // ring slots before the segment; the last one filled, plus one
    bool ok = true;
    for (int i = 0; ok; ++i) {
      if (!(ok = warp_wait(b, &b->seg_full[i % kSegs], (i / kSegs) & 1, err))) break;
      const Segment s = b->seg[i % kSegs];
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->seg_empty[i % kSegs]);
      if (s.end) break;
      if (s.len == 0) continue;                    // nothing to read
      const int* row = a.c.table + static_cast<long long>(s.seq) * a.c.max_pages;
      const int n = s.t1 - s.t0;
      auto raw_page = [&](int tile) {
        const int p = tile * kN + lane * a.box;
        return tile < s.t1 && lane < per_tile && p < s.len ? row[p / a.c.page_size] : 0;
      };
      int now = raw_page(s.t0), next = raw_page(s.t0 + 1);
      for (int j = 0; j < n && ok; ++j) {
        const int t = s.t0 + j;
        const int after = raw_page(t + 2);
        if (now < 0 || now >= a.c.n_pages) {
          atomicOr(err, MK_DEVERR_BAD_PAGE);
          now = a.c.n_pages;                       // outside the tensor map: reads as zeros
        }
        const int boxes = min(per_tile, (s.len - t * kN + a.box - 1) / a.box);   // up to the sequence's end
        const int y0 = t * kN % a.c.page_size;                                   // a box never crosses a page
        int* pages = b->pages[is_v][j & 1];
        if (lane < per_tile) pages[lane] = now;
        __syncwarp();
        // the ring's releases come in the order of its slots too, and a producer is never more than kSlots
        // past its last wait, so no phase is skipped
        const uint32_t at = base + L::kCh * (is_v ? L::v_place(j, n) : L::k_place(j, n));
        for (int c = 0; c < L::kCh && ok; ++c) {
          const uint32_t slot = at + c, k = slot % L::kSlots;
          if (slot >= L::kSlots) ok = warp_wait(b, &b->empty[k], (slot / L::kSlots - 1) & 1, err);
          if (!ok) break;
          if (elect_lane()) {
            mbar_arrive_expect_tx(&b->full[k], boxes * a.box * L::kCW * 2);
            uint8_t* to = ring + k * L::kSlot;
            int y = y0;
            for (int i = 0; i < boxes; ++i, to += a.box * 128) {
              const int w = pages[i];
#pragma unroll
              for (int p = 0; p < L::kCW / 64; ++p) tma_box(to + p * kPanel, map, c * L::kCW + p * 64, y, s.kvh, w, &b->full[k]);
              y += a.box;
              if (y == a.c.page_size) y = 0;
            }
          }
          __syncwarp();
          last = slot + 1;
        }
        now = next;
        next = after;
      }
      base += 2u * L::kCh * n;
    }
    if (!ok && lane == 0) {                        // copies in flight land before the CTA ends (bounded)
      int never = 0;
      for (uint32_t i = last < L::kSlots ? 0u : last - L::kSlots; i < last; ++i)
        mbar_wait(&b->full[i % L::kSlots], (i / L::kSlots) & 1, &never, kWaitNs / 10);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---- MMA issuer (all lanes, one issues). Values are read as they lie in a slot: MN-major. The loops over
    // slots and panels stay loops: unrolled, this role's code made every role of its scheduler slower
    // (4096-token prompt of 256-wide heads 92 against 80 us).
    constexpr uint32_t id_o = tc::idesc_bf16_f32(kM, L::kCW) | kBMajorMN;
    const uint32_t id_s = tc::idesc_bf16_f32(kM, kN) | (a.negative ? kNegateA : 0u);   // the sign of the scale
    const uint32_t issue = elect_lane();
    const uint32_t q_lo = (smem_u32(smem) >> 4) | kLoK, ring_lo = smem_u32(ring) >> 4;
    uint32_t k = 0, phase = 0, it = 0, nq = 0;     // next ring slot and its phase
    bool ok = true;
    auto take = [&]() {                            // wait for the next slot in order
      ok = ok && warp_wait(b, &b->full[k], phase, err);
      tc::fence_after_sync();
      return ok;
    };
    auto pass = [&]() {                            // the slot is free once the MMAs so far are done
      commit(&b->empty[k], issue);
      if (++k == L::kSlots) k = 0, phase ^= 1;
    };
    uint32_t sbuf = 0, pbuf = 0, pphase = 0;       // score buffer of the next scores; of the next product, and its phase
    auto scores = [&] {                            // the buffer's P was consumed by a product issued before
      const uint32_t d = tmem + L::kColS + sbuf * kN;
#pragma unroll 1
      for (int c = 0; c < L::kCh; ++c) {
        if (!take()) return;
        const uint32_t b_lo = (ring_lo + k * (L::kSlot >> 4)) | kLoK;
#pragma unroll 1
        for (int p = 0; p < L::kCW / 64; ++p)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss(d, q_lo + ((c * (L::kCW / 64) + p) * kPanel + kk * 32) / 16, b_lo + (p * kPanel + kk * 32) / 16, id_s,
                   (c | p | kk) ? 1u : 0u, issue);
        pass();
      }
      commit(&b->s_full[sbuf], issue);
      sbuf = sbuf == L::kBufs - 1 ? 0 : sbuf + 1;
    };
    for (int i = 0; ok; ++i) {
      if (!(ok = warp_wait(b, &b->seg_full[i % kSegs], (i / kSegs) & 1, err))) break;
      const int len = b->seg[i % kSegs].len, n = b->seg[i % kSegs].t1 - b->seg[i % kSegs].t0, end = b->seg[i % kSegs].end;
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->seg_empty[i % kSegs]);
      if (end) break;
      if (len == 0) continue;
      if (!(ok = warp_wait(b, &b->q_full, nq++ & 1, err))) break;
      tc::fence_after_sync();
      for (int t = -L::kAhead; t < n && ok; ++t) {
        if (t + L::kAhead < n) {
          scores();
          if (t + L::kAhead == n - 1) commit(&b->q_free, issue);
        }
        if (t < 0) continue;
        if (!ok || !(ok = warp_wait(b, &b->p_full[pbuf], pphase, err))) break;
        const uint32_t pa = tmem + L::kColS + pbuf * kN, more = t > 0;
        if (++pbuf == L::kBufs) pbuf = 0, pphase ^= 1;
#pragma unroll 1
        for (int c = 0; c < L::kCh; ++c) {
          if (!take()) break;
          const uint32_t b_lo = (ring_lo + k * (L::kSlot >> 4)) | kLoMN;
#pragma unroll
          for (int kk = 0; kk < kN / 16; ++kk)
            mma_ts(tmem + c * L::kCW, pa + kk * 8, b_lo + kk * (2048 / 16), id_o, kk ? 1u : more, issue);
          pass();
        }
        if (ok) commit(&b->o_done[it & 1], issue);
        ++it;
      }
    }
    if (!ok) {                                     // products in flight end before TMEM is given back (bounded)
      int never = 0;
      commit(&b->mma_end, issue);
      if (lane == 0) mbar_wait(&b->mma_end, 0, &never, kWaitNs / 10);
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---- softmax and epilogue: thread = row r of the tile; the warps of group 0 take the even key
    // tiles of the CTA, those of group 1 the odd ones, so one group exponentiates while the other
    // loads the next scores and finds their maximum. m passes from tile to tile through shared
    // memory (published before the exponentials); each group keeps its own l.
    const int quarter = warp & 3, grp = warp >> 2, r = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t it = 0, slot = 0, meets = 0;
    Segment s;
    const int tok = r / a.group, head = r - tok * a.group;   // of this row in every row tile
    const int first_tok = quarter * 32 / a.group;            // of the warp's first row
    auto fetch = [&](int i) {
      if (!warp_wait(b, &b->seg_full[i % kSegs], (i / kSegs) & 1, err)) return false;
      s = b->seg[i % kSegs];
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->seg_empty[i % kSegs]);
      return true;
    };
    bool ok = fetch(0);
    for (int i = 0; ok && !s.end;) {
      const int tok0 = s.tile * a.tokens, rows = min(a.tokens, s.new_rows - tok0) * a.group;
      const bool live = quarter * 32 < rows;       // the warp has rows of the tile
      const int pos = s.pos0 + tok0 + tok, pos_first = s.pos0 + tok0 + first_tok;   // the row's, and the warp's lowest
      const int n = s.len == 0 ? 0 : s.t1 - s.t0;
      float l = 0.f, ml = -INFINITY;               // this group's sum, and the m (log2 units) it goes by
      for (int j = 0; j < n; ++j, ++it) {
        if ((it & 1) != static_cast<uint32_t>(grp)) continue;
        const int t = s.t0 + j;
        const uint32_t buf = it % L::kBufs, sb = tmem + lanes + L::kColS + buf * kN;
        // (of the tiles that had this buffer before, the last one's scores are complete: they were issued before
        // those of this group's last tile, so no phase is skipped)
        if (!(ok = warp_wait(b, &b->s_full[buf], (it / L::kBufs) & 1, err))) break;
        if (live) {
          tc::fence_after_sync();
          const int key0 = t * kN;
          const bool masked = key0 + kN - 1 > pos_first;
          // the row's 128 scores stay in registers: four loads in flight, and one pass for the maximum
          float x[kN];
#pragma unroll
          for (int c = 0; c < kN; c += 32) tmem_ld32(sb + c, x + c);
#pragma unroll
          for (int c = 0; c < kN; c += 32) tmem_wait_ld(x + c);
          if (masked) {
#pragma unroll
            for (int w = 0; w < kN / 32; ++w) {
              const int see = min(32, max(0, pos + 1 - key0 - 32 * w));   // visible columns of these 32
              const uint32_t bits = see >= 32 ? 0xFFFFFFFFu : (1u << see) - 1u;
#pragma unroll
              for (int c = 0; c < 32; ++c) x[32 * w + c] = bits >> c & 1 ? x[32 * w + c] : -INFINITY;
            }
          }
          float m0 = -INFINITY, m1 = m0, m2 = m0, m3 = m0;
#pragma unroll
          for (int c = 0; c < kN; c += 8) {
            m0 = max3(m0, x[c], x[c + 1]), m1 = max3(m1, x[c + 2], x[c + 3]);
            m2 = max3(m2, x[c + 4], x[c + 5]), m3 = max3(m3, x[c + 6], x[c + 7]);
          }
          const float top = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * a.c2;   // -inf where the row sees none
          float m = top;
          bool raise = false;
          if (j > 0) {
            if (!(ok = warp_wait(b, &b->m_full[grp ^ 1][quarter], ((it - 1) >> 1) & 1, err))) break;
            m = b->m[grp ^ 1][r];
            raise = r < rows && top > m + kRaise;
          }
          const float f = raise ? ex2(m - top) : 1.f;
          if (raise) m = top;
          b->m[grp][r] = m;
          __syncwarp();
          if (lane == 0) mbar_arrive(&b->m_full[grp][quarter]);
          if (__any_sync(0xFFFFFFFFu, raise)) {
            // the warp's rows of O are rescaled (factor 1 where the row keeps its m) once the
            // product before has completed
            if (!(ok = warp_wait(b, &b->o_done[grp ^ 1], ((it - 1) >> 1) & 1, err))) break;
            tc::fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tmem_ld32(tmem + lanes + c, o);
              tmem_wait_ld(o);
              uint32_t u[32];
#pragma unroll
              for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(o[k] * f);
              tmem_st32(tmem + lanes + c, u);
            }
            tmem_wait_st();
          }
          if (ml != m) l *= ex2(ml - m);           // m may have been raised at the other group's tile
          ml = m;
          const float sub = m == -INFINITY ? 0.f : -m;
          const uint64_t mul = f2_pack(a.c2, a.c2), add = f2_pack(sub, sub);
          uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
          for (int c = 0; c < kN; c += 32) {
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float2 u = f2_unpack(fma2(f2_pack(x[c + 2 * k], x[c + 2 * k + 1]), mul, add));
              const float2 w = f2_unpack(fma2(f2_pack(x[c + 2 * k + 2], x[c + 2 * k + 3]), mul, add));
              const float p0 = ex2(u.x), p1 = ex2(u.y), p2 = ex2(w.x), p3 = ex2(w.y);
              sum0 = add2(sum0, f2_pack(p0, p1));
              sum1 = add2(sum1, f2_pack(p2, p3));
              p[k] = pack_bf16(p0, p1);
              p[k + 1] = pack_bf16(p2, p3);
            }
            tmem_st16(sb + c / 2, p);              // over the scores, which have all been loaded
          }
          tmem_wait_st();
          l += f2_sum(add2(sum0, sum1));
        } else if (lane == 0) {
          mbar_arrive(&b->m_full[grp][quarter]);   // nothing to pass on, but the phases count tiles
        }
        if ((t + 1) * kN > s.len) {
          // positions from len on: whatever lies there must not meet a weight of zero as NaN
          const uint32_t at = slot + L::kCh * L::v_place(j, n);
          for (int c = 0; c < L::kCh && ok; ++c) {
            const uint32_t k = (at + c) % L::kSlots;
            ok = warp_wait(b, &b->full[k], ((at + c) / L::kSlots) & 1, err);
            if (!ok) break;
            const int first = s.len - t * kN;
            for (int v = threadIdx.x & 127; v < (kN - first) * (L::kCW / 8); v += 128) {
              const int row = first + v / (L::kCW / 8), e = v % (L::kCW / 8);
              *reinterpret_cast<uint4*>(ring + k * L::kSlot + (e >> 3) * kPanel + row * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
          }
          if (!ok) break;
          tc::fence_proxy_async_smem();
        }
        // this group's product before is done by now, but a parity wait must not skip a phase
        if (it >= 2 && !(ok = warp_wait(b, &b->o_done[grp], ((it >> 1) - 1) & 1, err))) break;
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->p_full[buf]);
      }
      if (!ok) break;
      slot += 2u * L::kCh * n;
      // output row and partial slot of this segment
      const int part = s.part;
      uint16_t* out = a.o + static_cast<long long>(s.row0 + tok0 + tok) * a.ldo + static_cast<long long>(s.kvh * a.group + head) * D;
      if (!(ok = fetch(++i))) break;
      float m = -INFINITY;
      if (n > 0) {
        // the last product and the one before it, in order: no phase is skipped
        if (n > 1 && !(ok = warp_wait(b, &b->o_done[it & 1], ((it - 2) >> 1) & 1, err))) break;
        if (!(ok = warp_wait(b, &b->o_done[(it - 1) & 1], ((it - 1) >> 1) & 1, err))) break;
        tc::fence_after_sync();
      }
      if (live) {
        if (n > 0) m = b->m[(it - 1) & 1][r];      // the last tile's
        if (ml != m) l *= ex2(ml - m);             // a group without a tile has l = 0 and ml = -inf
        b->l[grp][r] = l;
        if (!(ok = pair_sync(b, quarter, meets, err))) break;
        l += b->l[grp ^ 1][r];
        const float inv = l > 0.f ? 1.f / l : 0.f;   // a row that saw nothing takes exact zeros
#ifdef MK_TEST_SLOW_EPILOGUE_NS
        // a build for tests: the group that does not have the next tile reads O late
        if (grp != static_cast<int>(it & 1))
          for (const uint64_t t0 = global_ns(); global_ns() - t0 < MK_TEST_SLOW_EPILOGUE_NS;) __nanosleep(1000);
        __syncwarp();
#endif
        // half the columns each, every lane its row in whole sectors (transposing within 8 lanes, for 128-byte stores,
        // was no faster)
        float* dst = a.part + (static_cast<long long>(part) * a.max_rows + r) * D;
#pragma unroll 1
        for (int c = grp * (D / 2); c < (grp + 1) * (D / 2); c += 32) {
          float o[32];
          if (n > 0) {
            tmem_ld32(tmem + lanes + c, o);
            tmem_wait_ld(o);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0.f;
          }
          if (r < rows) {
            if (part < 0) {
              uint32_t u[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) u[k] = pack_bf16(o[2 * k] * inv, o[2 * k + 1] * inv);
              store32(out + c, u);
              store32(out + c + 16, u + 8);
            } else {
#pragma unroll
              for (int k = 0; k < 32; k += 8) store32(dst + c + k, reinterpret_cast<const uint32_t*>(o) + k);
            }
          }
        }
        if (part >= 0 && grp == 0 && r < rows) a.ml[static_cast<long long>(part) * a.max_rows + r] = make_float2(m, l);
        // The next row tile's first product overwrites O and waits for the weights of one group only, so
        // that group goes on once the other one has read its half (and l) too. (A barrier of its own that the MMA warp
        // waits on was slower: ragged chunks 78 against 74 us.)
        tc::fence_before_sync();
        if (!(ok = pair_sync(b, quarter, meets, err))) break;
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

// Joins the partial results of the row tiles whose keys were cut (a row tile has kJoinY blocks whatever its rows, so a few rows
// join in one round, and a full row tile over a long context in many, one after another): with M the largest m of the
// contributors, o = sum 2^(m - M) O / sum 2^(m - M) l. blockIdx.x is the leading CTA; a task is (up to) 128 columns of
// a row. Up to four contributors (a prompt's row tile is cut once or twice, and there are many rows) are
// read at once by one warp, for two tasks at a time; more (a long context's few rows have one contributor
// per CTA) are shared by the 8 warps of a block and joined in a fixed order.
constexpr int kJoinY = 8;
template <int D>
struct Joined {
  static constexpr int kCols = D < 128 ? D : 128, E = kCols / 32, kParts = D / kCols;
  float m = -INFINITY, l = 0.f, o[E] = {};
  int r, col;
  __device__ Joined(int task, int lane) : r(task / kParts), col(task % kParts * kCols + lane * E) {}
  // contributors k0, k0 + step, .. (four of them, below n)
  __device__ __forceinline__ void take(const AttnArgs& a, int cta, int lead, int k0, int step, int n) {
    float2 ml[4];
    float x[4][E];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + i * step;
      ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) x[i][e] = 0.f;
      if (k < n) {
        const long long at = static_cast<long long>(k ? 2 * (cta + k) : lead) * a.max_rows + r;
        ml[i] = a.ml[at];
        const float* src = a.part + at * D + col;
        if constexpr (E == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          x[i][0] = v.x, x[i][1] = v.y;
        }
      }
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = fmaxf(top, ml[i].x);
    const float base = top == -INFINITY ? 0.f : top;   // a row that sees nothing so far
    const float f = ex2(m - base);
    l *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float w = ex2(ml[i].x - base);
      l = fmaf(ml[i].y, w, l);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(x[i][e], w, o[e]);
    }
    m = top;
  }
  __device__ __forceinline__ void store(const AttnArgs& a, int tile, int kvh, int row0) const {
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int tr = r / a.group, tok = tile * a.tokens + tr, h = kvh * a.group + r - tr * a.group;
    uint32_t* out = reinterpret_cast<uint32_t*>(a.o + static_cast<long long>(row0 + tok) * a.ldo + static_cast<long long>(h) * D + col);
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
    else
      *out = pack_bf16(o[0] * inv, o[1] * inv);
  }
};
template <int D>
__global__ void __launch_bounds__(256) join_parts(const __grid_constant__ AttnArgs a) {
  using J = Joined<D>;
  constexpr int E = J::E;
  __shared__ float so[8][J::kCols];
  __shared__ float2 sm[8];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int cta = blockIdx.x;
  const int4 lead = a.lead[2 * cta], where = a.lead[2 * cta + 1];
  const int n = min(lead.y, static_cast<int>(gridDim.x) - cta), tasks = lead.z * J::kParts;
  if (n <= 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (n <= 4) {
    const int stride = gridDim.y * 8;
    for (int t = blockIdx.y * 8 + warp; t < tasks; t += 2 * stride) {
      J x(t, lane), y(min(t + stride, tasks - 1), lane);
      x.take(a, cta, lead.x, 0, 1, n);
      y.take(a, cta, lead.x, 0, 1, n);
      x.store(a, lead.w, where.x, where.y);
      if (t + stride < tasks) y.store(a, lead.w, where.x, where.y);
    }
    return;
  }
  for (int t = blockIdx.y; t < tasks; t += gridDim.y) {
    J x(t, lane);
    for (int k0 = warp; k0 < n; k0 += 32) x.take(a, cta, lead.x, k0, 8, n);
    if (lane == 0) sm[warp] = make_float2(x.m, x.l);
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = x.o[e];
    __syncthreads();
    if (warp == 0) {
      float top = -INFINITY;
      for (int k = 0; k < 8; ++k) top = fmaxf(top, sm[k].x);
      const float base = top == -INFINITY ? 0.f : top;
      x.l = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) x.o[e] = 0.f;
      for (int k = 0; k < 8; ++k) {
        const float f = ex2(sm[k].x - base);
        x.l = fmaf(sm[k].y, f, x.l);
#pragma unroll
        for (int e = 0; e < E; ++e) x.o[e] = fmaf(so[k][lane * E + e], f, x.o[e]);
      }
      x.store(a, lead.w, where.x, where.y);
    }
    __syncthreads();
  }
}

template <int D>
cudaError_t launch_attn(const CUtensorMap& tq, const CUtensorMap& tq1, const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, int grid, cudaStream_t s) {
  static std::atomic<uint64_t> attr_set{0};   // per device
  cudaError_t e = once_per_device(attr_set, [] {
    // the register split must fit what a CTA is launched with: a larger one would wait for ever
    cudaFuncAttributes f{};
    const cudaError_t got = cudaFuncGetAttributes(&f, paged_attn_kernel<D>);
    if (got != cudaSuccess) return got;
    if (f.numRegs * kThreads_ < kSoftWarps * 32 * kSoftRegs + (kThreads_ - kSoftWarps * 32) * kOtherRegs) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(paged_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kSmem);
  });
  if (e != cudaSuccess) return e;
  // both kernels come up while the one before them in the stream drains, and wait for it themselves
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads_);
  cfg.dynamicSmemBytes = Lay<D>::kSmem;
  e = cudaLaunchKernelEx(&cfg, paged_attn_kernel<D>, tq, tq1, tk, tv, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(grid, kJoinY);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_parts<D>, a);
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
  size_t part, ml, lead, total;
};
Scratch scratch_of(int grid, int max_rows, int d) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  Scratch s{};
  const size_t rows = 2ull * grid * max_rows;
  s.ml = up(rows * d * sizeof(float));
  s.lead = s.ml + up(rows * sizeof(float2));
  s.total = s.lead + up(2ull * grid * sizeof(int4));
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
  if (mk::paged_cache_problem(c) || rows < 0 || q_heads < 1 || q_heads % c->kv_heads || q_heads / c->kv_heads > mk::kM) return 0;
  return mk::scratch_of(mk::sm_count(), mk::max_rows_of(c, rows, q_heads), c->head_dim).total;
}

extern "C" int mk_paged_attention(const mk_paged_cache* c, int32_t layer, const void* d_q, int64_t ldq, int32_t rows,
                                  int32_t q_heads, const int32_t* d_seq_start, const int32_t* d_seqs, int32_t n, float scale,
                                  void* d_out, int64_t ldo, void* d_scratch, size_t scratch_bytes, void* stream) {
  using mk::refuse;
  if (const char* why = mk::paged_cache_problem(c)) return refuse(why);
  if (layer < 0 || layer >= c->n_layers) return refuse("layer out of range");
  if (rows < 0 || n < 0 || n > mk::kMaxSeqs) return refuse("rows must not be negative, n must lie in 0 .. 65536");
  if (q_heads < 1 || q_heads % c->kv_heads) return refuse("q_heads must be a positive multiple of kv_heads");
  if (!(std::fabs(scale) <= 2e38f)) return refuse("scale must lie within -2e38 .. 2e38");   // its log2 units are an fp32 factor
  if (q_heads / c->kv_heads > mk::kM) return refuse("at most 128 query heads per kv head");
  if (rows == 0 || n == 0) return MK_OK;
  const int64_t dq = static_cast<int64_t>(q_heads) * c->head_dim;
  if (!d_q || !d_out || !d_seq_start || !d_scratch) return refuse("NULL pointer");
  if (ldq < dq || ldo < dq || ldq % 8 || ldo % 8) return refuse("row pitches must be multiples of 8 that hold the heads");
  if (!mk::aligned16(d_q) || !mk::aligned16(d_out) || (reinterpret_cast<uintptr_t>(d_scratch) & 31))
    return refuse("d_q and d_out must be 16-byte, d_scratch 32-byte aligned");
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
    // A scale of zero (the mean of the values) becomes the smallest factor there is, so that a masked score stays
    // minus infinity: times any fp32 score it is below 2^-20.
    const float c2 = std::max(std::fabs(scale) * 1.4426950408889634f, std::numeric_limits<float>::denorm_min());
    const mk::AttnArgs a{*c, layer, rows, q_heads, q_heads / c->kv_heads, box, static_cast<const uint16_t*>(d_q), ldq,
                         static_cast<uint16_t*>(d_out), ldo, mk::kM / (q_heads / c->kv_heads),
                         std::min(mk::kM / (q_heads / c->kv_heads), (rows + n - 1) / n), c->head_dim == 256 ? 2 : c->head_dim == 128 ? 3 : 5, c2, scale < 0 ? 1 : 0,
                         n <= 32 && static_cast<int64_t>(rows) * (q_heads / c->kv_heads) >= static_cast<int64_t>(n) * mk::kM ? 1 : 0,
                         mk::NewRows{d_seq_start, d_seqs, n}, reinterpret_cast<float*>(ws), reinterpret_cast<float2*>(ws + sc.ml),
                         reinterpret_cast<int4*>(ws + sc.lead), max_rows};
    CUtensorMap tq, tq1, tk, tv;
    const uint64_t dims[3] = {static_cast<uint64_t>(c->head_dim), static_cast<uint64_t>(q_heads), static_cast<uint64_t>(rows)};
    const uint64_t strides[2] = {2ull * c->head_dim, 2ull * ldq};
    const uint32_t boxes[3] = {64, static_cast<uint32_t>(a.group), static_cast<uint32_t>(a.tokens)};
    const uint32_t boxes1[3] = {64, static_cast<uint32_t>(a.group), static_cast<uint32_t>(a.few)};
    if (!mk::tensor_map_bf16_nd(&tq, d_q, 3, dims, strides, boxes) || !mk::tensor_map_bf16_nd(&tq1, d_q, 3, dims, strides, boxes1))
      return refuse("the queries' pitch cannot be described to the copy engine");
    if (!mk::page_map(&tk, *c, c->k, layer, box) || !mk::page_map(&tv, *c, c->v, layer, box))
      return refuse("the cache's strides cannot be described to the copy engine");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    e = c->head_dim == 256   ? mk::launch_attn<256>(tq, tq1, tk, tv, a, grid, s)
        : c->head_dim == 128 ? mk::launch_attn<128>(tq, tq1, tk, tv, a, grid, s)
                             : mk::launch_attn<64>(tq, tq1, tk, tv, a, grid, s);
  }
  if (e == cudaSuccess) return MK_OK;
  mk_set_last_error(std::string("mk_paged_attention: ") + cudaGetErrorString(e));
  return MK_ERR_CUDA;
}
