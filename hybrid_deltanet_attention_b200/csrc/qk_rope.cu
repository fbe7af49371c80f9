// Per-head RMS norm of queries and keys, their rotation, and the append of keys and values to
// the pages of a cache, in one pass: every projection entry is read once and every result
// written once, so many rows are bound by HBM and one row by the latency of its dependent loads.
//
// A warp takes up to 32 heads of one row, fewer (down to one) when there are too few rows to fill
// the GPU, and has the next head on its way while it works on one (4568 rows of 32 heads of 256: 43.5 us with up to 32
// heads a warp, 46 with 16, 50 with 8, 58 with 4; four blocks of 256 threads an SM). A lane holds head_dim / 32 consecutive entries, so
// loads and stores are one 8- to 32-byte vector a lane and the mean of squares is one warp sum. The
// rotation partner of entry i is entry i + rot_dim / 2, which lies 16 rot_dim / head_dim lanes on
// at the same place in the lane: one shuffle per entry. The angles of the row, position *
// theta^(-2i / rot_dim) in float64, reduced to half a turn there, sine and cosine in fp32, are
// computed once per warp while the first heads are on their way; two lanes that are partners share
// their angles, so each computes half of them (one float64 power, the others by the common ratio: at
// most three more roundings of 2^-53).
#include <algorithm>
#include <cmath>
#include <string>

#include "dev.cuh"
#include "mk_internal.h"
#include "mk_model.h"
#include "paged.h"

namespace mk {
namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
  int rows, hq, hkv, rot;
  int parts;               // warps that share a row's heads
  double log2_ratio, ratio;   // theta^(-2 / rot_dim)
  float eps;
  const void *q, *k, *v;
  long long ldq, ldk, ldv;
  const uint16_t *gq, *gk;
  uint16_t *qo, *ko;
  long long ldqo, ldko;
  const int* positions;
  int layer;
  NewRows w;
  mk_paged_cache c;
};

// E consecutive entries as fp32, E = 2, 4 or 8.
template <int E>
__device__ __forceinline__ void load_row(const float* p, float* x) {
  if constexpr (E == 2) {
    const float2 t = *reinterpret_cast<const float2*>(p);
    x[0] = t.x, x[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const float4 t = __ldcs(reinterpret_cast<const float4*>(p + i));
      x[i] = t.x, x[i + 1] = t.y, x[i + 2] = t.z, x[i + 3] = t.w;
    }
  }
}
template <int E>
__device__ __forceinline__ void load_row(const uint16_t* p, float* x) {
  uint32_t u[E / 2];
  if constexpr (E == 8) {
    const uint4 t = *reinterpret_cast<const uint4*>(p);
    u[0] = t.x, u[1] = t.y, u[2] = t.z, u[3] = t.w;
  } else if constexpr (E == 4) {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    u[0] = t.x, u[1] = t.y;
  } else {
    u[0] = *reinterpret_cast<const uint32_t*>(p);
  }
#pragma unroll
  for (int i = 0; i < E / 2; ++i) x[2 * i] = bf16lo(u[i]), x[2 * i + 1] = bf16hi(u[i]);
}
// The one rounding of a result: fp32 to bf16, ties to even (NaN and infinities kept).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int E>
__device__ __forceinline__ void store_row(uint16_t* p, const float* x) {
  uint32_t u[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) u[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
  if constexpr (E == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  else if constexpr (E == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = u[0];
}

constexpr double kLog2TwoPi = 2.6514961294723187980432933;

// Cosine and sine of pos * per turns: the whole turns are dropped in float64 (positions are large), so
// the fp32 functions see at most half a turn.
__device__ __forceinline__ void turn_cs(int pos, double per, float& c, float& s) {
  const double t = pos * per;
  sincospif(static_cast<float>(2.0 * (t - rint(t))), &s, &c);
}

constexpr int kHeads = 32;   // heads of a warp, at most

template <int D, typename T>
__global__ void __launch_bounds__(kRopeThreads, 4) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long task = blockIdx.x * static_cast<long long>(kRopeThreads / 32) + (threadIdx.x >> 5);
  const int r = static_cast<int>(task / a.parts), part = static_cast<int>(task - static_cast<long long>(r) * a.parts);
  if (r >= a.rows) return;
  const bool paged = a.positions == nullptr;
  const int heads = a.hq + a.hkv * (paged ? 2 : 1);
  const int h0 = static_cast<int>(static_cast<long long>(heads) * part / a.parts);
  const int h1 = static_cast<int>(static_cast<long long>(heads) * (part + 1) / a.parts);
  int pos;
  uint16_t *krow = nullptr, *vrow = nullptr;   // this row's slot of head 0
  bool ok = true;
  if (paged) {
    if (r < a.w.start[0] || r >= a.w.start[a.w.n]) return;   // the same for the whole warp
    const int i = find_rows(a.w, r), s = a.w.seqs ? a.w.seqs[i] : i;
    ok = s >= 0 && s < a.c.n_seqs;
    pos = ok ? a.c.len[s] - a.w.start[i + 1] + r : 0;
    ok = ok && pos >= 0 && pos < a.c.max_pages * a.c.page_size;
    const int page = ok ? a.c.table[static_cast<long long>(s) * a.c.max_pages + pos / a.c.page_size] : -1;
    ok = ok && page >= 0 && page < a.c.n_pages;
    if (ok) {
      const long long at = a.layer * a.c.layer_stride + page * a.c.page_stride + (pos % a.c.page_size) * a.c.slot_stride;
      krow = static_cast<uint16_t*>(a.c.k) + at;
      vrow = static_cast<uint16_t*>(a.c.v) + at;
    } else if (lane == 0) {
      atomicOr(a.c.err, MK_DEVERR_BAD_PAGE);
    }
  } else {
    pos = a.positions[r];
  }
  const int half = a.rot / 2, shift = half / E;      // entries and lanes between rotation partners
  const bool first = lane < shift, turn = lane < 2 * shift;
  const int partner = first ? lane + shift : turn ? lane - shift : lane;
  float co[E], si[E];                                // this lane's angles; the first half subtracts
  // the first lane of a pair computes its first E/2 angles, the second one the others
  double per = turn ? exp2(((first ? lane : lane - shift) * E + (first ? 0 : E / 2)) * a.log2_ratio - kLog2TwoPi) : 0.0;
#pragma unroll
  for (int j = 0; j < E / 2; ++j) {
    float c, s;
    turn_cs(pos, per, c, s);                         // lanes that do not turn: cosine 1, sine 0
    per *= a.ratio;
    const float oc = __shfl_sync(0xFFFFFFFFu, c, partner), os = __shfl_sync(0xFFFFFFFFu, s, partner);
    co[j] = first ? c : oc;
    co[j + E / 2] = first ? oc : c;
    si[j] = first ? -s : os;
    si[j + E / 2] = first ? -os : s;
  }
  // heads [i0, i1) of one kind (queries, keys, values), the next one on its way
  const bool whole = a.rot == D;
  auto work = [&](const void* from, long long ld, uint16_t* to, long long step, const uint16_t* gain, bool rotate, int i0, int i1) {
    if (i0 >= i1) return;
    const T* src = static_cast<const T*>(from) + r * ld + lane * E;
    float x[E], next[E], g[E];
    load_row<E>(src + i0 * D, next);
    if (gain) load_row<E>(gain + lane * E, g);
    to += lane * E;
    for (int i = i0; i < i1; ++i) {
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = next[j];
      if (i + 1 < i1) load_row<E>(src + (i + 1) * D, next);
      if (gain) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) ss = fmaf(x[j], x[j], ss);
        const float inv = rsqrtf(warp_sum(ss) * (1.0f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] *= inv * g[j];
      }
      if (rotate) {
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const float y = __shfl_sync(0xFFFFFFFFu, x[j], partner), z = fmaf(x[j], co[j], y * si[j]);
          x[j] = whole || turn ? z : x[j];
        }
      }
      if (!ok) {
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] = 0.f;
      }
      store_row<E>(to + i * step, x);
    }
  };
  const int hk = a.hq + a.hkv;
  work(a.q, a.ldq, a.qo + r * a.ldqo, D, a.gq, true, h0, min(h1, a.hq));
  if (!paged) {
    work(a.k, a.ldk, a.ko + r * a.ldko, D, a.gk, true, max(h0 - a.hq, 0), h1 - a.hq);
  } else if (ok) {
    work(a.k, a.ldk, krow, a.c.head_stride, a.gk, true, max(h0 - a.hq, 0), min(h1 - a.hq, a.hkv));
    work(a.v, a.ldv, vrow, a.c.head_stride, nullptr, false, max(h0 - hk, 0), h1 - hk);
  }
}

template <int D>
cudaError_t launch_rope(RopeArgs a, bool f32, cudaStream_t s) {
  const int heads = a.hq + a.hkv * (a.positions ? 1 : 2);
  int per = kHeads;   // heads of a warp, halved until the GPU has 16 warps per SM
  while (per > 1 && static_cast<long long>(a.rows) * ((heads + per - 1) / per) < 148 * 16) per /= 2;
  a.parts = (heads + per - 1) / per;
  const long long warps = static_cast<long long>(a.rows) * a.parts;
  const int grid = static_cast<int>((warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32));
  if (f32)
    qk_norm_rope_kernel<D, float><<<grid, kRopeThreads, 0, s>>>(a);
  else
    qk_norm_rope_kernel<D, uint16_t><<<grid, kRopeThreads, 0, s>>>(a);
  return cudaGetLastError();
}

int refuse(const std::string& why) {
  mk_set_last_error("mk_qk_norm_rope: " + why);
  return MK_ERR_ARG;
}

}  // namespace
}  // namespace mk

// ---------------------------------------------------------------- C ABI
extern "C" int mk_qk_norm_rope(const mk_qk_rope* a, void* stream) {
  using mk::aligned16;
  using mk::refuse;
  if (!a) return refuse("NULL arguments");
  if (a->dtype != MK_DT_F32 && a->dtype != MK_DT_BF16) return refuse("dtype must be MK_DT_F32 or MK_DT_BF16");
  if (!mk::head_dim_ok(a->head_dim)) return refuse("head_dim must be 64, 128 or 256");
  if (a->rows < 0 || a->q_heads < 1 || a->kv_heads < 1) return refuse("bad row or head count");
  if (a->rot_dim < 0 || a->rot_dim > a->head_dim || a->rot_dim % (a->head_dim / 16))
    return refuse("rot_dim must be a multiple of head_dim / 16, at most head_dim");
  if (!(a->theta > 0) || std::isinf(a->theta) || !(a->eps >= 0)) return refuse("theta must be positive and finite, eps not negative");
  const mk_paged_cache* c = a->cache;
  if (c) {
    if (const char* why = mk::paged_cache_problem(c)) return refuse(why);
    if (c->head_dim != a->head_dim || c->kv_heads != a->kv_heads) return refuse("the cache has other heads");
    if (a->layer < 0 || a->layer >= c->n_layers) return refuse("layer out of range");
    if (a->n < 0) return refuse("negative sequence count");
  }
  if (a->rows == 0 || (c && a->n == 0)) return MK_OK;
  const int64_t dq = static_cast<int64_t>(a->q_heads) * a->head_dim, dk = static_cast<int64_t>(a->kv_heads) * a->head_dim;
  if (!a->q || !a->k || !a->q_out || (c ? !a->v || !a->seq_start : !a->k_out || !a->positions)) return refuse("NULL pointer");
  if (a->ldq < dq || a->ldk < dk || a->ldq_out < dq || a->ldq % 8 || a->ldk % 8 || a->ldq_out % 8 ||
      (c ? a->ldv < dk || a->ldv % 8 : a->ldk_out < dk || a->ldk_out % 8))
    return refuse("row pitches must be multiples of 8 that hold the heads");
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->q_out) || (c ? !aligned16(a->v) : !aligned16(a->k_out)) ||
      !aligned16(a->q_gain) || !aligned16(a->k_gain))
    return refuse("pointers must be 16-byte aligned");
  mk::RopeArgs r{};
  r.rows = a->rows, r.hq = a->q_heads, r.hkv = a->kv_heads, r.rot = a->rot_dim;
  r.log2_ratio = a->rot_dim ? -2.0 / a->rot_dim * std::log2(a->theta) : 0.0, r.ratio = std::exp2(r.log2_ratio), r.eps = a->eps;
  r.q = a->q, r.k = a->k, r.v = a->v, r.ldq = a->ldq, r.ldk = a->ldk, r.ldv = a->ldv;
  r.gq = static_cast<const uint16_t*>(a->q_gain), r.gk = static_cast<const uint16_t*>(a->k_gain);
  r.qo = static_cast<uint16_t*>(a->q_out), r.ldqo = a->ldq_out;
  r.ko = static_cast<uint16_t*>(a->k_out), r.ldko = a->ldk_out;
  if (c) {
    r.layer = a->layer;
    r.w = mk::NewRows{a->seq_start, a->seqs, a->n};
    r.c = *c;
  } else {
    r.positions = a->positions;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = a->dtype == MK_DT_F32;
  const cudaError_t e = a->head_dim == 256   ? mk::launch_rope<256>(r, f32, s)
                        : a->head_dim == 128 ? mk::launch_rope<128>(r, f32, s)
                                             : mk::launch_rope<64>(r, f32, s);
  if (e == cudaSuccess) return MK_OK;
  mk_set_last_error(std::string("mk_qk_norm_rope: ") + cudaGetErrorString(e));
  return MK_ERR_CUDA;
}
