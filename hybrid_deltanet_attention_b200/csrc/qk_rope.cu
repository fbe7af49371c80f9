// Per-head RMS norm of queries and keys, their rotation, and the append of keys and values to
// the pages of a cache, in one pass: every projection entry is read once and every result
// written once, so many rows are bound by HBM and one row by the latency of its dependent loads.
//
// One CTA per row, one warp per head: a lane holds head_dim / 32 consecutive entries, so loads
// and stores are one 8- to 32-byte vector a lane and the mean of squares is one warp sum. The
// rotation partner of entry i is entry i + rot_dim / 2, which lies 16 rot_dim / head_dim lanes on
// at the same place in the lane: one shuffle per entry. The row's angles are shared by
// all heads: position * theta^(-2i / rot_dim) in float64, reduced to [-pi, pi] there, sine and
// cosine in fp32, kept in shared memory.
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
  double log2_theta;
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
      const float4 t = *reinterpret_cast<const float4*>(p + i);
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

template <int D, typename T>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int E = D / 32;
  __shared__ float2 cs[D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.x;
  const bool paged = a.positions == nullptr;
  int pos;
  uint16_t *krow = nullptr, *vrow = nullptr;   // this row's slot of head 0
  bool ok = true;
  if (paged) {
    if (r < a.w.start[0] || r >= a.w.start[a.w.n]) return;   // the same for the whole CTA
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
    } else if (threadIdx.x == 0) {
      atomicOr(a.c.err, MK_DEVERR_BAD_PAGE);
    }
  } else {
    pos = a.positions[r];
  }
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    const double freq = exp2(-2.0 * i / a.rot * a.log2_theta);
    float c, s;
    rope_cs(pos * freq, c, s);
    cs[i] = make_float2(c, s);
  }
  __syncthreads();
  const int shift = half / E;                        // lanes between rotation partners
  const bool first = lane < shift, turn = lane < 2 * shift;
  const int partner = first ? lane + shift : turn ? lane - shift : lane;
  float co[E], si[E];                                // this lane's angles; the first half subtracts
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const float2 t = turn ? cs[(first ? lane : lane - shift) * E + j] : make_float2(1.f, 0.f);
    co[j] = t.x;
    si[j] = first ? -t.y : t.y;
  }
  const int heads = a.hq + a.hkv * (paged ? 2 : 1);
  for (int h = warp; h < heads; h += kRopeThreads / 32) {
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hkv;
    const int hh = is_q ? h : is_v ? h - a.hq - a.hkv : h - a.hq;
    const T* src = static_cast<const T*>(is_q ? a.q : is_v ? a.v : a.k) + r * (is_q ? a.ldq : is_v ? a.ldv : a.ldk) + hh * D;
    uint16_t* dst = is_q ? a.qo + r * a.ldqo + hh * D
                    : !paged ? a.ko + r * a.ldko + hh * D
                    : !ok ? nullptr
                          : (is_v ? vrow : krow) + hh * a.c.head_stride;
    if (!dst) continue;
    float x[E];
    load_row<E>(src + lane * E, x);
    if (!is_v) {
      const uint16_t* gain = is_q ? a.gq : a.gk;
      if (gain) {
        float g[E], ss = 0.f;
        load_row<E>(gain + lane * E, g);
#pragma unroll
        for (int j = 0; j < E; ++j) ss = fmaf(x[j], x[j], ss);
        const float inv = rsqrtf(warp_sum(ss) * (1.0f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] *= inv * g[j];
      }
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float y = __shfl_sync(0xFFFFFFFFu, x[j], partner);
        if (turn) x[j] = fmaf(x[j], co[j], y * si[j]);
      }
    }
    if (!ok) {
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = 0.f;
    }
    store_row<E>(dst + lane * E, x);
  }
}

template <int D>
cudaError_t launch_rope(const RopeArgs& a, bool f32, cudaStream_t s) {
  if (f32)
    qk_norm_rope_kernel<D, float><<<a.rows, kRopeThreads, 0, s>>>(a);
  else
    qk_norm_rope_kernel<D, uint16_t><<<a.rows, kRopeThreads, 0, s>>>(a);
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
  if (!(a->theta > 0) || !(a->eps >= 0)) return refuse("theta must be positive and eps not negative");
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
  r.log2_theta = std::log2(a->theta), r.eps = a->eps;
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
