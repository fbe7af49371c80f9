// Causal attention of new tokens over the pages of a KV cache.
//
// One warp per (row, query head): the query and the output stay in registers, D / 32 entries a
// lane, and the keys are walked once with a running maximum m and sum l:
//   z = scale q.k;  m' = max(m, z);  o = o e^(m - m') + e^(z - m') v;  l = l e^(m - m') + e^(z - m')
// Every row reads its keys and values again, so L2 bandwidth and the chain of warp sums bound it.
#include <algorithm>
#include <string>

#include "dev.cuh"
#include "mk_internal.h"
#include "mk_model.h"
#include "paged.h"

namespace mk {
namespace {

constexpr int kAttnThreads = 256;

struct AttnArgs {
  mk_paged_cache c;
  int layer, rows, hq;
  const uint16_t* q;
  long long ldq;
  uint16_t* o;
  long long ldo;
  float scale;
  NewRows w;
};

template <int E>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float* x) {
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p + i);
    x[i] = bf16lo(u), x[i + 1] = bf16hi(u);
  }
}

template <int D>
__global__ void __launch_bounds__(kAttnThreads) paged_attn_rows(const __grid_constant__ AttnArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long item = blockIdx.x * static_cast<long long>(kAttnThreads / 32) + (threadIdx.x >> 5);
  if (item >= static_cast<long long>(a.rows) * a.hq) return;
  const int r = static_cast<int>(item / a.hq), h = static_cast<int>(item % a.hq), g = h / (a.hq / a.c.kv_heads);
  if (r < a.w.start[0] || r >= a.w.start[a.w.n]) return;
  const int i = find_rows(a.w, r), s = a.w.seqs ? a.w.seqs[i] : i;
  int pos = -1;
  if (s >= 0 && s < a.c.n_seqs) pos = a.c.len[s] - a.w.start[i + 1] + r;
  else if (lane == 0) atomicOr(a.c.err, MK_DEVERR_BAD_PAGE);
  if (pos >= a.c.max_pages * a.c.page_size) {
    if (lane == 0) atomicOr(a.c.err, MK_DEVERR_BAD_PAGE);
    pos = -1;
  }
  float q[E], o[E], m = -INFINITY, l = 0.f;
  load_bf16<E>(a.q + r * a.ldq + h * D + lane * E, q);
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int p = 0; p <= pos; ++p) {
    const int page = a.c.table[static_cast<long long>(s) * a.c.max_pages + p / a.c.page_size];
    const bool ok = page >= 0 && page < a.c.n_pages;
    if (!ok && lane == 0) atomicOr(a.c.err, MK_DEVERR_BAD_PAGE);
    const long long at = a.layer * a.c.layer_stride + (ok ? page : 0) * a.c.page_stride + g * a.c.head_stride +
                         (p % a.c.page_size) * a.c.slot_stride + lane * E;
    float k[E], v[E], z = 0.f;
    load_bf16<E>(static_cast<const uint16_t*>(a.c.k) + at, k);
    load_bf16<E>(static_cast<const uint16_t*>(a.c.v) + at, v);
#pragma unroll
    for (int e = 0; e < E; ++e) z = fmaf(q[e], ok ? k[e] : 0.f, z);
    z = warp_sum(z) * a.scale;
    const float m2 = fmaxf(m, z), f = __expf(m - m2), w = __expf(z - m2);
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * (ok ? v[e] : 0.f);
    m = m2;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint16_t* dst = a.o + r * a.ldo + h * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) dst[e] = f_to_bf16(o[e] * inv);   // the one rounding of the result
}

template <int D>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t s) {
  const long long items = static_cast<long long>(a.rows) * a.hq;
  paged_attn_rows<D><<<static_cast<unsigned>((items + kAttnThreads / 32 - 1) / (kAttnThreads / 32)), kAttnThreads, 0, s>>>(a);
  return cudaGetLastError();
}

int refuse(const std::string& why) {
  mk_set_last_error("mk_paged_attention: " + why);
  return MK_ERR_ARG;
}

}  // namespace
}  // namespace mk

// ---------------------------------------------------------------- C ABI
extern "C" size_t mk_paged_attention_scratch(const mk_paged_cache* c, int32_t rows, int32_t q_heads) {
  if (mk::paged_cache_problem(c) || rows < 0 || q_heads < 1 || q_heads % c->kv_heads) return 0;
  return 256;
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
  if (rows == 0 || n == 0) return MK_OK;
  const int64_t dq = static_cast<int64_t>(q_heads) * c->head_dim;
  if (!d_q || !d_out || !d_seq_start || !d_scratch) return refuse("NULL pointer");
  if (ldq < dq || ldo < dq || ldq % 8 || ldo % 8) return refuse("row pitches must be multiples of 8 that hold the heads");
  if (!mk::aligned16(d_q) || !mk::aligned16(d_out) || !mk::aligned16(d_scratch)) return refuse("pointers must be 16-byte aligned");
  if (scratch_bytes < mk_paged_attention_scratch(c, rows, q_heads)) return refuse("scratch too small");
  const mk::AttnArgs a{*c,  layer, rows, q_heads, static_cast<const uint16_t*>(d_q), ldq, static_cast<uint16_t*>(d_out), ldo,
                       scale, mk::NewRows{d_seq_start, d_seqs, n}};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = c->head_dim == 256   ? mk::launch_rows<256>(a, s)
                        : c->head_dim == 128 ? mk::launch_rows<128>(a, s)
                                             : mk::launch_rows<64>(a, s);
  if (e == cudaSuccess) return MK_OK;
  mk_set_last_error(std::string("mk_paged_attention: ") + cudaGetErrorString(e));
  return MK_ERR_CUDA;
}
