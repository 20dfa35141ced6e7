// Attention over a paged cache (clo_paged_attention).
//
// out = sum_j p_j V_j, p = softmax of scale * q . K_j over the tokens that a row sees, in one pass with a running
// maximum and sum: for a new score s, m' = max(m, s), the sum and the accumulator shrink by 2^(m - m') and
// gain 2^(s - m') times 1 and V_j (scores in units of log2).
#include <cuda_runtime.h>

#include <cmath>

#include "clo.h"
#include "clo_paged.cuh"

namespace clo {
namespace {

constexpr int kThreads = 128;

// One row by one warp: lane i holds elements i * D / 32 and on.  Right for every input; no speed.
template <int D, int BITS>
__device__ void attend_row(const AttendParams& a, int b, const SeqRows& s, int row, int head, int lane) {
  constexpr int E = D / 32;
  const PagedParams& p = a.c;
  const int kvh = head / a.group, pos = s.pos0 + row;
  const int64_t t = s.first + row;
  const Visible v = visible_of(pos, s.kv_len, a.window, a.sinks);
  float q[E], acc[E], m = -INFINITY, l = 0.f;
  const uint16_t* qp = a.q + t * a.q_token + (int64_t)head * a.q_head;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = bf16_bits_to_f32(qp[lane * E + i]);
    acc[i] = 0.f;
  }
  auto value = [&](int side, int page, int slot, int e) {
    const PagedSide& sd = p.side[side];
    const int64_t at = (int64_t)page * sd.stride_page + (int64_t)kvh * sd.stride_head + (int64_t)slot * sd.stride_token + e;
    if (BITS == 16) return bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(sd.pages)[at]);
    return e4m3_to_f32x2(reinterpret_cast<const uint8_t*>(sd.pages)[at]).x *
           fmaxf(sd.scales[(int64_t)page * p.n_kv_heads + kvh], kMinScale);
  };
  int j = v.sink_end > 0 ? 0 : v.lo;
  for (; j < v.hi; j = j + 1 == v.sink_end ? v.lo : j + 1) {
    const int page = page_of(p, b, j >> p.page_shift);
    if (page < 0) continue;
    const int slot = j & (p.page_size - 1);
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) d = fmaf(q[i], value(0, page, slot, lane * E + i), d);
    const float sc = warp_sum(d) * a.scale_log2;
    const float mn = fmaxf(m, sc);
    const float keep = m == mn ? 1.f : exp2f(m - mn);
    const float w = mn == -INFINITY ? 0.f : exp2f(sc - mn);
    l = l * keep + w;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = acc[i] * keep + w * value(1, page, slot, lane * E + i);
    m = mn;
  }
  uint16_t* o = a.out + t * a.o_token + (int64_t)head * a.o_head;
#pragma unroll
  for (int i = 0; i < E; ++i) o[lane * E + i] = (uint16_t)pack_bf16(l == 0.f ? 0.f : acc[i] / l, 0.f);
}

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads) k_attend_rows(const AttendParams a) {
  const int lane = threadIdx.x & 31;
  const int64_t job = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = job / a.n_q_heads;
  if (t >= a.c.total_q) return;
  const int b = seq_of_row(a.c, (int)t, lane);
  if (b >= a.c.batch) return;
  const SeqRows s = seq_rows(a.c, b);
  if (t - s.first >= s.n) return;
  attend_row<D, BITS>(a, b, s, (int)(t - s.first), (int)(job % a.n_q_heads), lane);
}

}  // namespace

cudaError_t launch_paged_attention(const AttendParams& a, int head_dim, int kv_bits, cudaStream_t st) {
  const unsigned blocks = (unsigned)(((int64_t)a.c.total_q * a.n_q_heads + 3) / 4);
  if (head_dim == 128) {
    if (kv_bits == 16) k_attend_rows<128, 16><<<blocks, kThreads, 0, st>>>(a);
    else k_attend_rows<128, 8><<<blocks, kThreads, 0, st>>>(a);
  } else {
    if (kv_bits == 16) k_attend_rows<64, 16><<<blocks, kThreads, 0, st>>>(a);
    else k_attend_rows<64, 8><<<blocks, kThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace clo

using namespace clo;

extern "C" CLO_API clo_status clo_paged_attention(const clo_paged_cache* cache, const clo_paged_batch* batch, const clo_rows* q,
                                                  const clo_rows* out, int32_t n_q_heads, float softmax_scale, int32_t window,
                                                  int32_t sinks, void* stream) {
  const char* who = "clo_paged_attention";
  AttendParams a{};
  if (const char* f = paged_params(cache, batch, &a.c)) return paged_fail(CLO_ERR_INVALID, "%s: %s", who, f);
  const int hkv = cache->n_kv_heads;
  if (n_q_heads < 1 || n_q_heads % hkv || n_q_heads / hkv > kMaxGroup)
    return paged_fail(CLO_ERR_INVALID, "%s: n_q_heads must be a multiple of n_kv_heads, at most %d per kv head", who, kMaxGroup);
  if (window < 0 || sinks < 0) return paged_fail(CLO_ERR_INVALID, "%s: window and sinks must not be negative", who);
  if (!std::isfinite(softmax_scale) || softmax_scale < 0.f) return paged_fail(CLO_ERR_INVALID, "%s: softmax_scale must be >= 0", who);
  if (batch->batch == 0 || batch->total_q == 0 || a.c.max_q == 0) return CLO_OK;
  for (const clo_rows* r : {q, out}) {
    if (!r || !r->ptr) return paged_fail(CLO_ERR_INVALID, "%s: null pointer", who);
    if ((reinterpret_cast<uintptr_t>(r->ptr) & 15u) || r->stride_token % 8 || r->stride_head % 8)
      return paged_fail(CLO_ERR_INVALID, "%s: rows must lie on 16-byte boundaries (strides multiples of 8 elements)", who);
  }
  if (q->ptr == out->ptr) return paged_fail(CLO_ERR_INVALID, "%s: out must not overlap q", who);
  a.q = static_cast<const uint16_t*>(q->ptr);
  a.out = static_cast<uint16_t*>(out->ptr);
  a.q_token = q->stride_token;
  a.q_head = q->stride_head;
  a.o_token = out->stride_token;
  a.o_head = out->stride_head;
  a.n_q_heads = n_q_heads;
  a.group = n_q_heads / hkv;
  a.window = window;
  a.sinks = sinks;
  a.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt((float)cache->head_dim)) * 1.4426950408889634f;
  const cudaError_t e = launch_paged_attention(a, cache->head_dim, cache->kv_bits, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return paged_fail(CLO_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return CLO_OK;
}
