// Entry point of the paged append (clo_paged_append).
#include <algorithm>

#include "clo_paged_append.cuh"

using namespace clo;

extern "C" CLO_API clo_status clo_paged_append(const clo_paged_cache* cache, const clo_paged_batch* batch, const clo_rope_plan* plan,
                                               const int64_t* positions, const clo_rows* k, const clo_rows* v, const clo_rows* q,
                                               const clo_rows* q_out, int32_t n_q_heads, void* stream) {
  const char* who = "clo_paged_append";
  AppendParams a{};
  if (const char* f = paged_params(cache, batch, &a.c)) return paged_fail(CLO_ERR_INVALID, "%s: %s", who, f);
  if (plan) {
    if (const char* f = plan_fault(plan, cache->head_dim)) return paged_fail(CLO_ERR_INVALID, "%s: %s", who, f);
    if (plan->rot_dim % 16) return paged_fail(CLO_ERR_INVALID, "%s: rot_dim must be a multiple of 16 (rotate with clo_rope and append without a plan)", who);
  }
  if (!q != !q_out) return paged_fail(CLO_ERR_INVALID, "%s: q and q_out come together", who);
  if (q && (n_q_heads < 1 || n_q_heads > 65535)) return paged_fail(CLO_ERR_INVALID, "%s: n_q_heads must be 1 .. 65535", who);
  if (q && !plan) return paged_fail(CLO_ERR_INVALID, "%s: q without a plan", who);
  if (reinterpret_cast<uintptr_t>(positions) & 7u) return paged_fail(CLO_ERR_INVALID, "%s: positions must be 8-byte aligned int64", who);
  if (batch->batch == 0 || batch->total_q == 0 || a.c.max_q == 0) return CLO_OK;
  for (const clo_rows* r : {k, v})
    if (const char* f = rows_fault(r, true)) return paged_fail(CLO_ERR_INVALID, "%s: k, v: %s", who, f);
  if (q)
    for (const clo_rows* r : {q, q_out})
      if (const char* f = rows_fault(r, true)) return paged_fail(CLO_ERR_INVALID, "%s: q, q_out: %s", who, f);
  if (q && q->ptr == q_out->ptr && (q->stride_token != q_out->stride_token || q->stride_head != q_out->stride_head))
    return paged_fail(CLO_ERR_INVALID, "%s: q and q_out may be the same rows only with the same strides", who);
  a.in[0] = rows_of(k);
  a.in[1] = rows_of(v);
  a.positions = positions;
  if (plan) a.rope.plan = *plan;
  // A sequence with n rows touches at most (n - 1) / page_size + 2 pages, and no more than n.
  const int64_t t = a.c.total_q;
  int64_t items = t / a.c.page_size + 2 * (int64_t)a.c.batch;
  if (items > t) items = t;
  a.items = (int32_t)items;
  // Warps per job: as many as hold the most rows that a page can get (a single token: one).
  const int rows = std::min(a.c.page_size, a.c.max_q), units = rows * (cache->head_dim / 16);
  const int per = units <= 32 * kUnits ? 1 : units <= 64 * kUnits ? 2 : units <= 128 * kUnits ? 4 : 8;
  const int64_t jobs = items * 2 * a.c.n_kv_heads;
  const int64_t kv_blocks = (jobs * per + kWarps - 1) / kWarps;
  int64_t q_blocks = 0;
  if (q) {
    const int heads = (per == 1 ? kShortIters : kLongIters) * 32 / (cache->head_dim / 16);  // per warp
    a.q = rows_of(q);
    a.q_out = rows_of(q_out);
    a.n_q_heads = n_q_heads;
    a.q_chunks = (n_q_heads + heads - 1) / heads;
    q_blocks = (t * a.q_chunks + kWarps - 1) / kWarps;
  }
  if (kv_blocks + q_blocks > 0x7fffffff) return paged_fail(CLO_ERR_INVALID, "%s: too many rows for one call", who);
  a.kv_blocks = (int32_t)kv_blocks;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t blocks = kv_blocks + q_blocks;
  (cache->kv_bits == 16 ? launch_append_bf16 : cache->kv_bits == 8 ? launch_append_e4m3 : launch_append_e2m1)(a, cache->head_dim, blocks, per, st);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return paged_fail(CLO_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return CLO_OK;
}

