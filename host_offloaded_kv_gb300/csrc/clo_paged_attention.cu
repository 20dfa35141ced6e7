// Attention over a paged cache (clo_paged_attention).
//
// out = sum_j p_j V_j, p = softmax of scale * q . K_j over the tokens that a row sees, in one pass with a running
// maximum and sum: for a new score s, m' = max(m, s), the sum and the accumulator shrink by 2^(m - m') and
// gain 2^(s - m') times 1 and V_j (scores in units of log2).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "clo.h"
#include "clo_paged_attend.cuh"

namespace clo {
namespace {


using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once per process (a host function, the same for every device).
EncodeFn tensor_map_encoder() {
  static std::atomic<EncodeFn> fn{nullptr};
  EncodeFn f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    f = reinterpret_cast<EncodeFn>(p);
    fn.store(f, std::memory_order_release);
  }
  return f;
}

}  // namespace

cudaError_t prepare_kernel(const void* f, int smem, std::atomic<uint64_t>* prepared) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (prepared->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) prepared->fetch_or(bit, std::memory_order_release);
  return e;
}

const char* make_page_maps(const PagedParams& c, int head_dim, int kv_bits, int rows, PageMaps* maps) {
  EncodeFn encode = tensor_map_encoder();
  if (!encode) return "no tensor map encoder in the driver";
  const int bytes = kv_bits / 8, span = std::min(head_dim * bytes, 128);
  for (int s = 0; s < 2; ++s) {
    const PagedSide& sd = c.side[s];
    const cuuint64_t dims[4] = {(cuuint64_t)head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.n_kv_heads, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)sd.stride_token * bytes, (cuuint64_t)sd.stride_head * bytes, (cuuint64_t)sd.stride_page * bytes};
    const cuuint32_t box[4] = {(cuuint32_t)(span / bytes), (cuuint32_t)rows, 1, 1}, step[4] = {1, 1, 1, 1};
    const CUresult r = encode(&maps->side[s], bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, sd.pages, dims, strides,
                              box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, span == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return "the driver refused a tensor map of the pages";
  }
  return nullptr;
}

}  // namespace clo

using namespace clo;

// The kernels' view of a call, or what is wrong with it.
static const char* attend_params(const clo_paged_cache* cache, const clo_paged_batch* batch, int32_t n_q_heads, int32_t window, int32_t sinks,
                                 AttendParams* a) {
  if (const char* f = paged_params(cache, batch, &a->c)) return f;
  const int hkv = cache->n_kv_heads;
  if (n_q_heads < 1 || n_q_heads % hkv || n_q_heads / hkv > kMaxGroup) return "n_q_heads must be a multiple of n_kv_heads, at most 16 per kv head";
  if (window < 0 || sinks < 0) return "window and sinks must not be negative";
  a->n_q_heads = n_q_heads;
  a->group = n_q_heads / hkv;
  a->group_inv = (uint32_t)(((uint64_t(1) << 32) + a->group - 1) / a->group);
  a->window = window;
  a->sinks = sinks;
  const int64_t rows = (int64_t)a->c.max_q * a->group;
  if (rows >= int64_t(1) << 28) return "max_q times the heads per kv head must be below 2^28";
  a->part_rows = (int32_t)rows;
  return nullptr;
}

// Up to this many rows per kv head go to the decode kernel, more to the tcgen05 kernel.  (32 rows there, four fragments wide:
// 193 us for 132 at 16 sequences of 8 tokens by 4 heads over 8000 to 16,000 tokens of bf16, 178 for 123 with 8-bit pages.)
constexpr int kFewRows = 16;

extern "C" CLO_API clo_status clo_paged_attention_workspace(const clo_paged_cache* cache, const clo_paged_batch* batch, int32_t n_q_heads,
                                                            int32_t window, int32_t sinks, int64_t* bytes) {
  const char* who = "clo_paged_attention_workspace";
  AttendParams a{};
  if (!bytes) return paged_fail(CLO_ERR_INVALID, "%s: null pointer", who);
  *bytes = 0;
  if (const char* f = attend_params(cache, batch, n_q_heads, window, sinks, &a)) return paged_fail(CLO_ERR_INVALID, "%s: %s", who, f);
  if (a.c.batch == 0 || a.c.total_q == 0 || a.c.max_q == 0) return CLO_OK;
  if (a.part_rows > kFewRows)
    *bytes = attend_many_bytes(a, cache->head_dim);
  else
    *bytes = cache->kv_bits == 16 ? attend_few_bf16_bytes(a, cache->head_dim) : attend_few_e4m3_bytes(a, cache->head_dim);
  return CLO_OK;
}

extern "C" CLO_API clo_status clo_paged_attention(const clo_paged_cache* cache, const clo_paged_batch* batch, const clo_rows* q,
                                                  const clo_rows* out, int32_t n_q_heads, float softmax_scale, int32_t window,
                                                  int32_t sinks, void* workspace, int64_t workspace_bytes, void* stream) {
  const char* who = "clo_paged_attention";
  AttendParams a{};
  if (const char* f = attend_params(cache, batch, n_q_heads, window, sinks, &a)) return paged_fail(CLO_ERR_INVALID, "%s: %s", who, f);
  if (!std::isfinite(softmax_scale) || softmax_scale < 0.f) return paged_fail(CLO_ERR_INVALID, "%s: softmax_scale must be >= 0", who);
  if (workspace_bytes < 0 || (reinterpret_cast<uintptr_t>(workspace) & 15u))
    return paged_fail(CLO_ERR_INVALID, "%s: workspace must be 16-byte aligned, its size not negative", who);
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
  a.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt((float)cache->head_dim)) * 1.4426950408889634f;
  a.part = static_cast<float*>(workspace);
  a.part_bytes = workspace ? workspace_bytes : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.part_rows > kFewRows)
    e = launch_attend_many(a, cache->head_dim, cache->kv_bits, st);
  else
    e = cache->kv_bits == 16 ? launch_attend_few_bf16(a, cache->head_dim, st) : launch_attend_few_e4m3(a, cache->head_dim, st);
  if (e != cudaSuccess) return paged_fail(CLO_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return CLO_OK;
}
