// Rotary positions (clo_rope) and the read-back of pages (clo_paged_read): one pass over the rows each, bounded by HBM
// traffic (large calls) or by one launch and two or three dependent loads (single-token steps).
//
// Measured: 8192 tokens of 32 heads of 128, on one axis or three, 23.1 to 24.4 us, 5.5 to 5.8 TB/s (81 to 86 % of a copy's rate); 30,000 tokens
// 74 us, 97 %; one token 2.0 us in a graph.  Read-back of 8 x 8192 tokens: bf16 82 us, 6.5 TB/s, 8-bit pages 70 us, 5.8 TB/s; of 13,751 tokens of
// 4-bit pages 18.5 us, 3.9 TB/s.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <type_traits>

#include "clo.h"
#include "clo_rope.cuh"

namespace clo {

clo_status paged_fail(clo_status st, const char* fmt, ...) {
  char text[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof text, fmt, ap);
  va_end(ap);
  try {
    set_last_error_text(text);
  } catch (...) {  // out of host memory: the status alone
  }
  return st;
}

namespace {

template <int D, int ITERS, bool AXES>
__global__ void __launch_bounds__(kThreads, ITERS == kMidIters ? 3 : 4) k_rope(const Rope r, const Rows x, const Rows y, const int64_t* __restrict__ positions,
                                                   int64_t n_tokens, int n_heads, int chunks) {
  __shared__ __align__(16) uint64_t s_turn[kTurns<AXES>];
  stage_turns<AXES>(r, s_turn);
  const int64_t job = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = job / chunks;
  if (t >= n_tokens) return;
  auto position = [&](Place<AXES>* where) {
    *where = place_of<AXES>(r, positions, t, n_tokens, 0);
    return true;
  };
  rotate_heads<D, ITERS, AXES>(r, s_turn, x, y, t, position, (int)(job % chunks) * heads_per_warp<D>(ITERS), n_heads, threadIdx.x & 31);
}

// Any strides, alignment, rot_dim and head_dim: one pair, or one copied element, per thread and step.
// The angle is computed anew for every head: 8192 tokens of 32 heads of 96, 109 us, 0.9 TB/s.
__global__ void __launch_bounds__(kThreads) k_rope_any(const Rope r, const Rows x, const Rows y, const int64_t* __restrict__ positions,
                                                       int64_t n_tokens, int n_heads, int head_dim) {
  const int half = r.plan.rot_dim / 2, per_row = half + (head_dim - r.plan.rot_dim);
  const int64_t total = n_tokens * n_heads * per_row;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < total; e += (int64_t)gridDim.x * kThreads) {
    const int i = (int)(e % per_row);
    const int64_t row = e / per_row, t = row / n_heads, h = row % n_heads;
    const uint16_t* src = x.p + t * x.token + h * x.head;
    uint16_t* dst = y.p + t * y.token + h * y.head;
    if (i >= half) {
      dst[r.plan.rot_dim + i - half] = src[r.plan.rot_dim + i - half];
      continue;
    }
    const int a = r.plan.interleaved ? 2 * i : i, b = r.plan.interleaved ? 2 * i + 1 : i + half;
    const int64_t at = r.plan.n_axes > 1 ? r.plan.axis[i] * n_tokens + t : t;
    float2 c = rope_cos_sin(positions[at], r.plan.turn[i], r.plan.magnitude);
    if (r.transpose) c.y = -c.y;
    const float p = bf16_bits_to_f32(src[a]), q = bf16_bits_to_f32(src[b]);
    dst[a] = (uint16_t)pack_bf16(fmaf(p, c.x, -q * c.y), 0.f);
    dst[b] = (uint16_t)pack_bf16(fmaf(q, c.x, p * c.y), 0.f);
  }
}

// ---------------------------------------------------------------------------- read-back
struct ReadParams {
  PagedParams c;
  Rows out[2];
};

// A warp per row of the batch, K then V; 8 elements per lane and step.
template <int D, int BITS>
__global__ void __launch_bounds__(kThreads) k_paged_read(const ReadParams a) {
  const PagedParams& p = a.c;
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= p.total_q) return;
  const int b = seq_of_row(p, (int)t, lane);
  if (b >= p.batch) return;
  const SeqRows s = seq_rows(p, b);
  if (t - s.first >= s.n) return;
  const int64_t pos = (int64_t)s.pos0 + (t - s.first);
  const int page = pos < 0 || pos >= kMaxPagedTokens ? -1 : page_of(p, b, (int)(pos >> p.page_shift));
  const int slot = (int)(pos & (p.page_size - 1));
  constexpr int kVecs = D / 8;
  const int n = p.n_kv_heads * kVecs;
  constexpr int kBatch = 8;  // loads in flight per lane
  for (int v0 = lane; v0 < 2 * n; v0 += 32 * kBatch) {
    uint4 w[kBatch];
    float scale[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int v = v0 + 32 * i;
      const bool second = v >= n;
      const PagedSide& sd = p.side[second];
      const int h = (second ? v - n : v) / kVecs, e = v % kVecs * 8;
      w[i] = make_uint4(0, 0, 0, 0);
      scale[i] = 1.f;
      if (v < 2 * n && page >= 0) {
        const char* src = sd.pages + ((int64_t)page * sd.stride_page + (int64_t)h * sd.stride_head + (int64_t)slot * sd.stride_token + e) * (BITS / 8);
        if (BITS == 16) {
          w[i] = __ldg(reinterpret_cast<const uint4*>(src));
        } else {
          const uint2 c = __ldg(reinterpret_cast<const uint2*>(src));
          w[i].x = c.x;
          w[i].y = c.y;
          scale[i] = __ldg(sd.scales + (int64_t)page * p.n_kv_heads + h);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int v = v0 + 32 * i;
      if (v >= 2 * n) break;
      const bool second = v >= n;
      const Rows& out = a.out[second];
      const int h = (second ? v - n : v) / kVecs, e = v % kVecs * 8;
      if (BITS == 8) {
        const float f = fmaxf(scale[i], kMinScale);
        float x[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 d = e4m3_to_f32x2(((k < 2 ? w[i].x : w[i].y) >> (16 * (k & 1))) & 0xffffu);
          x[2 * k] = d.x * f;
          x[2 * k + 1] = d.y * f;
        }
        w[i] = pack8(x);
      }
      *reinterpret_cast<uint4*>(out.p + t * out.token + (int64_t)h * out.head + e) = w[i];
    }
  }
}

// 4-bit pages: a group of 16 elements per lane and step.
template <int D>
__global__ void __launch_bounds__(kThreads) k_paged_read4(const ReadParams a) {
  const PagedParams& p = a.c;
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= p.total_q) return;
  const int b = seq_of_row(p, (int)t, lane);
  if (b >= p.batch) return;
  const SeqRows s = seq_rows(p, b);
  if (t - s.first >= s.n) return;
  const int64_t pos = (int64_t)s.pos0 + (t - s.first);
  const int page = pos < 0 || pos >= kMaxPagedTokens ? -1 : page_of(p, b, (int)(pos >> p.page_shift));
  const int slot = (int)(pos & (p.page_size - 1));
  constexpr int kGroups = D / 16, kBatch = 4;
  const int n = p.n_kv_heads * kGroups;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const PagedSide& sd = p.side[side];
    const Rows& out = a.out[side];
    for (int v0 = lane; v0 < n; v0 += 32 * kBatch) {
      uint2 w[kBatch];
      uint32_t group[kBatch];
      float scale[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int v = v0 + 32 * i, h = v / kGroups, g = v % kGroups;
        w[i] = make_uint2(0u, 0u);
        group[i] = 0u;
        scale[i] = 1.f;
        if (v < n && page >= 0) {
          w[i] = __ldg(reinterpret_cast<const uint2*>(sd.pages + ((int64_t)page * sd.stride_page + (int64_t)h * sd.stride_head + (int64_t)slot * sd.stride_token + g * 16) / 2));
          group[i] = __ldg(sd.groups + groups_at<D>(p, page, h, slot) + g);
          scale[i] = __ldg(sd.scales + (int64_t)page * p.n_kv_heads + h);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int v = v0 + 32 * i, h = v / kGroups, g = v % kGroups;
        if (v >= n) break;
        // a code times its group's scale is exact and below 2^12; the page's scale comes last, as group scale times page scale may pass fp32's
        // range where the code is zero or a half.  Powers of two leave the product exact, other scales round it to fp32.
        const float f = e4m3_to_f32x2(group[i]).x, page_scale = fmaxf(scale[i], kMinScale);
        uint16_t* dst = out.p + t * out.token + (int64_t)h * out.head + g * 16;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t c[4];
          e2m1_to_f16x8(half ? w[i].y : w[i].x, c);
          float x[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&c[k]));
            x[2 * k] = d.x * f * page_scale;
            x[2 * k + 1] = d.y * f * page_scale;
          }
          *reinterpret_cast<uint4*>(dst + 8 * half) = pack8(x);
        }
      }
    }
  }
}

}  // namespace

// Checks a cache and a batch and fills the kernels' view of them; null or what is wrong.
const char* paged_params(const clo_paged_cache* c, const clo_paged_batch* b, PagedParams* p) {
  if (!c || !b) return "null pointer";
  if (!c->k_pages || !c->v_pages) return "null pages";
  if (c->head_dim != 64 && c->head_dim != 128) return "head_dim must be 64 or 128";
  if (c->kv_bits != 16 && c->kv_bits != 8 && c->kv_bits != 4) return "kv_bits must be 16, 8 or 4";
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return "page_size must be 16, 32, 64 or 128";
  if (c->n_kv_heads < 1 || c->n_kv_heads > 65535) return "n_kv_heads must be 1 .. 65535";
  if (c->n_pages < 1 || c->n_pages > 0x7fffffff) return "n_pages must be 1 .. 2^31 - 1";
  const int64_t per16 = 128 / c->kv_bits;
  const int64_t strides[6] = {c->k_stride_page, c->k_stride_head, c->k_stride_token, c->v_stride_page, c->v_stride_head, c->v_stride_token};
  for (int64_t s : strides)
    if (s <= 0 || s % per16 || s >= (int64_t(8) << 40) / c->kv_bits) return "page strides must be positive multiples of 16 bytes, below 2^40 bytes";
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return "pages must be 16-byte aligned";
  if (c->kv_bits != 16 && (!c->k_scales || !c->v_scales || (reinterpret_cast<uintptr_t>(c->k_scales) & 3u) || (reinterpret_cast<uintptr_t>(c->v_scales) & 3u)))
    return "8-bit and 4-bit pages need 4-byte aligned scales";
  if (c->kv_bits == 4 && (!c->k_group_scales || !c->v_group_scales || !aligned16(c->k_group_scales) || !aligned16(c->v_group_scales)))
    return "4-bit pages need 16-byte aligned group scales";
  if (b->batch < 0 || b->batch > 65535) return "batch must be 0 .. 65535";
  if (b->total_q < 0 || b->total_q > kMaxPagedTokens || b->max_q < 0) return "total_q must be 0 .. 2^30, max_q not negative";
  if (b->max_pages < 0 || (int64_t)b->max_pages * c->page_size >= kMaxPagedTokens) return "max_pages * page_size must be below 2^30";
  if (b->batch > 0 && b->total_q > 0) {
    if (!b->q_starts || !b->kv_lens || (!b->block_table && b->max_pages > 0)) return "null pointer in the batch";
    if ((reinterpret_cast<uintptr_t>(b->q_starts) | reinterpret_cast<uintptr_t>(b->kv_lens) | reinterpret_cast<uintptr_t>(b->block_table)) & 3u)
      return "the batch's arrays must be 4-byte aligned";
  }
  // (callers of other pages may have been compiled before the struct had these fields)
  void* const groups[2] = {c->kv_bits == 4 ? c->k_group_scales : nullptr, c->kv_bits == 4 ? c->v_group_scales : nullptr};
  p->side[0] = PagedSide{static_cast<char*>(c->k_pages), c->k_scales, static_cast<uint8_t*>(groups[0]), c->k_stride_page, c->k_stride_head, c->k_stride_token};
  p->side[1] = PagedSide{static_cast<char*>(c->v_pages), c->v_scales, static_cast<uint8_t*>(groups[1]), c->v_stride_page, c->v_stride_head, c->v_stride_token};
  p->q_starts = b->q_starts;
  p->kv_lens = b->kv_lens;
  p->table = b->block_table;
  p->table_stride = b->table_stride;
  p->n_pages = (int32_t)c->n_pages;
  p->max_pages = b->max_pages;
  p->batch = b->batch;
  p->total_q = b->total_q;
  p->max_q = b->max_q < b->total_q ? b->max_q : b->total_q;
  p->n_kv_heads = c->n_kv_heads;
  p->page_size = c->page_size;
  p->page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  return nullptr;
}

}  // namespace clo

using namespace clo;

extern "C" CLO_API void clo_rope_config_default(clo_rope_config* cfg) {
  if (!cfg) return;
  memset(cfg, 0, sizeof *cfg);
  cfg->theta = 10000.0;
  cfg->factor = 1.0;
  cfg->low_freq = 1.0;
  cfg->high_freq = 4.0;
  cfg->beta_fast = 32.0;
  cfg->beta_slow = 1.0;
}

extern "C" CLO_API clo_status clo_rope_plan_init(const clo_rope_config* c, clo_rope_plan* plan) {
  const char* who = "clo_rope_plan_init";
  if (!c || !plan) return paged_fail(CLO_ERR_INVALID, "%s: null pointer", who);
  const int rot = c->rot_dim;
  if (rot < 2 || rot % 2 || rot > 2 * CLO_ROPE_MAX_PAIRS)
    return paged_fail(CLO_ERR_INVALID, "%s: rot_dim must be even, 2 .. %d", who, 2 * CLO_ROPE_MAX_PAIRS);
  if (!(c->theta > 1.0) || !std::isfinite(c->theta)) return paged_fail(CLO_ERR_INVALID, "%s: theta must be > 1", who);
  if (c->scaling < CLO_ROPE_NONE || c->scaling > CLO_ROPE_YARN) return paged_fail(CLO_ERR_INVALID, "%s: unknown scaling %d", who, c->scaling);
  if (!(c->factor >= 1.0) || !std::isfinite(c->factor)) return paged_fail(CLO_ERR_INVALID, "%s: factor must be >= 1", who);
  if (!(c->magnitude >= 0.0) || !std::isfinite(c->magnitude)) return paged_fail(CLO_ERR_INVALID, "%s: magnitude must be >= 0", who);
  if (c->scaling >= CLO_ROPE_BANDS && c->original_max < 1)
    return paged_fail(CLO_ERR_INVALID, "%s: original_max must be >= 1 for this scaling", who);
  if (c->scaling == CLO_ROPE_BANDS && !(c->low_freq < c->high_freq && std::isfinite(c->low_freq) && std::isfinite(c->high_freq)))
    return paged_fail(CLO_ERR_INVALID, "%s: need low_freq < high_freq", who);
  if (c->scaling == CLO_ROPE_YARN && !(c->beta_slow > 0.0 && c->beta_fast > c->beta_slow && std::isfinite(c->beta_fast)))
    return paged_fail(CLO_ERR_INVALID, "%s: need beta_fast > beta_slow > 0", who);
  if (c->n_axes < 0 || c->n_axes > CLO_ROPE_MAX_AXES) return paged_fail(CLO_ERR_INVALID, "%s: n_axes must be 0 .. %d", who, CLO_ROPE_MAX_AXES);
  const int axes = c->n_axes > 1 ? c->n_axes : 1;
  if (axes > 1) {
    int64_t sum = 0;
    for (int a = 0; a < axes; ++a) {
      if (c->axis_pairs[a] < 1) return paged_fail(CLO_ERR_INVALID, "%s: axis_pairs must be 1 or more for each axis", who);
      sum += c->axis_pairs[a];
    }
    if (sum != rot / 2) return paged_fail(CLO_ERR_INVALID, "%s: axis_pairs must add up to rot_dim / 2", who);
    if (c->axis_order != CLO_ROPE_SECTIONS && c->axis_order != CLO_ROPE_CYCLED)
      return paged_fail(CLO_ERR_INVALID, "%s: unknown axis_order %d", who, c->axis_order);
  }
  const double two_pi = 6.283185307179586476925;
  memset(plan, 0, sizeof *plan);
  int used[CLO_ROPE_MAX_AXES] = {0, 0, 0, 0}, turn = 0;
  for (int p = 0; p < rot / 2; ++p) {
    int axis = 0;
    if (axes > 1 && c->axis_order == CLO_ROPE_SECTIONS) {
      while (used[axis] == c->axis_pairs[axis]) ++axis;
    } else if (axes > 1) {
      while (used[turn % axes] == c->axis_pairs[turn % axes]) ++turn;
      axis = turn++ % axes;
    }
    // the pair's index, and the dimensions that its series runs over
    const bool own = axes > 1 && c->axis_own_freqs != 0;
    const int i = own ? used[axis] : p, n = own ? 2 * c->axis_pairs[axis] : rot;
    ++used[axis];
    plan->axis[p] = (uint8_t)axis;
    double f = std::pow(c->theta, -2.0 * i / n);
    double keep = 1.0;  // share of the unscaled frequency
    if (c->scaling == CLO_ROPE_LINEAR) keep = 0.0;
    if (c->scaling == CLO_ROPE_BANDS) keep = ((double)c->original_max * f / two_pi - c->low_freq) / (c->high_freq - c->low_freq);
    if (c->scaling == CLO_ROPE_YARN) {
      auto pair_of = [&](double turns) { return n * std::log((double)c->original_max / (turns * two_pi)) / (2.0 * std::log(c->theta)); };
      const double lo = std::fmax(0.0, std::floor(pair_of(c->beta_fast))), hi = std::fmin(n - 1.0, std::ceil(pair_of(c->beta_slow)));
      keep = 1.0 - std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 1e-3)));
    }
    keep = std::fmin(1.0, std::fmax(0.0, keep));
    f = keep * f + (1.0 - keep) * f / c->factor;
    // f <= 1 radian per position, so the fraction of a turn is below 1/6
    plan->turn[p] = (uint64_t)std::llrint(std::ldexp(f / two_pi, 62)) << 2;
  }
  plan->magnitude = c->magnitude > 0.0 ? (float)c->magnitude
                    : c->scaling == CLO_ROPE_YARN ? (float)(0.1 * std::log(c->factor) + 1.0) : 1.f;
  plan->rot_dim = rot;
  plan->interleaved = c->interleaved != 0;
  plan->n_axes = axes;
  plan->ready = 1;
  return CLO_OK;
}

const char* clo::plan_fault(const clo_rope_plan* p, int head_dim) {
  if (!p) return "null plan";
  if (p->ready != 1 || p->rot_dim < 2 || p->rot_dim % 2 || p->rot_dim > 2 * CLO_ROPE_MAX_PAIRS || p->n_axes < 1 || p->n_axes > CLO_ROPE_MAX_AXES)
    return "plan not set by clo_rope_plan_init";
  for (int i = 0; p->n_axes > 1 && i < p->rot_dim / 2; ++i)  // the kernels read a position of each pair's axis
    if (p->axis[i] >= p->n_axes) return "plan not set by clo_rope_plan_init";
  if (p->rot_dim > head_dim) return "rot_dim is larger than head_dim";
  return nullptr;
}

extern "C" CLO_API clo_status clo_rope(const clo_rope_plan* plan, const clo_rows* x, const clo_rows* y, const int64_t* positions,
                                       int64_t n_tokens, int32_t n_heads, int32_t head_dim, int32_t transpose, void* stream) {
  const char* who = "clo_rope";
  if (head_dim < 2 || head_dim % 2 || head_dim > 1024) return paged_fail(CLO_ERR_INVALID, "%s: head_dim must be even, 2 .. 1024", who);
  if (n_tokens < 0 || n_heads < 0 || n_tokens > (int64_t(1) << 40) || n_heads > 65535)
    return paged_fail(CLO_ERR_INVALID, "%s: n_tokens must be 0 .. 2^40, n_heads 0 .. 65535", who);
  if (const char* f = plan_fault(plan, head_dim)) return paged_fail(CLO_ERR_INVALID, "%s: %s", who, f);
  if (n_tokens == 0 || n_heads == 0) return CLO_OK;
  for (const clo_rows* r : {x, y})
    if (const char* f = rows_fault(r, false)) return paged_fail(CLO_ERR_INVALID, "%s: %s", who, f);
  if (!positions || (reinterpret_cast<uintptr_t>(positions) & 7u)) return paged_fail(CLO_ERR_INVALID, "%s: positions must be 8-byte aligned int64", who);
  if (x->ptr == y->ptr && (x->stride_token != y->stride_token || x->stride_head != y->stride_head))
    return paged_fail(CLO_ERR_INVALID, "%s: x and y may be the same rows only with the same strides", who);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Rope r{*plan, transpose != 0};
  const bool vec = !rows_fault(x, true) && !rows_fault(y, true) && plan->rot_dim % 16 == 0 && (head_dim == 64 || head_dim == 128);
  if (vec) {
    const int rows = 32 / (head_dim / 16);  // heads per round
    const int iters = n_tokens < kLongTokens || n_heads <= kShortIters * rows ? kShortIters : kMidIters;
    const int per = iters * rows;  // heads per warp
    const int chunks = (n_heads + per - 1) / per;
    const int64_t blocks = (n_tokens * chunks + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffff) return paged_fail(CLO_ERR_INVALID, "%s: too many rows for one call", who);
    auto kernel = [&](auto d, auto axes) {
      constexpr int D = decltype(d)::value;
      constexpr bool AXES = decltype(axes)::value;
      return iters == kMidIters ? k_rope<D, kMidIters, AXES> : k_rope<D, kShortIters, AXES>;
    };
    using D128 = std::integral_constant<int, 128>;
    using D64 = std::integral_constant<int, 64>;
    auto* f = plan->n_axes > 1 ? (head_dim == 128 ? kernel(D128{}, std::true_type{}) : kernel(D64{}, std::true_type{}))
                               : (head_dim == 128 ? kernel(D128{}, std::false_type{}) : kernel(D64{}, std::false_type{}));
    f<<<(unsigned)blocks, kThreads, 0, st>>>(r, rows_of(x), rows_of(y), positions, n_tokens, n_heads, chunks);
  } else {
    const int64_t pairs = n_tokens * n_heads * (head_dim - plan->rot_dim / 2);
    const int64_t blocks = (pairs + kThreads - 1) / kThreads;
    k_rope_any<<<(unsigned)(blocks < 65536 ? blocks : 65536), kThreads, 0, st>>>(r, rows_of(x), rows_of(y), positions, n_tokens, n_heads, head_dim);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return paged_fail(CLO_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return CLO_OK;
}

extern "C" CLO_API clo_status clo_paged_read(const clo_paged_cache* cache, const clo_paged_batch* batch, const clo_rows* k_out,
                                             const clo_rows* v_out, void* stream) {
  const char* who = "clo_paged_read";
  ReadParams a{};
  if (const char* f = paged_params(cache, batch, &a.c)) return paged_fail(CLO_ERR_INVALID, "%s: %s", who, f);
  if (batch->batch == 0 || batch->total_q == 0 || a.c.max_q == 0) return CLO_OK;
  for (const clo_rows* r : {k_out, v_out})
    if (const char* f = rows_fault(r, true)) return paged_fail(CLO_ERR_INVALID, "%s: %s", who, f);
  a.out[0] = rows_of(k_out);
  a.out[1] = rows_of(v_out);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned blocks = (unsigned)((a.c.total_q + kWarps - 1) / kWarps);
  if (cache->head_dim == 128) {
    if (cache->kv_bits == 16) k_paged_read<128, 16><<<blocks, kThreads, 0, st>>>(a);
    else if (cache->kv_bits == 8) k_paged_read<128, 8><<<blocks, kThreads, 0, st>>>(a);
    else k_paged_read4<128><<<blocks, kThreads, 0, st>>>(a);
  } else {
    if (cache->kv_bits == 16) k_paged_read<64, 16><<<blocks, kThreads, 0, st>>>(a);
    else if (cache->kv_bits == 8) k_paged_read<64, 8><<<blocks, kThreads, 0, st>>>(a);
    else k_paged_read4<64><<<blocks, kThreads, 0, st>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return paged_fail(CLO_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return CLO_OK;
}
