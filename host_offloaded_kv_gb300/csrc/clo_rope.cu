// Rotary positions (clo_rope), paged append with the rotation on the way (clo_paged_append) and the
// read-back (clo_paged_read): one pass over the rows each, bounded by HBM traffic (large calls) or by
// one launch and two or three dependent loads (single-token steps).
//
// The unit of work is 16 elements of one head's row: the two 8-element vectors whose elements pair up
// (half layout: elements [8u, 8u + 8) and the same offset by rot_dim / 2; interleaved: 16 adjacent ones; a
// head's rest behind rot_dim: 16 adjacent ones, copied).  d / 16 lanes cover a row, so that a lane keeps
// its unit while its warp walks over rows.
//
// Measured: 8192 tokens of 32 heads of 128, 24.9 us, 5.4 TB/s (80 % of a copy's rate); 30,000 tokens 75 us, 96 %; one token 2.2 us in a
// graph.  Append with queries, 32 over 8 heads: 11,000 tokens, bf16 pages 52 us, 5.2 TB/s, 8-bit pages 54 us, 4.6 TB/s (registers hold two
// blocks to an SM: a page's rows stay in them until its scale is known); 64 single tokens, in a graph, 3.8 and 4.5 us.  Read-back of
// 8 x 8192 tokens: bf16 82 us, 6.5 TB/s, 8-bit pages 70 us, 5.8 TB/s.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "clo.h"
#include "clo_paged.cuh"

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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Rope {
  clo_rope_plan plan;  // rot_dim 0: copy
  int transpose;
};

// What a lane knows about its 16-element unit.
template <int D>
struct Unit {
  int a, b;       // element offsets of the two vectors
  bool rotate, interleaved;
  uint64_t turn[8];
  float magnitude;
};

// The plan's turns in shared memory: lanes read their units' with wide loads, where the parameter space would serve one address at a time.
__device__ __forceinline__ void stage_turns(const Rope& r, uint64_t* s_turn) {
  if (threadIdx.x < CLO_ROPE_MAX_PAIRS) s_turn[threadIdx.x] = r.plan.turn[threadIdx.x];
  __syncthreads();
}

template <int D>
__device__ __forceinline__ Unit<D> unit_of_lane(const Rope& r, const uint64_t* s_turn, int u) {
  Unit<D> x;
  const int rot = r.plan.rot_dim;
  x.rotate = u * 16 < rot;
  x.interleaved = r.plan.interleaved != 0;
  x.magnitude = r.plan.magnitude;
  if (x.rotate && !x.interleaved) {
    x.a = u * 8;
    x.b = rot / 2 + u * 8;
  } else {
    x.a = u * 16;
    x.b = u * 16 + 8;
  }
  if (x.rotate) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(s_turn + u * 8 + i);
      x.turn[i] = t.x;
      x.turn[i + 1] = t.y;
    }
  }
  return x;
}

struct CosSin {
  float2 v[8];
};

template <int D>
__device__ __forceinline__ CosSin cos_sin_of(const Unit<D>& u, int64_t pos, int transpose) {
  CosSin c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c.v[i] = rope_cos_sin(pos, u.turn[i], u.magnitude);
    if (transpose) c.v[i].y = -c.v[i].y;
  }
  return c;
}

// Rotates a unit: x[0..8) are the elements at a, x[8..16) those at b.
template <int D>
__device__ __forceinline__ void rotate_unit(const Unit<D>& u, const CosSin& c, float* x) {
  if (u.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = x[2 * i], q = x[2 * i + 1];
      x[2 * i] = fmaf(p, c.v[i].x, -q * c.v[i].y);
      x[2 * i + 1] = fmaf(q, c.v[i].x, p * c.v[i].y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = x[i], q = x[8 + i];
      x[i] = fmaf(p, c.v[i].x, -q * c.v[i].y);
      x[8 + i] = fmaf(q, c.v[i].x, p * c.v[i].y);
    }
  }
}

struct Rows {
  uint16_t* p;
  int64_t token, head;
};

// ---------------------------------------------------------------------------- rows of one token
// A warp takes one token and up to ITERS rounds of its heads: the cosines and sines of a lane's unit are computed
// once for all of them.
template <int D, int ITERS, typename F>
__device__ __forceinline__ void rotate_heads(const Rope& r, const uint64_t* s_turn, const Rows& x, const Rows& y, int64_t token, F&& position,
                                             int head0, int n_heads, int lane) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  const Unit<D> u = unit_of_lane<D>(r, s_turn, lane % kLanes);
  const uint16_t* src = x.p + token * x.token;
  uint16_t* dst = y.p + token * y.token;
  uint4 va[ITERS], vb[ITERS];
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int h = head0 + i * kRows + lane / kLanes;
    if (h < n_heads) {
      va[i] = *reinterpret_cast<const uint4*>(src + (int64_t)h * x.head + u.a);
      vb[i] = *reinterpret_cast<const uint4*>(src + (int64_t)h * x.head + u.b);
    }
  }
  int64_t pos;
  if (!position(&pos)) return;
  CosSin c;
  if (u.rotate) c = cos_sin_of<D>(u, pos, r.transpose);
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int h = head0 + i * kRows + lane / kLanes;
    if (h < n_heads) {
      if (u.rotate) {
        float f[16];
        unpack8(va[i], f);
        unpack8(vb[i], f + 8);
        rotate_unit<D>(u, c, f);
        va[i] = pack8(f);
        vb[i] = pack8(f + 8);
      }
      *reinterpret_cast<uint4*>(dst + (int64_t)h * y.head + u.a) = va[i];
      *reinterpret_cast<uint4*>(dst + (int64_t)h * y.head + u.b) = vb[i];
    }
  }
}

// Rounds of heads per warp: many for long calls, where the sines count, few for short ones, where the latency does, and no more
// than the heads fill.  8192 tokens of 128-element heads, us with 8 / 4 / 2 rounds: 8 heads (floor 5.0) 11.0 / - / 7.5, 16 heads (9.9)
// 13.0 / 10.7 / -, 40 heads (24.7) 33.6 / 30.4 / -; 2000 tokens, 32 heads (4.8) 6.3 / 7.1 / -.
constexpr int kLongIters = 8, kMidIters = 4, kShortIters = 2;
constexpr int64_t kLongTokens = 8 * 152;  // a warp per SM and slot of eight
template <int D>
__host__ __device__ constexpr int heads_per_warp(int iters) { return iters * 32 / (D / 16); }

template <int D, int ITERS>
__global__ void __launch_bounds__(kThreads, ITERS == kLongIters ? 2 : ITERS == kMidIters ? 3 : 4) k_rope(const Rope r, const Rows x, const Rows y, const int64_t* __restrict__ positions,
                                                   int64_t n_tokens, int n_heads, int chunks) {
  __shared__ __align__(16) uint64_t s_turn[CLO_ROPE_MAX_PAIRS];
  stage_turns(r, s_turn);
  const int64_t job = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = job / chunks;
  if (t >= n_tokens) return;
  auto position = [&](int64_t* pos) {
    *pos = positions[t];
    return true;
  };
  rotate_heads<D, ITERS>(r, s_turn, x, y, t, position, (int)(job % chunks) * heads_per_warp<D>(ITERS), n_heads, threadIdx.x & 31);
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
    float2 c = rope_cos_sin(positions[t], r.plan.turn[i], r.plan.magnitude);
    if (r.transpose) c.y = -c.y;
    const float p = bf16_bits_to_f32(src[a]), q = bf16_bits_to_f32(src[b]);
    dst[a] = (uint16_t)pack_bf16(fmaf(p, c.x, -q * c.y), 0.f);
    dst[b] = (uint16_t)pack_bf16(fmaf(q, c.x, p * c.y), 0.f);
  }
}

// ---------------------------------------------------------------------------- paged append
struct AppendParams {
  PagedParams c;
  Rows in[2];  // k, v
  Rows q, q_out;
  const int64_t* positions;
  int32_t n_q_heads;   // 0: no queries
  int32_t q_chunks;    // warps per query token
  int32_t items;       // upper bound of (sequence, touched page) pairs
  int32_t kv_blocks;   // blocks that write pages; the others rotate queries
  Rope rope;
};

// The item-th (sequence, touched page) of the batch, by the whole warp; false past the last one.
__device__ __forceinline__ bool item_of(const PagedParams& p, int item, int lane, int* seq, int* logical, SeqRows* rows) {
  int before = 0;
  for (int c = 0; c < p.batch; c += 32) {
    int pages = 0;
    SeqRows s;
    if (c + lane < p.batch) {
      s = seq_rows(p, c + lane);
      if (s.n > 0) {
        // positions [pos0, pos0 + n) clipped to [0, capacity)
        const int lo = max(s.pos0, 0), hi = min((int64_t)s.pos0 + s.n, (int64_t)p.max_pages << p.page_shift);
        if (hi > lo) pages = ((hi - 1) >> p.page_shift) - (lo >> p.page_shift) + 1;
      }
    }
    int incl = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned m = __ballot_sync(0xffffffffu, before + incl > item);
    if (m) {
      const int l = __ffs(m) - 1;
      const int b = c + l;
      const int skip = item - before - (__shfl_sync(0xffffffffu, incl, l) - __shfl_sync(0xffffffffu, pages, l));
      *seq = b;
      *rows = seq_rows(p, b);
      *logical = (max(rows->pos0, 0) >> p.page_shift) + skip;
      return true;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// One job: (touched page, kv head, K or V), by kPer warps.  A lane holds kUnits units (16 elements of a row each) in registers from
// the load to the store, so that rows are read and rotated once also where the page's scale comes in between; kPer warps
// hold the most rows that a page can get from the call.
constexpr int kUnits = 4;

template <int D, int BITS, int kPer>
__device__ __forceinline__ void write_page(const AppendParams& a, const uint64_t* s_turn, int item, int head, int side, int part, int lane, float* s_red,
                                           int group) {
  const PagedParams& p = a.c;
  int b, logical;
  SeqRows s;
  if (!item_of(p, item, lane, &b, &logical, &s)) return;
  const int page = page_of(p, b, logical);
  if (page < 0) return;
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  const int base = logical << p.page_shift;             // position of slot 0
  const int lo = max(max(s.pos0, 0), base), hi = min(s.pos0 + s.n, base + p.page_size);
  const PagedSide& sd = p.side[side];
  const Rows& in = a.in[side];
  Unit<D> u = unit_of_lane<D>(a.rope, s_turn, lane % kLanes);
  const bool rotate = side == 0 && u.rotate;
  if (side == 1) {
    u.a = (lane % kLanes) * 16;
    u.b = u.a + 8;
  }
  char* dst0 = sd.pages + ((int64_t)page * sd.stride_page + (int64_t)head * sd.stride_head) * (BITS / 8);
  const int first = lo + part * kRows + lane / kLanes;  // this lane's rows: first, + kPer * kRows, ...

  uint4 va[kUnits], vb[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int pos = first + i * kPer * kRows;
    if (pos < hi) {
      const uint16_t* src = in.p + (int64_t)(s.first + (pos - s.pos0)) * in.token + (int64_t)head * in.head;
      va[i] = __ldg(reinterpret_cast<const uint4*>(src + u.a));
      vb[i] = __ldg(reinterpret_cast<const uint4*>(src + u.b));
    }
  }
  float f[kUnits][16], amax = 0.f;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int pos = first + i * kPer * kRows;
    if (pos < hi) {
      unpack8(va[i], f[i]);
      unpack8(vb[i], f[i] + 8);
      if (rotate) {
        const int64_t at = a.positions ? __ldg(a.positions + s.first + (pos - s.pos0)) : pos;
        rotate_unit<D>(u, cos_sin_of<D>(u, at, 0), f[i]);
      }
      if (BITS == 16) {
        char* dst = dst0 + (int64_t)(pos - base) * sd.stride_token * 2;
        *reinterpret_cast<uint4*>(dst + u.a * 2) = pack8(f[i]);
        *reinterpret_cast<uint4*>(dst + u.b * 2) = pack8(f[i] + 8);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float m = fabsf(f[i][k]);
          amax = fmaxf(amax, m < INFINITY ? m : 0.f);
        }
      }
    }
  }
  if (BITS == 16) return;
  amax = warp_max(amax);
  if (kPer > 1) {
    if (lane == 0) s_red[group * kPer + part] = amax;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(kPer * 32) : "memory");
#pragma unroll
    for (int i = 0; i < kPer; ++i) amax = fmaxf(amax, s_red[group * kPer + i]);
  }
  // smallest e with amax <= 1.75 * 2^(8 + e), from the bits of amax
  const int bits = __float_as_int(amax);
  int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  e = max(e, kMinScaleExp);
  float scale = __int_as_float((e + 127) << 23);
  float* sp = sd.scales + (int64_t)page * p.n_kv_heads + head;
  if (lo > base) {
    const float old = *sp;
    if (old >= scale) {  // a scale that is no number is replaced
      scale = old;
    } else if (old > 0.f) {
      const float f = old / scale;
      for (int v = part * 32 + lane; v < (lo - base) * (D / 8); v += kPer * 32) {
        uint2* c = reinterpret_cast<uint2*>(dst0 + (int64_t)(v / (D / 8)) * sd.stride_token + v % (D / 8) * 8);
        const uint2 w = *c;
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 d = e4m3_to_f32x2(((i < 2 ? w.x : w.y) >> (16 * (i & 1))) & 0xffffu);
          x[2 * i] = d.x * f;
          x[2 * i + 1] = d.y * f;
        }
        *c = pack8_e4m3(x);
      }
    }
  }
  const float inv = 1.f / scale;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int pos = first + i * kPer * kRows;
    if (pos < hi) {
#pragma unroll
      for (int k = 0; k < 16; ++k) f[i][k] *= inv;
      char* dst = dst0 + (int64_t)(pos - base) * sd.stride_token;
      *reinterpret_cast<uint2*>(dst + u.a) = pack8_e4m3(f[i]);
      *reinterpret_cast<uint2*>(dst + u.b) = pack8_e4m3(f[i] + 8);
    }
  }
  // every warp has read the old scale
  if (kPer > 1) asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(kPer * 32) : "memory");
  __syncwarp();
  if (part == 0 && lane == 0) *sp = scale;
}

template <int D, int BITS, int kPer>
__global__ void __launch_bounds__(kThreads) k_paged_append(const AppendParams a) {
  __shared__ __align__(16) uint64_t s_turn[CLO_ROPE_MAX_PAIRS];
  __shared__ float s_red[kWarps];
  stage_turns(a.rope, s_turn);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((int)blockIdx.x < a.kv_blocks) {
    const int64_t job = (int64_t)blockIdx.x * (kWarps / kPer) + warp / kPer;
    const int heads = a.c.n_kv_heads;
    const int64_t item = job / (2 * heads);
    if (item >= a.items) return;
    write_page<D, BITS, kPer>(a, s_turn, (int)item, (int)(job % heads), (int)(job / heads & 1), warp % kPer, lane, s_red, warp / kPer);
    return;
  }
  constexpr int kIters = kPer == 1 ? kShortIters : kLongIters;
  const int64_t job = (int64_t)((int)blockIdx.x - a.kv_blocks) * kWarps + warp;
  const int64_t t = job / a.q_chunks;
  if (t >= a.c.total_q) return;
  // the row's sequence is looked up while its elements are on their way
  auto position = [&](int64_t* pos) {
    const int b = seq_of_row(a.c, (int)t, lane);
    if (b >= a.c.batch) return false;
    const SeqRows s = seq_rows(a.c, b);
    if (t - s.first >= s.n) return false;  // beyond max_q: left out, as its key is
    *pos = a.positions ? __ldg(a.positions + t) : (int64_t)s.pos0 + (t - s.first);
    return true;
  };
  rotate_heads<D, kIters>(a.rope, s_turn, a.q, a.q_out, t, position, (int)(job % a.q_chunks) * heads_per_warp<D>(kIters), a.n_q_heads, lane);
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

// ---------------------------------------------------------------------------- arguments
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

const char* rows_fault(const clo_rows* r, bool vectors) {
  if (!r || !r->ptr) return "null pointer";
  if (reinterpret_cast<uintptr_t>(r->ptr) & 1u) return "rows must be 2-byte aligned";
  if (vectors && (!aligned16(r->ptr) || r->stride_token % 8 || r->stride_head % 8))
    return "rows must lie on 16-byte boundaries (strides multiples of 8 elements)";
  return nullptr;
}

Rows rows_of(const clo_rows* r) { return Rows{static_cast<uint16_t*>(r->ptr), r->stride_token, r->stride_head}; }

}  // namespace

// Checks a cache and a batch and fills the kernels' view of them; null or what is wrong.
const char* paged_params(const clo_paged_cache* c, const clo_paged_batch* b, PagedParams* p) {
  if (!c || !b) return "null pointer";
  if (!c->k_pages || !c->v_pages) return "null pages";
  if (c->head_dim != 64 && c->head_dim != 128) return "head_dim must be 64 or 128";
  if (c->kv_bits != 16 && c->kv_bits != 8) return "kv_bits must be 16 or 8";
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return "page_size must be 16, 32, 64 or 128";
  if (c->n_kv_heads < 1 || c->n_kv_heads > 65535) return "n_kv_heads must be 1 .. 65535";
  if (c->n_pages < 1 || c->n_pages > 0x7fffffff) return "n_pages must be 1 .. 2^31 - 1";
  const int64_t per16 = 128 / c->kv_bits;
  const int64_t strides[6] = {c->k_stride_page, c->k_stride_head, c->k_stride_token, c->v_stride_page, c->v_stride_head, c->v_stride_token};
  for (int64_t s : strides)
    if (s <= 0 || s % per16 || s * (c->kv_bits / 8) >= (int64_t(1) << 40)) return "page strides must be positive multiples of 16 bytes, below 2^40 bytes";
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return "pages must be 16-byte aligned";
  if (c->kv_bits == 8 && (!c->k_scales || !c->v_scales || (reinterpret_cast<uintptr_t>(c->k_scales) & 3u) || (reinterpret_cast<uintptr_t>(c->v_scales) & 3u)))
    return "8-bit pages need 4-byte aligned scales";
  if (b->batch < 0 || b->batch > 65535) return "batch must be 0 .. 65535";
  if (b->total_q < 0 || b->total_q > kMaxPagedTokens || b->max_q < 0) return "total_q must be 0 .. 2^30, max_q not negative";
  if (b->max_pages < 0 || (int64_t)b->max_pages * c->page_size >= kMaxPagedTokens) return "max_pages * page_size must be below 2^30";
  if (b->batch > 0 && b->total_q > 0) {
    if (!b->q_starts || !b->kv_lens || (!b->block_table && b->max_pages > 0)) return "null pointer in the batch";
    if ((reinterpret_cast<uintptr_t>(b->q_starts) | reinterpret_cast<uintptr_t>(b->kv_lens) | reinterpret_cast<uintptr_t>(b->block_table)) & 3u)
      return "the batch's arrays must be 4-byte aligned";
  }
  p->side[0] = PagedSide{static_cast<char*>(c->k_pages), c->k_scales, c->k_stride_page, c->k_stride_head, c->k_stride_token};
  p->side[1] = PagedSide{static_cast<char*>(c->v_pages), c->v_scales, c->v_stride_page, c->v_stride_head, c->v_stride_token};
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
  const double two_pi = 6.283185307179586476925;
  memset(plan, 0, sizeof *plan);
  double lo = 0.0, hi = 0.0;
  if (c->scaling == CLO_ROPE_YARN) {
    auto pair_of = [&](double n) { return rot * std::log((double)c->original_max / (n * two_pi)) / (2.0 * std::log(c->theta)); };
    lo = std::fmax(0.0, std::floor(pair_of(c->beta_fast)));
    hi = std::fmin(rot - 1.0, std::ceil(pair_of(c->beta_slow)));
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(c->theta, -2.0 * i / rot);
    double keep = 1.0;  // share of the unscaled frequency
    if (c->scaling == CLO_ROPE_LINEAR) keep = 0.0;
    if (c->scaling == CLO_ROPE_BANDS) keep = ((double)c->original_max * f / two_pi - c->low_freq) / (c->high_freq - c->low_freq);
    if (c->scaling == CLO_ROPE_YARN) keep = 1.0 - std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 1e-3)));
    keep = std::fmin(1.0, std::fmax(0.0, keep));
    f = keep * f + (1.0 - keep) * f / c->factor;
    // f <= 1 radian per position, so the fraction of a turn is below 1/6
    plan->turn[i] = (uint64_t)std::llrint(std::ldexp(f / two_pi, 62)) << 2;
  }
  plan->magnitude = c->magnitude > 0.0 ? (float)c->magnitude
                    : c->scaling == CLO_ROPE_YARN ? (float)(0.1 * std::log(c->factor) + 1.0) : 1.f;
  plan->rot_dim = rot;
  plan->interleaved = c->interleaved != 0;
  plan->ready = 1;
  return CLO_OK;
}

static const char* plan_fault(const clo_rope_plan* p, int head_dim) {
  if (!p) return "null plan";
  if (p->ready != 1 || p->rot_dim < 2 || p->rot_dim % 2 || p->rot_dim > 2 * CLO_ROPE_MAX_PAIRS) return "plan not set by clo_rope_plan_init";
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
    const int iters = n_tokens < kLongTokens || n_heads <= kShortIters * rows ? kShortIters : n_heads % (kLongIters * rows) ? kMidIters : kLongIters;
    const int per = iters * rows;  // heads per warp
    const int chunks = (n_heads + per - 1) / per;
    const int64_t blocks = (n_tokens * chunks + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffff) return paged_fail(CLO_ERR_INVALID, "%s: too many rows for one call", who);
    auto* f = head_dim == 128 ? (iters == kLongIters ? k_rope<128, kLongIters> : iters == kMidIters ? k_rope<128, kMidIters> : k_rope<128, kShortIters>)
                              : (iters == kLongIters ? k_rope<64, kLongIters> : iters == kMidIters ? k_rope<64, kMidIters> : k_rope<64, kShortIters>);
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

template <int D, int BITS>
static void launch_append(const AppendParams& a, int64_t blocks, int per, cudaStream_t st) {
  auto* f = per == 1 ? k_paged_append<D, BITS, 1> : per == 2 ? k_paged_append<D, BITS, 2> : per == 4 ? k_paged_append<D, BITS, 4> : k_paged_append<D, BITS, 8>;
  f<<<(unsigned)blocks, kThreads, 0, st>>>(a);
}

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
  if (cache->head_dim == 128) {
    if (cache->kv_bits == 16) launch_append<128, 16>(a, blocks, per, st);
    else launch_append<128, 8>(a, blocks, per, st);
  } else {
    if (cache->kv_bits == 16) launch_append<64, 16>(a, blocks, per, st);
    else launch_append<64, 8>(a, blocks, per, st);
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
    else k_paged_read<128, 8><<<blocks, kThreads, 0, st>>>(a);
  } else {
    if (cache->kv_bits == 16) k_paged_read<64, 16><<<blocks, kThreads, 0, st>>>(a);
    else k_paged_read<64, 8><<<blocks, kThreads, 0, st>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return paged_fail(CLO_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return CLO_OK;
}
