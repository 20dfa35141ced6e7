// Device parts of the rotation by positions, shared by clo_rope and clo_paged_append.
//
// The unit of work is 16 elements of one head's row: the two 8-element vectors whose elements pair up
// (half layout: elements [8u, 8u + 8) and the same offset by rot_dim / 2; interleaved: 16 adjacent ones; a
// head's rest behind rot_dim: 16 adjacent ones, copied).  d / 16 lanes cover a row, so that a lane keeps
// its unit while its warp walks over rows.
#pragma once

#include <stddef.h>

#include "clo_paged.cuh"

namespace clo {

struct Rope {
  clo_rope_plan plan;  // rot_dim 0: copy
  int transpose;
};

struct Rows {
  uint16_t* p;
  int64_t token, head;
};

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;


// What a lane knows about its 16-element unit.
template <int D>
struct Unit {
  int a, b;       // element offsets of the two vectors
  bool rotate, interleaved;
  uint64_t turn[8];
  uint64_t axes;  // AXES: a byte per pair
  float magnitude;
};

// The plan's turns in shared memory: lanes read their units' with wide loads, where the parameter space would serve one address at a time.
// AXES: behind them the axes of each unit's eight pairs, a byte each.
template <bool AXES>
constexpr int kTurns = CLO_ROPE_MAX_PAIRS + (AXES ? CLO_ROPE_MAX_PAIRS / 8 : 0);
static_assert(offsetof(clo_rope_plan, axis) % 8 == 0, "the axes are read by eight");
template <bool AXES>
__device__ __forceinline__ void stage_turns(const Rope& r, uint64_t* s_turn) {
  if (threadIdx.x < CLO_ROPE_MAX_PAIRS) s_turn[threadIdx.x] = r.plan.turn[threadIdx.x];
  if (AXES && threadIdx.x < CLO_ROPE_MAX_PAIRS / 8) s_turn[CLO_ROPE_MAX_PAIRS + threadIdx.x] = reinterpret_cast<const uint64_t*>(r.plan.axis)[threadIdx.x];
  __syncthreads();
}

// Where a row stands, on every axis alike or on each.
template <bool AXES>
struct Place {
  int64_t pos;
  __device__ __forceinline__ int64_t on(uint32_t) const { return pos; }
};
template <>
struct Place<true> {
  int64_t pos[CLO_ROPE_MAX_AXES];
  __device__ __forceinline__ int64_t on(uint32_t axis) const {
    const int64_t lo = axis & 1 ? pos[1] : pos[0], hi = axis & 1 ? pos[3] : pos[2];
    return axis & 2 ? hi : lo;
  }
};
// Row `row` of a call's positions (null: it stands at `pos`), `n` rows in all.
template <bool AXES>
__device__ __forceinline__ Place<AXES> place_of(const Rope& r, const int64_t* positions, int64_t row, int64_t n, int64_t pos) {
  Place<AXES> w;
  if constexpr (AXES) {
#pragma unroll
    for (int a = 0; a < CLO_ROPE_MAX_AXES; ++a) w.pos[a] = positions && a < r.plan.n_axes ? __ldg(positions + a * n + row) : pos;
  } else {
    w.pos = positions ? __ldg(positions + row) : pos;
  }
  return w;
}

template <int D, bool AXES>
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
    if (AXES) x.axes = s_turn[CLO_ROPE_MAX_PAIRS + u];
  }
  return x;
}

struct CosSin {
  float2 v[8];
};

template <int D, bool AXES>
__device__ __forceinline__ CosSin cos_sin_of(const Unit<D>& u, const Place<AXES>& where, int transpose) {
  CosSin c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c.v[i] = rope_cos_sin(where.on(AXES ? (uint32_t)(u.axes >> (8 * i)) : 0u), u.turn[i], u.magnitude);
    if (transpose) c.v[i].y = -c.v[i].y;
  }
  return c;
}

// The same for a warp whose lanes all stand at one place: the lanes that share a unit compute a pair or two each and hand them around.
template <int D, bool AXES>
__device__ __forceinline__ CosSin cos_sin_shared(const Rope& r, const uint64_t* s_turn, const Place<AXES>& where, int lane) {
  constexpr int kLanes = D / 16, kShare = 32 / kLanes, kOwn = 8 / kShare;
  const int u = lane % kLanes, first = lane / kLanes;
  float2 own[kOwn];
#pragma unroll
  for (int j = 0; j < kOwn; ++j) {
    const int i = first + j * kShare;
    const uint32_t axis = AXES ? (uint32_t)(s_turn[CLO_ROPE_MAX_PAIRS + u] >> (8 * i)) : 0u;
    own[j] = rope_cos_sin(where.on(axis), s_turn[u * 8 + i], r.plan.magnitude);
    if (r.transpose) own[j].y = -own[j].y;
  }
  CosSin c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c.v[i].x = __shfl_sync(0xffffffffu, own[i / kShare].x, u + i % kShare * kLanes);
    c.v[i].y = __shfl_sync(0xffffffffu, own[i / kShare].y, u + i % kShare * kLanes);
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

// ---------------------------------------------------------------------------- rows of one token
// A warp takes one token and up to ITERS rounds of its heads: the cosines and sines of a lane's unit are computed
// once for all of them.
template <int D, int ITERS, bool AXES, typename F>
__device__ __forceinline__ void rotate_heads(const Rope& r, const uint64_t* s_turn, const Rows& x, const Rows& y, int64_t token, F&& position,
                                             int head0, int n_heads, int lane) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  const Unit<D> u = unit_of_lane<D, AXES>(r, s_turn, lane % kLanes);
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
  Place<AXES> where;
  if (!position(&where)) return;
  const CosSin c = cos_sin_shared<D, AXES>(r, s_turn, where, lane);
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

// Rounds of heads per warp: more for long calls, where the sines count, few for short ones, where the latency does, and no more than the
// heads fill.  8192 tokens of 128-element heads, us with 8 / 4 / 2 rounds: 32 heads (floor 19.8) 24.7 / 24.0 / 24.7, 40 heads (24.7)
// 28.8 / 28.8 / 29.1; 30,000 tokens of 32 heads (72.4) 74.7 / 73.8 / 75.9.  (Before lanes shared the sines, eight were best for 32 heads.)  The
// append's queries take eight, beside pages that are written by whole warps.
constexpr int kLongIters = 8, kMidIters = 4, kShortIters = 2;
constexpr int64_t kLongTokens = 8 * 152;  // a warp per SM and slot of eight
template <int D>
__host__ __device__ constexpr int heads_per_warp(int iters) { return iters * 32 / (D / 16); }

}  // namespace

// ---------------------------------------------------------------------------- arguments
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline const char* rows_fault(const clo_rows* r, bool vectors) {
  if (!r || !r->ptr) return "null pointer";
  if (reinterpret_cast<uintptr_t>(r->ptr) & 1u) return "rows must be 2-byte aligned";
  if (vectors && (!aligned16(r->ptr) || r->stride_token % 8 || r->stride_head % 8))
    return "rows must lie on 16-byte boundaries (strides multiples of 8 elements)";
  return nullptr;
}

inline Rows rows_of(const clo_rows* r) { return Rows{static_cast<uint16_t*>(r->ptr), r->stride_token, r->stride_head}; }

// What is wrong with a plan, or null.
const char* plan_fault(const clo_rope_plan* p, int head_dim);

}  // namespace clo
