// Paged append with the rotation on the way: the kernel and its launch, instantiated by the pages' type.  One pass over the rows, bounded
// by HBM traffic (large calls) or by one launch and two or three dependent loads (single-token steps).
//
// Measured with queries, 32 over 8 heads: 11,000 tokens, bf16 pages 52 us, 5.2 TB/s, 8-bit pages 53 us, 4.6 TB/s (registers hold two
// blocks to an SM: a page's rows stay in them until its scale is known); 64 single tokens, in a graph, 3.9 and 4.5 us.
// One sequence of 10,800 tokens at positions on three axes, in a graph, with queries / without / without rotation, us: bf16 55.6 / 31.7 / 20.6, 8-bit
// pages 56.2 / 33.3 / 21.2, 4-bit pages 73.6 / 59.4 / 33.2, where instructions bound it and 128 registers hold not all: 100 to 172 bytes a thread spill.
// 64 single tokens of 4-bit pages 5.8 us, and 8 us more where a pair is left open (rotate_exactly), one call in three or four.
#pragma once

#include <type_traits>

#include "clo_rope.cuh"
#include "clo_rotate_exact.cuh"

namespace clo {

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

// A call's launch, by the pages' type.
void launch_append_bf16(const AppendParams& a, int head_dim, int64_t blocks, int per, cudaStream_t st);
void launch_append_e4m3(const AppendParams& a, int head_dim, int64_t blocks, int per, cudaStream_t st);
void launch_append_e2m1(const AppendParams& a, int head_dim, int64_t blocks, int per, cudaStream_t st);

namespace {

// ---------------------------------------------------------------------------- paged append

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

// ---- 4-bit pages.  A group is 16 neighbouring elements, that is two 8-element vectors, of two lanes where a rotated row pairs up its halves.

// Where the other vectors of the groups of this lane's vectors are: the lane, and which of its two.
template <int D>
struct Partners {
  int lane_a, lane_b;
  bool second_a, second_b;
};
template <int D>
__device__ __forceinline__ Partners<D> partners_of(bool halves, int rot_dim, int lane) {
  constexpr int kLanes = D / 16;
  const int u = lane % kLanes, row = lane - u, n = halves ? rot_dim / 16 : 0;  // rotating units of a row in the half layout
  auto owner = [&](int vec, bool* second) {
    *second = vec < 2 * n ? vec >= n : vec & 1;
    return row + (vec < 2 * n ? (vec >= n ? vec - n : vec) : vec >> 1);
  };
  Partners<D> w;
  w.lane_a = owner((u < n ? u : 2 * u) ^ 1, &w.second_a);
  w.lane_b = owner((u < n ? n + u : 2 * u + 1) ^ 1, &w.second_b);
  return w;
}

// The error (clo_rotate_exact.cuh) of a job's largest element, which is no smaller than the other one of its pair, and what the products with it round.
constexpr float kMaxError = 4.06e-7f + 1.13e-7f + 0x1p-23f;

// Codes and group scales of a unit's two vectors.
struct Codes4 {
  uint32_t a, b, scale_a, scale_b;
  uint32_t open;  // what fp32's rotation left open, a bit per pair: a code or a scale lies within its error of a border
};

// x / d for a divisor whose reciprocal r is given: one correction by the exact remainder (Markstein's method).  It rounds the quotient correctly
// where r is the rounded reciprocal; with an r that is a unit off, quotients of few bits, as on a border between two codes, still come out exactly.
__device__ __forceinline__ float quotient(float x, float d, float r) {
  const float t = x * r;
  return fmaf(fmaf(-t, d, x), r, t);
}

// e4m3 code of the scale of a group whose largest |x|, over the page's scale, has these bits (infinity: the largest scale; NaN: NaN).
__device__ __forceinline__ uint32_t group_scale_of(uint32_t bits) {
  if (bits >= 0x7f800000u) return bits == 0x7f800000u ? 0x7eu : 0x7fu;
  return pack_e4m3(quotient(__uint_as_float(bits), 6.f, 1.f / 6.f), 0.f);
}

// x: a unit's values; inv: one over the page's scale (a power of two); rotated: x carries fp32's errors (ROTATED false: no lane's does); one: the
// rotation's magnitude is 1.  All lanes of the warp take part.
template <int D, bool ROTATED>
__device__ __forceinline__ Codes4 encode_unit(const float* x, float inv, bool rotated, bool one, bool interleaved, const Partners<D>& with) {
  float y[16];
  uint32_t key[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    y[k] = x[k] * inv;
    key[k / 8] = max(key[k / 8], __float_as_uint(y[k]) & 0x7fffffffu);
  }
  float off[8], most = 0.f;
#pragma unroll
  for (int i = 0; ROTATED && i < 8; ++i) {
    const float o = interleaved ? rotation_error(y[2 * i], y[2 * i + 1], one) : rotation_error(y[i], y[8 + i], one);
    off[i] = rotated && o < INFINITY ? o : 0.f;
    most = fmaxf(most, off[i]);
  }
  Codes4 c;
  c.open = 0;
  uint32_t code[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const int from = v ? with.lane_b : with.lane_a;
    const bool second = v ? with.second_b : with.second_a;
    const uint32_t ka = __shfl_sync(0xffffffffu, key[0], from), kb = __shfl_sync(0xffffffffu, key[1], from);
    const float o = ROTATED ? fmaxf(most, __shfl_sync(0xffffffffu, most, from)) : 0.f;
    const uint32_t all = max(key[v], second ? kb : ka);
    const float m = __uint_as_float(all);
    const uint32_t scale = group_scale_of(o > 0.f ? __float_as_uint(m + o) : all);
    if (o > 0.f && all < 0x7f800000u && group_scale_of(__float_as_uint(fmaxf(m - o, 0.f))) != scale) c.open = 0xffu;
    const float s = e4m3_to_f32x2(scale).x;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    r = s > 0.f ? r : 0.f;
    if (all >= 0x7f800000u) {  // infinities: +-6 times the largest scale
#pragma unroll
      for (int k = 0; k < 8; ++k) y[8 * v + k] = fminf(fmaxf(y[8 * v + k], -1e30f), 1e30f);
    }
    float lo[8], hi[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      lo[k] = quotient(y[8 * v + k], s, r);
      if (ROTATED) {
        const float e = (interleaved ? off[4 * v + k / 2] : off[k]) * r;
        hi[k] = lo[k] + e;
        lo[k] -= e;
      }
    }
    code[v] = pack8_e2m1(lo);
    // a nibble for each element; halves: element k of either vector is of pair k; neighbours: elements 2 i, 2 i + 1 of vector v of pair 4 v + i
    const uint32_t top = ROTATED ? pack8_e2m1(hi) : code[v];
    if (top != code[v] && rotated) {
      const uint32_t d = codes_differ(&code[v], top);
#pragma unroll
      for (int k = 0; k < 8; ++k) c.open |= (d >> (4 * k) & 1u) << (interleaved ? 4 * v + k / 2 : k);
    }
    if (v) c.scale_b = scale;
    else c.scale_a = scale;
  }
  c.a = code[0];
  c.b = code[1];
  return c;
}

// One pair in integers (clo_rotate_exact.cuh), out of line.
__device__ __noinline__ float2 rotate_exactly(uint32_t p, uint32_t q, uint64_t angle, float magnitude) {
  float2 r;
  rotate_exact((uint16_t)p, (uint16_t)q, angle, magnitude, &r.x, &r.y);
  return r;
}

// One job: (touched page, kv head, K or V), by kPer warps.  A lane holds kUnits units (16 elements of a row each) in registers from
// the load to the store, so that rows are read and rotated once also where the page's scale comes in between; kPer warps
// hold the most rows that a page can get from the call.
constexpr int kUnits = 4;

template <int D, int BITS, int kPer, bool AXES>
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
  Unit<D> u = unit_of_lane<D, AXES>(a.rope, s_turn, lane % kLanes);
  const bool rotate = side == 0 && u.rotate;
  if (side == 1) {
    u.a = (lane % kLanes) * 16;
    u.b = u.a + 8;
  }
  char* dst0 = sd.pages + ((int64_t)page * sd.stride_page + (int64_t)head * sd.stride_head) * BITS / 8;
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
        rotate_unit<D>(u, cos_sin_of<D, AXES>(u, place_of<AXES>(a.rope, a.positions, s.first + (pos - s.pos0), p.total_q, pos), 0), f[i]);
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
  // the job's largest, of its warps' lanes
  auto over_warps = [&](float m) {
    m = warp_max(m);
    if (kPer > 1) {
      if (lane == 0) s_red[group * kPer + part] = m;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(kPer * 32) : "memory");
#pragma unroll
      for (int i = 0; i < kPer; ++i) m = fmaxf(m, s_red[group * kPer + i]);
    }
    return m;
  };
  // smallest e >= kMinScaleExp with m <= 448 * 2^e (8 bits: 1.75 * 2^8) or 2688 * 2^e (4 bits: 1.3125 * 2^11), from the bits of m
  auto exponent_of = [](float m) {
    constexpr int kTopExp = BITS == 8 ? 8 : 11, kTopMantissa = BITS == 8 ? 0x600000 : 0x280000;
    const int bits = __float_as_int(m);
    return max((bits >> 23) - 127 - kTopExp + ((bits & 0x7fffff) > kTopMantissa ? 1 : 0), kMinScaleExp);
  };
  // Pair n of the lane's unit of a row, in integers.
  auto exact_pair = [&](int pos, int n) {
    const int64_t row = s.first + (pos - s.pos0);
    const uint16_t* src = in.p + row * in.token + (int64_t)head * in.head;
    const int unit = lane % kLanes, ep = u.interleaved ? u.a + 2 * n : u.a + n, eq = u.interleaved ? ep + 1 : u.b + n;
    const uint64_t axis = AXES ? s_turn[CLO_ROPE_MAX_PAIRS + unit] >> (8 * n) & 0xffu : 0;
    const int64_t at = a.positions ? __ldg(a.positions + axis * p.total_q + row) : pos;
    return rotate_exactly(src[ep], src[eq], (uint64_t)at * s_turn[unit * 8 + n], u.magnitude);
  };
  const float mine = amax;
  amax = over_warps(amax);
  int e = exponent_of(amax);
  if (BITS == 4 && side == 0 && a.rope.plan.rot_dim > 0 && exponent_of(amax * (1.f - kMaxError)) != exponent_of(amax * (1.f + kMaxError))) {
    // fp32 leaves the page's scale open: the largest element once more, exactly
    float m = rotate ? 0.f : mine;
#pragma unroll 1
    for (int i = 0; rotate && i < kUnits * 8; ++i) {
      const int pos = first + (i >> 3) * kPer * kRows;
      if (pos >= hi) break;
      const float2 y = exact_pair(pos, i & 7);
      const float x0 = fabsf(y.x), x1 = fabsf(y.y);
      m = fmaxf(m, fmaxf(x0 < INFINITY ? x0 : 0.f, x1 < INFINITY ? x1 : 0.f));
    }
    // every warp has read the first sums
    if (kPer > 1) asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(kPer * 32) : "memory");
    __syncwarp();
    e = exponent_of(over_warps(m));
  }
  float scale = __int_as_float((e + 127) << 23);
  float* sp = sd.scales + (int64_t)page * p.n_kv_heads + head;
  if (lo > base) {
    const float old = *sp;
    if (old >= scale) {  // a scale that is no number is replaced
      scale = old;
    } else if (old > 0.f) {
      const float f = old / scale;
      if (BITS == 4) {
        // the earlier tokens' group scales, four at a time (a row's are one or two words)
        uint32_t* const words = reinterpret_cast<uint32_t*>(sd.groups + groups_at<D>(p, page, head, 0));
        for (int v = part * 32 + lane; v < (lo - base) * (D / 64); v += kPer * 32) {
          const uint32_t w = words[v];
          const float2 x = e4m3_to_f32x2(w & 0xffffu), y = e4m3_to_f32x2(w >> 16);
          words[v] = pack_e4m3(x.x * f, x.y * f) | pack_e4m3(y.x * f, y.y * f) << 16;
        }
      }
      for (int v = part * 32 + lane; BITS == 8 && v < (lo - base) * (D / 8); v += kPer * 32) {
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
  if constexpr (BITS == 4) {
    const Partners<D> with = partners_of<D>(rotate && !u.interleaved, a.rope.plan.rot_dim, lane);
    uint8_t* const groups = sd.groups + groups_at<D>(p, page, head, 0);
    // One copy of the code for all units: several did not fit the instruction cache (13,600 tokens with queries 144 us for 96).
    auto encode_rows = [&](auto turned) {
      constexpr bool kTurned = decltype(turned)::value;
#pragma unroll 1
      for (int i = 0; i < kUnits && lo + part * kRows + i * kPer * kRows < hi; ++i) {
        const int pos = first + i * kPer * kRows;
        float x[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          x[k] = f[0][k];
#pragma unroll
          for (int n = 1; n < kUnits; ++n) x[k] = i == n ? f[n][k] : x[k];
          x[k] = pos < hi ? x[k] : 0.f;
        }
        Codes4 c;
#pragma unroll 1
        for (bool again = false;; again = true) {
          c = encode_unit<D, kTurned>(x, inv, rotate && !again, u.magnitude == 1.f, u.interleaved, with);
          if (!kTurned || again || !__any_sync(0xffffffffu, c.open != 0)) break;
          // what fp32 left open: those pairs once more, exactly
#pragma unroll 1
          for (; c.open; c.open &= c.open - 1) {
            const int n = __ffs(c.open) - 1;
            const float2 y = exact_pair(pos, n);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (k != n) continue;
              if (u.interleaved) {
                x[2 * k] = y.x;
                x[2 * k + 1] = y.y;
              } else {
                x[k] = y.x;
                x[8 + k] = y.y;
              }
            }
          }
        }
        if (pos < hi) {
          char* dst = dst0 + (int64_t)(pos - base) * sd.stride_token / 2;
          *reinterpret_cast<uint32_t*>(dst + u.a / 2) = c.a;
          *reinterpret_cast<uint32_t*>(dst + u.b / 2) = c.b;
          // the vector with the group's first elements writes its scale
          uint8_t* const g = groups + (pos - base) * (D / 16);
          if (u.a % 16 == 0) g[u.a / 16] = (uint8_t)c.scale_a;
          if (u.b % 16 == 0) g[u.b / 16] = (uint8_t)c.scale_b;
        }
      }
    };
    if (side == 0 && a.rope.plan.rot_dim > 0)
      encode_rows(std::true_type{});
    else
      encode_rows(std::false_type{});
  }
#pragma unroll
  for (int i = 0; BITS == 8 && i < kUnits; ++i) {
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

template <int D, int BITS, int kPer, bool AXES>
__global__ void __launch_bounds__(kThreads, 2) k_paged_append(const AppendParams a) {
  __shared__ __align__(16) uint64_t s_turn[kTurns<AXES>];
  __shared__ float s_red[kWarps];
  stage_turns<AXES>(a.rope, s_turn);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((int)blockIdx.x < a.kv_blocks) {
    const int64_t job = (int64_t)blockIdx.x * (kWarps / kPer) + warp / kPer;
    const int heads = a.c.n_kv_heads;
    const int64_t item = job / (2 * heads);
    if (item >= a.items) return;
    write_page<D, BITS, kPer, AXES>(a, s_turn, (int)item, (int)(job % heads), (int)(job / heads & 1), warp % kPer, lane, s_red, warp / kPer);
    return;
  }
  constexpr int kIters = kPer == 1 ? kShortIters : kLongIters;
  const int64_t job = (int64_t)((int)blockIdx.x - a.kv_blocks) * kWarps + warp;
  const int64_t t = job / a.q_chunks;
  if (t >= a.c.total_q) return;
  // the row's sequence is looked up while its elements are on their way
  auto position = [&](Place<AXES>* where) {
    const int b = seq_of_row(a.c, (int)t, lane);
    if (b >= a.c.batch) return false;
    const SeqRows s = seq_rows(a.c, b);
    if (t - s.first >= s.n) return false;  // beyond max_q: left out, as its key is
    *where = place_of<AXES>(a.rope, a.positions, t, a.c.total_q, (int64_t)s.pos0 + (t - s.first));
    return true;
  };
  rotate_heads<D, kIters, AXES>(a.rope, s_turn, a.q, a.q_out, t, position, (int)(job % a.q_chunks) * heads_per_warp<D>(kIters), a.n_q_heads, lane);
}

template <int BITS>
void launch_append_bits(const AppendParams& a, int head_dim, int64_t blocks, int per, cudaStream_t st) {
  auto launch = [&](auto* one, auto* two, auto* four, auto* eight) { (per == 1 ? one : per == 2 ? two : per == 4 ? four : eight)<<<(unsigned)blocks, kThreads, 0, st>>>(a); };
  if (a.rope.plan.n_axes > 1) {
    if (head_dim == 128) launch(k_paged_append<128, BITS, 1, true>, k_paged_append<128, BITS, 2, true>, k_paged_append<128, BITS, 4, true>, k_paged_append<128, BITS, 8, true>);
    else launch(k_paged_append<64, BITS, 1, true>, k_paged_append<64, BITS, 2, true>, k_paged_append<64, BITS, 4, true>, k_paged_append<64, BITS, 8, true>);
  } else {
    if (head_dim == 128) launch(k_paged_append<128, BITS, 1, false>, k_paged_append<128, BITS, 2, false>, k_paged_append<128, BITS, 4, false>, k_paged_append<128, BITS, 8, false>);
    else launch(k_paged_append<64, BITS, 1, false>, k_paged_append<64, BITS, 2, false>, k_paged_append<64, BITS, 4, false>, k_paged_append<64, BITS, 8, false>);
  }
}

}  // namespace

}  // namespace clo
