// Shared parts of the paged-cache operators: kernel parameters, the phase of a rotary pair,
// e4m3 conversion and the addressing of a ragged batch.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "clo.h"
#include "clo_internal.cuh"

namespace clo {

constexpr int kMinScaleExp = -64;
constexpr float kMinScale = 1e-30f;   // smallest page scale that a reader uses
constexpr int kMaxGroup = 16;         // query heads per kv head
constexpr int64_t kMaxPagedTokens = int64_t(1) << 30;

// One of K or V: pages, scales (8-bit pages) and strides in elements.
struct PagedSide {
  char* pages;
  float* scales;
  int64_t stride_page, stride_head, stride_token;
};

struct PagedParams {
  PagedSide side[2];  // K, V
  const int32_t* q_starts;
  const int32_t* kv_lens;
  const int32_t* table;
  int64_t table_stride;
  int32_t n_pages;
  int32_t max_pages;
  int32_t batch;
  int32_t total_q;
  int32_t max_q;
  int32_t n_kv_heads;
  int32_t page_size;
  int32_t page_shift;
};

// Rows [first, first + n) of the call's tensors belong to sequence b; row i has position pos0 + i.
struct SeqRows {
  int first, n, pos0, kv_len;
};

// The device-side lengths, clamped to the sizes that the host vouches for.
__device__ __forceinline__ SeqRows seq_rows(const PagedParams& p, int b) {
  SeqRows s;
  int a = __ldg(p.q_starts + b), e = __ldg(p.q_starts + b + 1);
  a = min(max(a, 0), p.total_q);
  e = min(max(e, a), p.total_q);
  s.first = a;
  s.n = e - a;
  s.kv_len = min(max(__ldg(p.kv_lens + b), -(1 << 30)), 1 << 30);
  s.pos0 = s.kv_len - s.n;
  s.n = min(s.n, p.max_q);
  s.kv_len = min(max(s.kv_len, 0), p.max_pages << p.page_shift);
  return s;
}

// Page of a position, or -1 where there is none.
__device__ __forceinline__ int page_of(const PagedParams& p, int b, int logical) {
  if (logical < 0 || logical >= p.max_pages) return -1;
  const int id = __ldg(p.table + (int64_t)b * p.table_stride + logical);
  return (unsigned)id < (unsigned)p.n_pages ? id : -1;
}

// Sequence of row t by the whole warp: the number of sequences that end at or before t.
__device__ __forceinline__ int seq_of_row(const PagedParams& p, int t, int lane) {
  int b = 0;
  for (int c = 0; c < p.batch; c += 32) {
    const bool done = c + lane < p.batch && __ldg(p.q_starts + c + lane + 1) <= t;
    const unsigned m = __ballot_sync(0xffffffffu, done);
    b += __popc(m);
    if (m != 0xffffffffu) break;
  }
  return b;
}

// cos and sin of position * turn: the product modulo 2^64 is the angle as a fraction of a turn, so far positions lose nothing.
// Its upper 32 bits go to the nearest quarter turn in integers; the rest, r in [-1/4, 1/4] half turns, is off by 2^-27 at most
// after one rounding to fp32 (the whole angle would be by 2^-25, and more 8-bit codes would differ from an exact rotation's).
// There Taylor's series of sin(pi r) to r^9 and of cos(pi r) to r^10 leave less than 2^-28; results are off by 7.5e-8 at most.
__device__ __forceinline__ float2 rope_cos_sin(int64_t pos, uint64_t turn, float magnitude) {
  const uint32_t lo = (uint32_t)turn, hi = (uint32_t)(turn >> 32);
  const uint32_t plo = (uint32_t)pos, phi = (uint32_t)((uint64_t)pos >> 32);
  const uint32_t frac = __umulhi(plo, lo) + plo * hi + phi * lo;
  const uint32_t quarter = (frac + 0x20000000u) >> 30;
  const float r = (float)(int32_t)(frac - (quarter << 30)) * 4.656612873077393e-10f, r2 = r * r;
  constexpr double kPi = 3.14159265358979323846, kPi2 = kPi * kPi, kPi4 = kPi2 * kPi2;
  constexpr float kPiHi = (float)kPi, kPiLo = (float)(kPi - (double)kPiHi);
  float p = fmaf((float)(kPi4 * kPi4 * kPi / 362880.0), r2, (float)(-kPi4 * kPi2 * kPi / 5040.0));
  p = fmaf(fmaf(p, r2, (float)(kPi4 * kPi / 120.0)), r2, (float)(-kPi2 * kPi / 6.0));
  const float s = fmaf(r, kPiHi, r * fmaf(p, r2, kPiLo));
  float c = fmaf((float)(-kPi4 * kPi4 * kPi2 / 3628800.0), r2, (float)(kPi4 * kPi4 / 40320.0));
  c = fmaf(fmaf(c, r2, (float)(-kPi4 * kPi2 / 720.0)), r2, (float)(kPi4 / 24.0));
  c = fmaf(fmaf(c, r2, (float)(-kPi2 / 2.0)), r2, 1.f);
  float2 y = quarter & 1u ? make_float2(s, c) : make_float2(c, s);
  y.x *= (quarter + 1u) & 2u ? -magnitude : magnitude;
  y.y *= quarter & 2u ? -magnitude : magnitude;
  return y;
}

__device__ __forceinline__ void unpack8(const uint4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Two e4m3 codes of (lo, hi): nearest, ties to even, beyond +-448 (infinities too) to +-448, NaN stays.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 pack8_e4m3(const float* x) {
  return make_uint2(pack_e4m3(x[0], x[1]) | pack_e4m3(x[2], x[3]) << 16, pack_e4m3(x[4], x[5]) | pack_e4m3(x[6], x[7]) << 16);
}
// Two codes as an fp16 pair (exact: e4m3 is a subset of fp16).
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
// Four codes as two fp16 pairs.
__device__ __forceinline__ void e4m3_to_f16x4(uint32_t four, uint32_t* lo, uint32_t* hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(*lo), "=r"(*hi) : "r"(four));
}
__device__ __forceinline__ float2 e4m3_to_f32x2(uint32_t two) {
  const uint32_t h = e4m3_to_f16x2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A sequence's visible tokens for a row at position `pos` are [0, sink_end) and [lo, hi).
struct Visible {
  int sink_end, lo, hi;
};
__device__ __forceinline__ Visible visible_of(int pos, int kv_len, int window, int sinks) {
  Visible v;
  v.hi = min(pos + 1, kv_len);
  v.lo = window > 0 && pos >= window ? pos - window + 1 : 0;
  v.sink_end = min(window > 0 ? sinks : 0, min(v.lo, v.hi));
  return v;
}

struct AttendParams {
  PagedParams c;
  const uint16_t* q;
  uint16_t* out;
  int64_t q_token, q_head, o_token, o_head;
  int32_t group;      // query heads per kv head
  uint32_t group_inv; // ceil(2^32 / group)
  int32_t n_q_heads;
  int32_t window, sinks;
  float scale_log2;   // softmax scale * log2(e)
  int32_t part_rows;  // rows per (sequence, kv head), at most
  float* part;        // the caller's workspace, or null
  int64_t part_bytes;
};

// Row of a unit -> query token, for rows below 2^28 (group <= 16: the product's excess stays below one part in `group`).
__device__ __forceinline__ int token_of_row(const AttendParams& a, int row) {
  return a.group == 1 ? row : (int)__umulhi((uint32_t)row, a.group_inv);
}
// Offset of a unit's row in q-like rows with these strides.
__device__ __forceinline__ int64_t row_offset(const AttendParams& a, int first, int kvh, int row, int64_t stride_token, int64_t stride_head) {
  const int t = token_of_row(a, row);
  return (int64_t)(first + t) * stride_token + (int64_t)(kvh * a.group + row - t * a.group) * stride_head;
}

// Checks a cache and a batch and fills the kernels' view of them; null or what is wrong.
const char* paged_params(const clo_paged_cache* c, const clo_paged_batch* b, PagedParams* p);

// Records a CUDA-side or argument error as the calling thread's error text.
clo_status paged_fail(clo_status st, const char* fmt, ...);

// ---------------------------------------------------------------------------- TMA
// Tensor maps of K and V as [page][head][slot][element] with boxes of `rows` slots and one swizzle span (128
// bytes, or the whole row where that is 64) of elements.
struct PageMaps {
  CUtensorMap side[2];
};
// Null, or what failed.
const char* make_page_maps(const PagedParams& c, int head_dim, int kv_bits, int rows, PageMaps* maps);

// Nonzero in one thread of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}

// Fetches a kernel parameter's tensor map ahead of its first use.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) { asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory"); }

// One box to shared memory; pages outside the map read as zeros.  The instruction takes its operands from uniform registers: lanes that
// issue boxes of their own run one after the other, some 180 cycles each, so one thread issues all of a tile's.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int element, int slot, int head, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(element), "r"(slot), "r"(head), "r"(page), "r"(bar)
      : "memory");
}

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// One try that may suspend the thread for up to 20 us, so that waiting warps leave the issue slots to working ones.
__device__ __forceinline__ bool mbar_try_wait_long(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}

// Bounded wait: false after about two seconds, which no copy or product takes.  The clock is read only after
// many tries (reading it takes longer than most waits).
__device__ __forceinline__ bool mbar_wait_limited(uint64_t* bar, uint32_t parity) {
  if (mbar_test(bar, parity)) return true;
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait_long(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (global_timer_ns() - t0 < 2000000000ull)
    if (mbar_try_wait_long(bar, parity)) return true;
  return false;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace clo
