// Device parts shared by the two attention kernels over paged caches.
#pragma once

#include <atomic>

#include "clo_paged.cuh"

namespace clo {

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

// What becomes of a row's sums.  lost: a wait for a copy or product gave up, so they mean nothing, and the row is NaN whatever else holds
// (computing it again would hide that memory or the launch is broken).  spoilt: V had an infinity or NaN that the row does not see.
enum class RowEnd { store, nan, again };
__host__ __device__ constexpr RowEnd row_end(bool lost, bool spoilt) { return lost ? RowEnd::nan : spoilt ? RowEnd::again : RowEnd::store; }
// The same as a part's mark, for the kernel that joins the parts.
constexpr float kPartSpoilt = 1.f, kPartLost = 2.f;
__host__ __device__ constexpr float part_mark(RowEnd e) { return e == RowEnd::nan ? kPartLost : e == RowEnd::again ? kPartSpoilt : 0.f; }

// Shared-memory address of 16-byte chunk `chunk` of row `row` in a tile of `rows` rows as TMA's swizzle left it.
template <int SPAN>
__device__ __forceinline__ uint32_t swizzled(uint32_t base, int rows, int row, int chunk) {
  constexpr int kChunks = SPAN / 16;
  const int c = chunk % kChunks;
  const int x = SPAN == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3);
  return base + chunk / kChunks * rows * SPAN + row * SPAN + x * 16;
}

// True if one of the two 16-bit values is an infinity or NaN.
template <int BITS>
__device__ __forceinline__ bool not_finite2(uint32_t x) {
  constexpr uint32_t E = BITS == 16 ? 0x7f80u : 0x7c00u;
  return (x & E) == E || ((x >> 16) & E) == E;
}

template <int BITS>
__device__ __forceinline__ bool not_finite16(const uint4 w) {
  if (BITS == 16) return not_finite2<16>(w.x) || not_finite2<16>(w.y) || not_finite2<16>(w.z) || not_finite2<16>(w.w);
  uint32_t nan = 0;  // codes 0x7f and 0xff
#pragma unroll
  for (int i = 0; i < 4; ++i) nan |= __vcmpeq4((i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w) & 0x7f7f7f7fu, 0x7f7f7f7fu);
  return nan != 0;
}

// The tiles that some row of a unit sees: [0, sink_tiles) and [first, first + rest).
struct TileList {
  int sink_tiles, first, rest;
  __device__ __forceinline__ int count() const { return sink_tiles + rest; }
  __device__ __forceinline__ int at(int k) const { return k < sink_tiles ? k : first + k - sink_tiles; }
};
__device__ __forceinline__ TileList tiles_of(int pos_first, int pos_last, int kv_len, int window, int sinks, int tokens) {
  const Visible a = visible_of(pos_first, kv_len, window, sinks), z = visible_of(pos_last, kv_len, window, sinks);
  TileList t;
  t.sink_tiles = t.first = t.rest = 0;
  if (z.hi <= 0) return t;
  // a sink token that the first row sees through its window lies in the second range
  const int sink_end = window > 0 ? min(min(sinks, a.lo), z.hi) : 0;
  t.sink_tiles = (sink_end + tokens - 1) / tokens;
  t.first = max(a.lo / tokens, t.sink_tiles);
  t.rest = max((z.hi + tokens - 1) / tokens - t.first, 0);
  return t;
}

constexpr int kSms = 152;  // GB300

// ---------------------------------------------------------------------------- equal shares
// All units' tiles of tokens, each unit with a constant cost beside them, lie end to end and are cut into equal shares, one to a
// block.  A unit that a cut meets leaves one part per block in the caller's workspace: a record per block, then two
// parts per block (slot 1: of a unit that it begins, slot 0: of one that it ends or passes through), each [row][D elements, maximum,
// sum, mark, -].
struct PartRecord {
  int valid, b, qb, kvh;
  int last;  // the unit's parts are this block's slot 1 and slot 0 of the following ones up to `last`
  int own;   // this block
  int pad[2];
};
constexpr int kRecordBytes = 16384;
constexpr int kMostBlocks = 2 * kSms;
static_assert(kMostBlocks * sizeof(PartRecord) <= kRecordBytes, "records fit");

inline int64_t part_bytes(int blocks, int rows, int d) { return kRecordBytes + 2 * (int64_t)blocks * rows * (d + 4) * 4; }
__device__ __forceinline__ float* part_of(const AttendParams& a, int block, int slot, int rows, int d) {
  return a.part + kRecordBytes / 4 + (2 * (int64_t)block + slot) * rows * (d + 4);
}
__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sets a kernel's shared-memory size, once per device (`prepared`: a bit each).
cudaError_t prepare_kernel(const void* f, int smem, std::atomic<uint64_t>* prepared);

// A launch that may begin while the stream's previous kernel drains; the kernel waits for it (griddepcontrol.wait).
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*f)(Params...), dim3 grid, int threads, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, args...);
}

cudaError_t launch_attend_few_bf16(const AttendParams& a, int head_dim, cudaStream_t st);
cudaError_t launch_attend_few_e4m3(const AttendParams& a, int head_dim, cudaStream_t st);
int64_t attend_few_bf16_bytes(const AttendParams& a, int head_dim);
int64_t attend_few_e4m3_bytes(const AttendParams& a, int head_dim);
cudaError_t launch_attend_many(const AttendParams& a, int head_dim, int kv_bits, cudaStream_t st);
int64_t attend_many_bytes(const AttendParams& a, int head_dim);

}  // namespace clo
