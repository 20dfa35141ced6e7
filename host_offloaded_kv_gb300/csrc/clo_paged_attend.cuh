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
    if (BITS == 4) {
      uint32_t h[4];
      e2m1_to_f16x8(reinterpret_cast<const uint8_t*>(sd.pages)[at >> 1] >> (e & 1 ? 4 : 0), h);
      const float g = e4m3_to_f32x2(sd.groups[groups_at<D>(p, page, kvh, slot) + e / 16]).x;
      return __half22float2(*reinterpret_cast<const __half2*>(h)).x * g * fmaxf(sd.scales[(int64_t)page * p.n_kv_heads + kvh], kMinScale);
    }
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
// The same as a part's mark, for the kernel that joins the parts; kPartSeen: no finite number, and rightly.
constexpr float kPartSpoilt = 1.f, kPartLost = 2.f, kPartSeen = 3.f;
__host__ __device__ constexpr float part_mark(RowEnd e) { return e == RowEnd::nan ? kPartLost : e == RowEnd::again ? kPartSpoilt : 0.f; }

// Shared-memory address of 16-byte chunk `chunk` of row `row` in a tile of `rows` rows as TMA's swizzle left it.
template <int SPAN>
__device__ __forceinline__ uint32_t swizzled(uint32_t base, int rows, int row, int chunk) {
  constexpr int kChunks = SPAN / 16;
  const int c = chunk % kChunks;
  const int x = SPAN == 128 ? c ^ (row & 7) : SPAN == 64 ? c ^ ((row >> 1) & 3) : c ^ ((row >> 2) & 1);
  return base + chunk / kChunks * rows * SPAN + row * SPAN + x * 16;
}

// True if one of the two 16-bit values is an infinity or NaN.
template <int BITS>
__device__ __forceinline__ bool not_finite2(uint32_t x) {
  constexpr uint32_t E = BITS == 16 ? 0x7f80u : 0x7c00u;
  return (x & E) == E || ((x >> 16) & E) == E;
}

// True if one of four e4m3 codes is NaN (0x7f or 0xff).
__device__ __forceinline__ bool e4m3_nan4(uint32_t x) { return __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0; }

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

// Which of a warp's rows have to be computed again, of those (`want`, a lane each, at position `pos`) whose sums over the tiles [k0, k1)
// of `tl` are no finite numbers.  What a row sees may make it so, and stays: only where V has an infinity or NaN in a token of the tiles that
// the row does not see (zero times it is NaN), or where what it sees can pass fp32's range in the unnormalised sums alone
// (weights up to 2^15, 2^30 tokens: values from 2^80 on, scales below 2^-80), the row's sums are wrong.  So they are where an infinity
// had a weight too small for fp32: a NaN (`nan`) without one in V.  One look over V, up to eight loads of a warp in flight.
template <int D, int BITS>
__device__ __forceinline__ bool spoilt_rows(const AttendParams& a, int b, int kvh, const SeqRows& s, const TileList& tl, int k0, int k1, int tokens, int hi,
                                            bool want, int pos, bool nan, int lane) {
  const PagedParams& p = a.c;
  const PagedSide& sd = p.side[1];
  constexpr int kLanes = D * BITS / 64, kPer = 32 / kLanes;  // lanes of a row (8 bytes each), rows of a load; 4-bit pages have no use of these
  constexpr int kBatch = 16 / kPer < 8 ? 16 / kPer : 8;  // loads in flight
  constexpr uint32_t kRow = kLanes == 32 ? 0xffffffffu : (1u << kLanes) - 1u;
  bool spoilt = false, saw_nan = false, saw_inf = false;
  const int groups = k1 * (tokens / 16);
  for (int g0 = k0 * (tokens / 16); g0 < groups; g0 += 32) {
    auto first_of = [&](int g) { return tl.at(g * 16 / tokens) * tokens + g * 16 % tokens; };
    const int mine = g0 + lane < groups ? page_of(p, b, first_of(g0 + lane) >> p.page_shift) : -1;
    for (int g = g0; g < min(g0 + 32, groups); ++g) {
      const int page = __shfl_sync(0xffffffffu, mine, g - g0), j0 = first_of(g);
      if (page < 0 || j0 >= hi) continue;
      if constexpr (BITS == 4) {
        // codes are finite: a lane per token looks at its group scales
        const int64_t at = groups_at<D>(p, page, kvh, (j0 + (lane & 15)) & (p.page_size - 1));
        uint32_t w[2] = {0u, 0u};
        if (j0 + (lane & 15) < hi) {
          w[0] = __ldg(reinterpret_cast<const uint32_t*>(sd.groups + at));
          if (D == 128) w[1] = __ldg(reinterpret_cast<const uint32_t*>(sd.groups + at + 4));
        }
        const uint32_t nans = __ballot_sync(0xffffffffu, e4m3_nan4(w[0]) || e4m3_nan4(w[1])) & 0xffffu;
        const bool large = !(sd.scales[(int64_t)page * p.n_kv_heads + kvh] >= 0x1p-80f);
        if (nans || large) {
#pragma unroll 1
          for (int r = 0; r < 16 && j0 + r < hi; ++r) {
            const int j = j0 + r;
            const bool n = nans >> r & 1u, see = j <= pos && j < s.kv_len && (a.window == 0 || j > pos - a.window || j < a.sinks);
            spoilt |= see ? large : n;
            saw_nan |= see && n;
          }
        }
        if (!__any_sync(0xffffffffu, want && !spoilt)) return want;
        continue;
      }
      const char* src = sd.pages + ((int64_t)page * sd.stride_page + (int64_t)kvh * sd.stride_head) * (BITS / 8) + lane % kLanes * 8;
      const bool small_scale = BITS == 8 && !(sd.scales[(int64_t)page * p.n_kv_heads + kvh] >= 0x1p-80f);
#pragma unroll 1
      for (int i0 = 0; i0 < 16; i0 += kPer * kBatch) {
        uint2 w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int j = j0 + i0 + i * kPer + lane / kLanes;
          w[i] = j < hi ? __ldg(reinterpret_cast<const uint2*>(src + (int64_t)(j & (p.page_size - 1)) * sd.stride_token * (BITS / 8))) : make_uint2(0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          bool is_nan = false, is_inf = false, large = small_scale;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t x = k ? w[i].y : w[i].x;
            if (BITS == 8) {
              is_nan |= __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
            } else {
              const uint32_t lo = x & 0x7fffu, up = x >> 16 & 0x7fffu;
              is_nan |= max(lo, up) > 0x7f80u;
              is_inf |= lo == 0x7f80u || up == 0x7f80u;
              large |= (lo >= (127u + 80u) << 7 && lo < 0x7f80u) || (up >= (127u + 80u) << 7 && up < 0x7f80u);
            }
          }
          const uint32_t nans = __ballot_sync(0xffffffffu, is_nan), infs = __ballot_sync(0xffffffffu, is_inf), larges = __ballot_sync(0xffffffffu, large);
          if (!(nans | infs | larges)) continue;
#pragma unroll 1
          for (int r = 0; r < kPer; ++r) {
            const int j = j0 + i0 + i * kPer + r;
            if (j >= hi) break;
            const bool n = nans >> (r * kLanes) & kRow, f = infs >> (r * kLanes) & kRow, l = larges >> (r * kLanes) & kRow;
            const bool see = j <= pos && j < s.kv_len && (a.window == 0 || j > pos - a.window || j < a.sinks);
            spoilt |= see ? l : n || f;
            saw_nan |= see && n;
            saw_inf |= see && f;
          }
        }
      }
      if (!__any_sync(0xffffffffu, want && !spoilt)) return want;
    }
  }
  return want && (spoilt || (nan && saw_inf && !saw_nan));
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
constexpr int kRecordBytes = 20480;
constexpr int kMostBlocks = 4 * kSms;
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
cudaError_t launch_attend_few_e2m1(const AttendParams& a, int head_dim, cudaStream_t st);
int64_t attend_few_e2m1_bytes(const AttendParams& a, int head_dim);
int64_t attend_few_bf16_bytes(const AttendParams& a, int head_dim);
int64_t attend_few_e4m3_bytes(const AttendParams& a, int head_dim);
cudaError_t launch_attend_many(const AttendParams& a, int head_dim, int kv_bits, cudaStream_t st);
cudaError_t launch_attend_many_e4m3(const AttendParams& a, int head_dim, cudaStream_t st);
cudaError_t launch_attend_many_e2m1(const AttendParams& a, int head_dim, cudaStream_t st);
int64_t attend_many_bytes(const AttendParams& a, int head_dim);

}  // namespace clo
