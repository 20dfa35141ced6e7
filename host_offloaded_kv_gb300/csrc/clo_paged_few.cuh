// Attention of few rows per kv head over a paged cache (decode steps): the kernel and its launch, instantiated by type.
#pragma once

#include <algorithm>
#include <type_traits>

#include "clo_paged_attend.cuh"

namespace clo {
namespace {

// Decode: the rows of a (sequence, kv head) unit, at most 8 * NT of them, read every visible K and V row once, so HBM
// bounds the kernel and the products run on mma.sync m16n8k16 fragments: S^T = K Q^T (16 tokens by 8 rows), O^T = V^T P^T
// (16 elements by 8 rows), which waste none of the 16-wide side on absent rows; the weights pass from one product to the next
// with movmatrix.
//
// Each warp owns a ring of kStages 8 KB stages (16 tokens of bf16 K and V rows of 128, 64 tokens of 8-bit rows of 64) that it
// fills with TMA boxes (4-bit pages: 64 tokens and their group scales), so no warp waits for another before a unit's end, where they join through shared memory.
//
// All units' tiles are cut into equal shares, one per block of a single wave, so that ragged batches load the SMs alike and one
// long sequence fills the GPU; a second kernel joins what the cuts met.  Without a workspace units stay whole.  (Clusters that
// join through distributed shared memory were slower: 12 us for 6 at 8 x 200 tokens, and 16 blocks of a cluster find room only 7
// times on the SMs.)
//
// 8 sequences of 32,768 tokens of bf16, 32 over 8 heads of 128: 162 to 166 us, 6.6 TB/s, 97 % of a copy's rate; of 8-bit pages 89 us,
// 6.0 TB/s, where the conversions of the codes take issue slots too; of 4-bit pages 70 us, 4.3 TB/s: 320 instructions for 16 tokens of K and
// V, of which 80 conversions, 64 products with the groups' scales and 40 permutes take two cycles each, bound it (the copies alone: 50 us).  One token over 64 tokens, in a graph: 3.5 us, a launch and four
// loads that wait for each other (lengths, page, K, V).
constexpr int kStageBytes = 8192;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

// Two stages and two blocks to an SM.  Three stages keep more copies in flight than the memory answers well: 8 x 32,768 tokens of
// bf16 166 us for 163, one sequence of 524,288 tokens of 8-bit pages 173 us for 165, 64 sequences of 64-element heads 27 us for 22.
// Three blocks with 8-bit pages: 170 us and more for 165.
constexpr int kStages = 2;

// Blocks to an SM.  4-bit pages: conversions, scales and products take more issue slots than the memory takes time, so more warps are wanted:
// 8 x 32,768 tokens, us: two blocks 76, three 70.  Four with one stage to a warp, K and V refilled apart, 74; with tiles of 32 tokens 84.
template <int D, int BITS, int NT>
constexpr int kPerSm = BITS == 4 && !(D == 128 && NT == 2) && NT < 3 ? 3 : 2;
template <int D, int BITS, int NT>
constexpr int kWave = kPerSm<D, BITS, NT> * kSms;
// Calls whose units stay whole have a block each, in as many waves as the residency makes.  Bounded to 168 registers, three blocks are faster where
// they save a wave and slower where they do not, 8 kv heads, us (bf16, heads of 128, 4 rows; 12 rows; 8-bit pages, heads of 64, 12 rows):
//   two blocks / three   45 sequences of 1200 tokens 46.7 / 36.9; 128 of 300 46.5 / 44.5; 39 of 300 13.9 / 9.2
//                        64 of 1200 52.7 / 58.2; 64 of 1000 51.6 / 65.6; 64 of 300 15.0 / 16.5
// Where two blocks leave the compiler below that count by itself (one fragment of rows over 8-bit pages or with heads of 64), three run anyway.
template <int D, int BITS, int NT>
constexpr bool kThirdBlock = BITS != 4 && (NT > 1 || (D == 128 && BITS == 16));
constexpr bool third_block_pays(int64_t units) { return (units + 3 * kSms - 1) / (3 * kSms) < (units + 2 * kSms - 1) / (2 * kSms); }

// 8-bit pages: weights up to 2^14 (fp16 then holds them down to 2^-38 of the largest) are divided by their page's V scale, which may be as
// small as 1e-30, before they are summed.  The sums are kept 2^7 smaller, so that two million such weights stay in fp32's range; the
// reciprocal of the largest scale, 2^-135 then, still has 14 bits.
constexpr float kSumDown = 0x1p-7f;

template <int D, int BITS>
struct Tile {
  static constexpr int kRowBytes = D * BITS / 8;
  static constexpr int kSpan = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a row in one swizzled block
  static constexpr int kSpans = kRowBytes / kSpan;
  static constexpr int kTokens = BITS == 4 ? 64 : kStageBytes / (2 * kRowBytes);
  static constexpr int kM = kTokens / 16;
  static constexpr int kSideBytes = kTokens * kRowBytes;
  static constexpr int kGroupBytes = BITS == 4 ? kTokens * (D / 16) : 0;  // group scales, of K and then of V, behind the codes
  static constexpr int kStage = 2 * (kSideBytes + kGroupBytes);
  static constexpr int kSmem = kWarps * kStages * kStage + 1024;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// One, two or four words at once.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t* w) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <int BITS>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (BITS == 16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// c / x for positive x, without a branch and into the subnormal numbers: the hardware's reciprocal (off by one unit in the last place) flushes
// those of x above 2^126.
__device__ __forceinline__ float reciprocal(float x, float c) {
  const float k = x >= 0x1p64f ? 0x1p-32f : 1.f;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * k));
  return r * (k * c);
}

// Longest units, in tiles, that are left whole (no shares to find, no join): where there are fewer units than SMs, and where
// there are more.  Measured, whole against cut, us: 64 units of up to 12 tiles 6.5 / 11.8, 8 of 32 tiles 12.6 / 7.6; 256 units of
// 10 to 19 tiles 8.3 / 14.2, of 63 to 125 tiles 36.6 / 40.6, of 32 to 500 tiles 103 / 94 (8-bit pages, 16 to 250 tiles: 80 / 59).
// 4-bit pages, whose tiles hold 64 tokens and take longer, whole / cut: 8 sequences of 600 tokens, 8 heads 10.5 / 12.4, one of 2000 - / 12.4; 32 of
// 2500 30.9 / 37.5, 32 to 8000 72.6 / 49.6, 61 windows of 4096 80.4 / 74.1.
template <int BITS>
constexpr int kWholeFew = BITS == 4 ? 12 : 24;
template <int BITS>
constexpr int kWholeMany = BITS == 4 ? 48 : 128;
// What a unit costs beside its tiles, in tiles, and the least share of a block.  Cost 4 / 14 / 20, us: 61 windows of 4096 tokens of
// 8-bit pages 96.0 / 87.8 / 87.5, 32 sequences to 8000 tokens 59.5 / 53.8 / 54.0 (bf16: 94.2 / 91.1 / 91.3).
// Share 14 / 8 / 5, us: one sequence of 512 tokens 8.8 / 7.6 / 7.4, of 2000 9.3 / 8.6 / 9.0, of 8000 of 8-bit pages 12.4 / 11.2 / 11.1.
// 4-bit pages, share 8 / 4: one sequence of 8000 tokens 14.5 / 13.3; the cost makes no difference there (4, 8, 14, 22: 80.6 to 81.1 for the windows).
constexpr int kFewCost = 14;
template <int BITS>
constexpr int kFewShare = BITS == 4 ? 4 : 8;

// A block's share, and the unit that it begins in.
struct FewShare {
  int64_t first, last;
  int64_t base;  // where that unit begins
  int b, kvh;
};

// By every warp of the block.  Lanes take four sequences each.
template <int BITS>
__device__ __forceinline__ FewShare few_share(const AttendParams& a, int tokens, int lane) {
  const PagedParams& p = a.c;
  constexpr int kPer = 4;
  FewShare f;
  f.base = -1;
  f.b = f.kvh = 0;
  int cost[kPer];
  auto costs = [&](int c) {
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = c + lane * kPer + i;
      cost[i] = 0;
      if (b < p.batch) {
        const SeqRows s = seq_rows(p, b);
        if (s.n > 0) cost[i] = tiles_of(s.pos0, s.pos0 + s.n - 1, s.kv_len, a.window, a.sinks, tokens).count() + kFewCost;
      }
      sum += cost[i];
    }
    return (int64_t)sum;
  };
  int64_t mine = 0, total = 0;
  for (int c = 0; c < p.batch; c += 32 * kPer) {
    mine = costs(c);
    total += warp_sum64(mine);
  }
  total *= p.n_kv_heads;
  const int64_t share = max((total + gridDim.x - 1) / gridDim.x, (int64_t)kFewShare<BITS>);
  f.first = min(total, share * blockIdx.x);
  f.last = min(total, f.first + share);
  if (f.first >= f.last) return f;
  int64_t before = 0;
  for (int c = 0; c < p.batch; c += 32 * kPer) {
    if (p.batch > 32 * kPer) mine = costs(c);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned m = __ballot_sync(0xffffffffu, before + incl * p.n_kv_heads > f.first);
    if (m) {
      const int l = __ffs(m) - 1;
      int64_t at = before + (incl - mine) * p.n_kv_heads;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int64_t all = (int64_t)cost[i] * p.n_kv_heads;
        if (f.base < 0 && f.first < at + all && f.first >= at) {
          f.b = c + lane * kPer + i;
          f.kvh = (int)((f.first - at) / cost[i]);
          f.base = at + (int64_t)f.kvh * cost[i];
        }
        at += all;
      }
      f.b = __shfl_sync(0xffffffffu, f.b, l);
      f.kvh = __shfl_sync(0xffffffffu, f.kvh, l);
      f.base = __shfl_sync(0xffffffffu, f.base, l);
      return f;
    }
    before += __shfl_sync(0xffffffffu, incl, 31) * p.n_kv_heads;
  }
  return f;
}

template <int D, int BITS, int NT, int PER_SM>
__global__ void __launch_bounds__(kThreads, PER_SM) k_attend_few(const AttendParams a, const __grid_constant__ PageMaps maps) {
  using T = Tile<D, BITS>;
  constexpr int TOK = T::kTokens, KM = T::kM, KD = D / 16, ROWS = 8 * NT;
  constexpr float kOff = BITS == 16 ? 0.f : 14.f, kDown = BITS == 16 ? 1.f : kSumDown;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_full[kWarps][kStages];
  __shared__ __align__(16) float s_scale[kWarps][kStages][2][4];
  __shared__ uint32_t s_there[kWarps][kStages];
  __shared__ float s_m[kWarps][ROWS], s_l[kWarps][ROWS];
  __shared__ float s_cm[ROWS], s_cl[ROWS];
  __shared__ int s_odd, s_dead;

  const PagedParams& p = a.c;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t ring = smem + warp * kStages * T::kStage;
  uint8_t* const generic = smem_raw + (smem - smem_u32(smem_raw));
  FewShare share{0, 1, 0, (int)blockIdx.x, (int)blockIdx.y};
  if (a.part) share = few_share<BITS>(a, TOK, lane);
  int kvh = share.kvh, b = share.b;
  SeqRows s = seq_rows(p, b);
  if (tid == 0) s_odd = s_dead = 0;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) mbar_init(&s_full[warp][i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();

  const bool by_unit = (int64_t)p.batch * p.n_kv_heads <= kWave<D, BITS, NT>;  // where a unit's record stands
  PartRecord* const records = reinterpret_cast<PartRecord*>(a.part);
  if (tid == 0 && a.part && !by_unit) records[blockIdx.x].valid = 0;
  int st = 0;          // next stage, and its barrier's phase
  uint32_t phase = 0;
  int64_t base = share.first < share.last ? share.base : share.last;
  auto next_seq = [&]() {
    if (++b < p.batch) s = seq_rows(p, b);
  };
  auto next = [&](int64_t end) {
    base = end;
    if (++kvh == p.n_kv_heads) {
      kvh = 0;
      next_seq();
    }
  };
  while (base < share.last && b < p.batch) {
    const int rows = s.n * a.group;
    if (rows == 0) {
      if (!a.part) break;  // whole units have a block each: the next sequence's is not this one's
      next_seq();
      continue;
    }
    const TileList tl = tiles_of(s.pos0, s.pos0 + s.n - 1, s.kv_len, a.window, a.sinks, TOK);
    // this block's part of the unit
    const int all = tl.count();
    const int64_t end = base + (a.part ? all + kFewCost : 1);
    int t_begin = 0, n = all;
    bool part_here = base >= share.first;
    if (a.part && all > 0) {
      t_begin = base >= share.first ? 0 : max((int)(share.first - base) - kFewCost, 0);
      n = (end <= share.last ? all : max((int)(share.last - base) - kFewCost, 0)) - t_begin;
      part_here = n > 0;
    }
    const bool full = n == all;
    if (!part_here) {
      next(end);
      continue;
    }
    if (tid == 0 && a.part && t_begin == 0) {
      const PartRecord r{!full, b, 0, kvh, full ? 0 : (int)((end - 1) / (share.last - share.first)), (int)blockIdx.x};
      if (by_unit || !full) records[by_unit ? b * p.n_kv_heads + kvh : blockIdx.x] = r;
    }
    constexpr int stride = kWarps;
    const int k0 = t_begin + warp, n_tiles = t_begin + n;

    // Page of 16-token group `lane` of tile k, for the lanes below KM (the others: -1).
    auto page_for = [&](int k) {
      return lane < KM && k < n_tiles ? page_of(p, b, (tl.at(k) * TOK + lane * 16) >> p.page_shift) : -1;
    };
    auto issue = [&](int k, int page, int st) {
      const unsigned there = __ballot_sync(0xffffffffu, page >= 0);
      if (BITS != 16 && page >= 0) {  // lanes below KM
        const int64_t at = (int64_t)page * p.n_kv_heads + kvh;
#pragma unroll
        for (int side = 0; side < 2; ++side)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&s_scale[warp][st][side][lane])), "l"(p.side[side].scales + at) : "memory");
      }
      const int box = min(p.page_size, TOK), first = tl.at(k) * TOK;
      const uint32_t dst = ring + st * T::kStage, bar = smem_u32(&s_full[warp][st]);
      int id[KM];
#pragma unroll
      for (int g = 0; g < KM; ++g) id[g] = __shfl_sync(0xffffffffu, page, g);
      if constexpr (BITS == 4) {
        // group scales, 16 bytes a lane: of both sides at once where half the lanes hold a side's
        constexpr int kLanes = T::kGroupBytes / 16, kLaneTokens = TOK / kLanes;
        const int l = lane % kLanes, mine = __shfl_sync(0xffffffffu, page, l * kLaneTokens / 16), slot = (first + l * kLaneTokens) & (p.page_size - 1);
#pragma unroll
        for (int side = lane / kLanes; side < 2; side += 32 / kLanes)
          copy_groups<D>(dst + 2 * T::kSideBytes + side * T::kGroupBytes + l * 16, p, side ? p.side[1].groups : p.side[0].groups, mine, kvh, slot);
      }
      if (elect_one()) {
        s_there[warp][st] = there;
        mbar_arrive_expect_tx(&s_full[warp][st], 2 * T::kSideBytes);
        auto fetch = [&](int g, int page) {
          const int slot = (first + g * 16) & (p.page_size - 1);
#pragma unroll
          for (int side = 0; side < 2; ++side)
#pragma unroll
            for (int h = 0; h < T::kSpans; ++h)
              tma_box(dst + side * T::kSideBytes + h * TOK * T::kSpan + g * 16 * T::kSpan, &maps.side[side], h * (T::kSpan * 8 / BITS), slot, kvh, page, bar);
        };
        if (BITS == 4 && box == TOK) {
          fetch(0, id[0]);
        } else {
#pragma unroll
          for (int g = 0; g < KM; ++g)
            if ((g * 16 & (box - 1)) == 0) fetch(g, id[g]);
        }
      }
      __syncwarp();
      if (BITS != 16) cp_async_commit();
    };

    const bool dead = __any_sync(0xffffffffu, s_dead != 0);  // a copy was lost: the rest of the share is NaN
    int page_next[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) page_next[i] = page_for(k0 + i * stride);
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      if (k0 + i * stride < n_tiles && !dead) issue(k0 + i * stride, page_next[i], st + i < kStages ? st + i : st + i - kStages);
      else if (BITS != 16) cp_async_commit();
    }
    int page_ahead = page_for(k0 + kStages * stride);

    // Q^T fragments: column (row of the unit) nt * 8 + g.  bf16: elements kk * 16 + 2 t4 + {0, 1} and + 8.  8-bit pages: the lane's
    // four codes of a 16-element chunk are neighbours, so elements kk * 16 + 4 t4 + {0, 1} and {2, 3}; 4-bit pages: its eight codes of 32
    // elements, shared by two products; q in fp16, scaled by a power of two that puts the row's largest finite element into [2^14, 2^15).
    uint32_t qf[NT][KD][2];
    float fac[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
      const uint16_t* qp = a.q + row_offset(a, s.first, kvh, r, a.q_token, a.q_head);
      float row_fac = a.scale_log2;
      if (BITS == 16) {
#pragma unroll
        for (int kk = 0; kk < KD; ++kk) {
          qf[nt][kk][0] = r < rows ? *reinterpret_cast<const uint32_t*>(qp + kk * 16 + 2 * t4) : 0u;
          qf[nt][kk][1] = r < rows ? *reinterpret_cast<const uint32_t*>(qp + kk * 16 + 2 * t4 + 8) : 0u;
        }
      } else {
        uint2 raw[KD];
        float mx = 0.f;
#pragma unroll
        for (int kk = 0; kk < KD; ++kk) {
          raw[kk] = r < rows ? *reinterpret_cast<const uint2*>(qp + (BITS == 4 ? kk / 2 * 32 + 8 * t4 + kk % 2 * 4 : kk * 16 + 4 * t4)) : make_uint2(0u, 0u);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w = i < 2 ? raw[kk].x : raw[kk].y;
            const float v = fabsf(__uint_as_float(i & 1 ? w & 0xffff0000u : w << 16));
            mx = fmaxf(mx, v < INFINITY ? v : 0.f);
          }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127 - 14, -100), 112);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        row_fac *= __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int kk = 0; kk < KD; ++kk) {
          qf[nt][kk][0] = pack_f16(__uint_as_float(raw[kk].x << 16) * down, __uint_as_float(raw[kk].x & 0xffff0000u) * down);
          qf[nt][kk][1] = pack_f16(__uint_as_float(raw[kk].y << 16) * down, __uint_as_float(raw[kk].y & 0xffff0000u) * down);
        }
      }
      fac[nt][0] = __shfl_sync(0xffffffffu, row_fac, 8 * t4);
      fac[nt][1] = __shfl_sync(0xffffffffu, row_fac, 8 * t4 + 4);
    }

    float acc[KD][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[nt][i] = -INFINITY;
        l[nt][i] = 0.f;
      }
#pragma unroll
      for (int dt = 0; dt < KD; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[dt][nt][i] = 0.f;
    }
    const Visible va = visible_of(s.pos0, s.kv_len, a.window, a.sinks);
    const Visible vz = visible_of(s.pos0 + s.n - 1, s.kv_len, a.window, a.sinks);
    bool odd = false, ok = !dead;

    for (int k = k0; k < n_tiles && ok; k += stride) {
      if (BITS != 16) cp_async_wait<kStages - 1>();
      __syncwarp();
      ok = mbar_wait_limited(&s_full[warp][st], phase);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      const uint32_t kb = ring + st * T::kStage, vb = kb + T::kSideBytes;
      const int j0 = tl.at(k) * TOK;
      const uint32_t there = s_there[warp][st];
      // every row sees the whole tile
      // V of tokens that no row sees is cleared: its weight is zero, but zero times NaN is not.  What only some rows see
      // is looked over for the same reason.
      const bool whole = there == (1u << KM) - 1u && j0 + TOK <= va.hi && (j0 >= vz.lo || j0 + TOK <= (a.window > 0 ? a.sinks : 0));

      if (BITS == 4 && !whole) {
        // codes are finite: clearing a token's group scales clears its V
        constexpr int kWords = D / 64;
#pragma unroll 1
        for (int i = lane; i < TOK * kWords; i += 32) {
          const int r = i / kWords, j = j0 + r;
          const bool any = (there >> (r >> 4) & 1u) && j < vz.hi && (j >= va.lo || j < (a.window > 0 ? a.sinks : 0));
          uint32_t* at = reinterpret_cast<uint32_t*>(generic + (vb - smem) + T::kSideBytes + T::kGroupBytes) + i;
          if (!any)
            *at = 0u;
          else if (s.n > 1)
            odd |= e4m3_nan4(*at);
        }
        __syncwarp();
      } else if (!whole) {
        constexpr int kChunks = T::kRowBytes / 16;
#pragma unroll 1
        for (int i = lane; i < TOK * kChunks; i += 32) {
          const int r = i / kChunks, j = j0 + r;
          const bool any = (there >> (r >> 4) & 1u) && j < vz.hi && (j >= va.lo || j < (a.window > 0 ? a.sinks : 0));
          uint4* at = reinterpret_cast<uint4*>(generic + (swizzled<T::kSpan>(vb, TOK, r, i % kChunks) - smem));
          if (!any)
            *at = make_uint4(0, 0, 0, 0);
          else if (s.n > 1)
            odd |= not_finite16<BITS>(*at);
        }
        __syncwarp();
      }

      float my_ks = 1.f, my_lvs = 0.f, my_inv = 1.f;  // page scales: a lane per 16 tokens
      if (BITS != 16) {
        my_ks = fmaxf(s_scale[warp][st][0][lane & (KM - 1)], kMinScale);
        const float vs = fmaxf(s_scale[warp][st][1][lane & (KM - 1)], kMinScale);
        my_lvs = __log2f(vs);
        my_inv = reciprocal(vs, kDown);
      }
      float sc[KM][NT][4];
#pragma unroll
      for (int mt = 0; mt < KM; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[mt][nt][i] = 0.f;
        if (BITS == 16) {
#pragma unroll
          for (int kk = 0; kk < KD; ++kk) {
            uint32_t f[4];
            ldsm4(swizzled<T::kSpan>(kb, TOK, mt * 16 + (lane & 15), kk * 2 + (lane >> 4)), f);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<BITS>(sc[mt][nt], f, qf[nt][kk][0], qf[nt][kk][1]);
          }
        } else if (BITS == 4) {
          // A lane holds eight codes of 32 elements of tokens g and g + 8 (the pairs of two products) and the scale of the group they are in.
          const uint32_t gs = kb + 2 * T::kSideBytes + (mt * 16 + g) * (D / 16), pick = t4 < 2 ? 0x2200u : 0x3311u;
          uint32_t sw[2][D / 64];
#pragma unroll
          for (int h = 0; h < 2; ++h) lds_words<D / 64>(gs + h * 8 * (D / 16), sw[h]);
#pragma unroll
          for (int c = 0; c < D / 32; c += 2) {
            uint32_t r[4], sg[2][2];  // [token g, g + 8][chunk]: the scale, twice
            ldsm4(swizzled<T::kSpan>(kb, TOK, mt * 16 + (lane & 15), c + (lane >> 4)), r);
#pragma unroll
            for (int h = 0; h < 2; ++h) e4m3_to_f16x4(__byte_perm(sw[h][c / 2], 0u, pick), &sg[h][0], &sg[h][1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t x[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                e2m1_to_f16x8(r[2 * i + h], x[h]);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[h][e] = mul_f16x2(x[h][e], sg[h][i]);
              }
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t f[4] = {x[0][2 * j], x[1][2 * j], x[0][2 * j + 1], x[1][2 * j + 1]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma16816<BITS>(sc[mt][nt], f, qf[nt][2 * (c + i) + j][0], qf[nt][2 * (c + i) + j][1]);
              }
            }
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < KD; kk += 2) {
            uint32_t r[4];
            ldsm4(swizzled<T::kSpan>(kb, TOK, mt * 16 + (lane & 15), kk + (lane >> 4)), r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t f[4];
              e4m3_to_f16x4(r[2 * i], &f[0], &f[2]);
              e4m3_to_f16x4(r[2 * i + 1], &f[1], &f[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<BITS>(sc[mt][nt], f, qf[nt][kk + i][0], qf[nt][kk + i][1]);
            }
          }
        }
      }

      // Scores in log2 units.  8-bit and 4-bit pages: the page's V scale joins the exponent, so that the weights times the codes keep the
      // accumulator in range, and leaves the sum by its reciprocal.
      auto hide = [&](int mt, int nt, int i) {
        const int j = j0 + mt * 16 + g + (i >> 1) * 8;
        const int pos = s.pos0 + token_of_row(a, nt * 8 + 2 * t4 + (i & 1));
        const bool see = (there >> mt & 1u) && j <= pos && j < s.kv_len && (a.window == 0 || j > pos - a.window || j < a.sinks);
        if (!see) sc[mt][nt][i] = -INFINITY;
      };
      float inv_vs[KM];
#pragma unroll
      for (int mt = 0; mt < KM; ++mt) {
        float ks = 1.f, lvs = 0.f;
        inv_vs[mt] = 1.f;
        if (BITS != 16) {
          ks = __shfl_sync(0xffffffffu, my_ks, mt);
          lvs = __shfl_sync(0xffffffffu, my_lvs, mt);
          inv_vs[mt] = __shfl_sync(0xffffffffu, my_inv, mt);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float f = fac[nt][i & 1] * ks;
            sc[mt][nt][i] = BITS != 16 ? fmaf(sc[mt][nt][i], f, lvs) : sc[mt][nt][i] * f;
            if (BITS == 16 && !whole) hide(mt, nt, i);
          }
      }
      if (BITS != 16 && !whole) {  // (in the loop above: a branch for each score; 8-bit pages, 524,288 tokens: 168 us for 166)
#pragma unroll
        for (int mt = 0; mt < KM; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) hide(mt, nt, i);
      }
      uint32_t pf[KM][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float keep[2], ref[2];
        bool moved = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = sc[0][nt][i];
#pragma unroll
          for (int mt = 0; mt < KM; ++mt) mx = fmaxf(mx, fmaxf(sc[mt][nt][i], sc[mt][nt][i + 2]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float mn = fmaxf(m[nt][i], mx);
          moved |= mn != m[nt][i];
          keep[i] = m[nt][i] == mn ? 1.f : exp2_fast(m[nt][i] - mn);
          m[nt][i] = mn;
          ref[i] = mn == -INFINITY ? 0.f : mn - kOff;
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) l[nt][i] *= keep[i];
#pragma unroll
          for (int dt = 0; dt < KD; ++dt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[dt][nt][i] *= keep[i & 1];
        }
#pragma unroll
        for (int mt = 0; mt < KM; ++mt) {
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = exp2_fast(sc[mt][nt][i] - ref[i & 1]);
            l[nt][i & 1] = BITS != 16 ? fmaf(w[i], inv_vs[mt], l[nt][i & 1]) : l[nt][i & 1] + w[i];
          }
          // weights in the products' type: bf16 next to bf16 V, fp16 next to 8-bit V (three bits more, and V is exact in it)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t two = BITS == 16 ? pack_bf16(w[2 * i], w[2 * i + 1]) : pack_f16(w[2 * i], w[2 * i + 1]);
            pf[mt][nt][i] = transpose8x8(two);
          }
        }
      }

#pragma unroll
      for (int mt = 0; mt < KM; ++mt) {
        if (BITS == 16) {
#pragma unroll
          for (int dt = 0; dt < KD; ++dt) {
            uint32_t f[4];
            ldsm4_trans(swizzled<T::kSpan>(vb, TOK, mt * 16 + (lane & 7) + (lane >> 4) * 8, dt * 2 + (lane >> 3 & 1)), f);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<BITS>(acc[dt][nt], f, pf[mt][nt][0], pf[mt][nt][1]);
          }
        } else if (BITS == 4) {
          // A lane holds elements 4 g .. 4 g + 3 of 32, of tokens 2 t4 and 2 t4 + 1 (r[0]) and of those 8 on (r[1]); pairs of tokens are what
          // a product takes, so the halves change places: rows g and g + 8 of two products.
          const uint32_t gs = vb + T::kSideBytes + T::kGroupBytes + (mt * 16 + 2 * t4) * (D / 16), pick = g < 4 ? 0x6240u : 0x7351u;
          uint32_t sw[2][2 * (D / 64)];  // [tokens 2 t4.., 2 t4 + 8..][token, word]
#pragma unroll
          for (int h = 0; h < 2; ++h) lds_words<2 * (D / 64)>(gs + h * 8 * (D / 16), sw[h]);
#pragma unroll
          for (int c = 0; c < D / 32; c += 2) {
            uint32_t r[4], sg[2][2];  // [tokens][chunk]: both tokens' scales
            ldsm4_trans(swizzled<T::kSpan>(vb, TOK, mt * 16 + (lane & 15), c + (lane >> 4)), r);
#pragma unroll
            for (int h = 0; h < 2; ++h) e4m3_to_f16x4(__byte_perm(sw[h][c / 2], sw[h][D / 64 + c / 2], pick), &sg[h][0], &sg[h][1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t x[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t y[4];
                e2m1_to_f16x8(r[2 * i + h], y);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  x[h][2 * e] = mul_f16x2(__byte_perm(y[e], y[e + 2], 0x5410), sg[h][i]);
                  x[h][2 * e + 1] = mul_f16x2(__byte_perm(y[e], y[e + 2], 0x7632), sg[h][i]);
                }
              }
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t f[4] = {x[0][2 * j], x[0][2 * j + 1], x[1][2 * j], x[1][2 * j + 1]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma16816<BITS>(acc[2 * (c + i) + j][nt], f, pf[mt][nt][0], pf[mt][nt][1]);
              }
            }
          }
        } else {
          // two 16-element chunks per load; a lane's pairs of elements 2 g, 2 g + 1 of two tokens become rows g and g + 8
#pragma unroll
          for (int dt = 0; dt < KD; dt += 2) {
            uint32_t r[4];
            ldsm4_trans(swizzled<T::kSpan>(vb, TOK, mt * 16 + (lane & 15), dt + (lane >> 4)), r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t x = __byte_perm(r[2 * i], 0u, 0x3120), y = __byte_perm(r[2 * i + 1], 0u, 0x3120);
              uint32_t f[4];
              e4m3_to_f16x4(x, &f[0], &f[1]);
              e4m3_to_f16x4(y, &f[2], &f[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<BITS>(acc[dt + i][nt], f, pf[mt][nt][0], pf[mt][nt][1]);
            }
          }
        }
      }
      // refill the stage
      __syncwarp();
      const int kn = k + kStages * stride;
      if (kn < n_tiles) {
        fence_proxy_async_smem();
        issue(kn, page_ahead, st);
        page_ahead = page_for(kn + stride);
      } else if (BITS != 16) {
        cp_async_commit();
      }
      if (++st == kStages) {
        st = 0;
        phase ^= 1u;
      }
    }
    if (BITS != 16) cp_async_wait<0>();
    // A wait that gave up (a copy lost): the rows become NaN.  The copies in flight get the same limit again.
    if (!ok) {
      if (!dead)
        for (int i = 0; i < kStages; ++i) mbar_wait_limited(&s_full[warp][i], i < st ? phase ^ 1u : phase);
      if (lane == 0) s_dead = 1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) l[nt][i] = __int_as_float(0x7fffffff);
    }

    // Join the warps: every warp's accumulator in its own ring.
    float* part = reinterpret_cast<float*>(generic);
    constexpr int kPart = kStages * T::kStage / 4;
    static_assert(ROWS * (D + 4) <= kPart, "a warp's accumulator fits its ring");
    if (__any_sync(0xffffffffu, odd) && lane == 0) s_odd = 1;
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = l[nt][i];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        const int r = nt * 8 + 2 * t4 + i;
        if (g == 0) {
          s_m[warp][r] = m[nt][i];
          s_l[warp][r] = v;
        }
#pragma unroll
        for (int dt = 0; dt < KD; ++dt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int e = BITS == 4 ? dt / 2 * 32 + 4 * g + dt % 2 * 2 + h : dt * 16 + (BITS == 16 ? g + 8 * h : 2 * g + h);
            part[warp * kPart + r * (D + 4) + e] = acc[dt][nt][i + 2 * h];
          }
      }
    __syncthreads();
    if (tid < ROWS) {
      float mx = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][tid]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = s_m[w][tid] == mx ? 1.f : exp2_fast(s_m[w][tid] - mx);
        sum += s_l[w][tid] * f;
        s_m[w][tid] = f;
      }
      s_cm[tid] = mx;
      s_cl[tid] = sum;
    }
    __syncthreads();
    for (int e = tid; e < rows * D; e += kThreads) {
      const int r = e / D, at = r * (D + 4) + e % D;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += part[w * kPart + at] * s_m[w][r];
      part[at] = v;
    }
    __syncthreads();
    if (!full) {
      float* dst = part_of(a, blockIdx.x, t_begin == 0 ? 1 : 0, a.part_rows, D);
      for (int e = tid; e < rows * (D / 4); e += kThreads) {
        const int r = e / (D / 4), q4 = e % (D / 4) * 4;
        *reinterpret_cast<float4*>(dst + r * (D + 4) + q4) = *reinterpret_cast<const float4*>(part + r * (D + 4) + q4);
      }
      if (tid < rows) *reinterpret_cast<float4*>(dst + tid * (D + 4) + D) = make_float4(s_cm[tid], s_cl[tid], part_mark(row_end(s_dead, s_odd)), 0.f);
    } else if (row_end(s_dead, s_odd) != RowEnd::again) {  // a lost copy has made the sums NaN
      for (int e = tid; e < rows * (D / 2); e += kThreads) {
        const int r = e / (D / 2), d2 = e % (D / 2) * 2;
        const float sum = s_cl[r], inv = 1.f / sum * kDown;
        const float2 o = *reinterpret_cast<const float2*>(part + r * (D + 4) + d2);
        *reinterpret_cast<uint32_t*>(a.out + row_offset(a, s.first, kvh, r, a.o_token, a.o_head) + d2) = sum == 0.f ? 0u : pack_bf16(o.x * inv, o.y * inv);
      }
    } else {
      // an infinity or NaN in V that some rows see and others do not: row by row
      for (int r = warp; r < rows; r += kWarps) attend_row<D, BITS>(a, b, s, r / a.group, kvh * a.group + r % a.group, lane);
    }
    next(end);
    if (base >= share.last || b >= p.batch) break;
    fence_proxy_async_smem();  // the rings take copies again
    __syncthreads();
    if (tid == 0) s_odd = 0;
    __syncthreads();
  }
}

// Joins the parts of the units that the cuts met: a block per record and row, D / 4 threads per slice of the parts.
constexpr int kJoinThreads = 256;
template <int D, int BITS, int NT>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(const AttendParams a) {
  constexpr int kLanes = D / 4, kSlices = kJoinThreads / kLanes;
  __shared__ __align__(16) float s_o[kSlices][D];
  __shared__ float s_m[kSlices], s_l[kSlices];
  const int slice = threadIdx.x / kLanes, d4 = threadIdx.x % kLanes * 4, r = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PartRecord rec = reinterpret_cast<const PartRecord*>(a.part)[blockIdx.x];
  // by unit: nobody writes the record of a unit without rows
  const bool by_unit = (int64_t)a.c.batch * a.c.n_kv_heads <= kWave<D, BITS, NT>;
  const int b = by_unit ? blockIdx.x / a.c.n_kv_heads : rec.b, kvh = by_unit ? blockIdx.x % a.c.n_kv_heads : rec.kvh;
  if (!by_unit && !rec.valid) return;
  const SeqRows s = seq_rows(a.c, b);
  if (r >= s.n * a.group || !rec.valid) return;
  const int64_t row = (int64_t)r * (D + 4);
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  bool odd = false, lost = false;
#pragma unroll 4
  for (int c = rec.own + slice; c <= rec.last; c += kSlices) {
    const float* q = part_of(a, c, c == rec.own ? 1 : 0, a.part_rows, D) + row;
    const float4 t = *reinterpret_cast<const float4*>(q + D), v = *reinterpret_cast<const float4*>(q + d4);
    const float mn = fmaxf(m, t.x);
    const float keep = m == mn ? 1.f : exp2_fast(m - mn), f = t.x == mn ? 1.f : exp2_fast(t.x - mn);
    m = mn;
    odd |= t.z == kPartSpoilt;
    lost |= t.z == kPartLost;
    l = l * keep + t.y * f;
    o[0] = o[0] * keep + v.x * f;
    o[1] = o[1] * keep + v.y * f;
    o[2] = o[2] * keep + v.z * f;
    o[3] = o[3] * keep + v.w * f;
  }
  *reinterpret_cast<float4*>(&s_o[slice][d4]) = make_float4(o[0], o[1], o[2], o[3]);
  if (d4 == 0) {
    s_m[slice] = m;
    s_l[slice] = l;
  }
  const bool any_odd = __syncthreads_or(odd), any_lost = __syncthreads_or(lost);
  if (row_end(any_lost, any_odd) == RowEnd::again) {  // (a lost part's sum is NaN)
    if (threadIdx.x < 32) attend_row<D, BITS>(a, b, s, r / a.group, kvh * a.group + r % a.group, threadIdx.x);
    return;
  }
  const int d = threadIdx.x;
  if (d >= D) return;
  m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kSlices; ++i) m = fmaxf(m, s_m[i]);
  l = o[0] = 0.f;
#pragma unroll
  for (int i = 0; i < kSlices; ++i) {
    const float f = s_m[i] == m ? 1.f : exp2_fast(s_m[i] - m);
    l += s_l[i] * f;
    o[0] += s_o[i][d] * f;
  }
  // (o / l alone is 2^7 times the result, past fp32's range for outputs above 2^121)
  a.out[row_offset(a, s.first, kvh, r, a.o_token, a.o_head) + d] = (uint16_t)pack_bf16(l == 0.f ? 0.f : o[0] * (BITS == 16 ? 1.f : kSumDown) / l, 0.f);
}

// Bytes of workspace: none where no unit can be long, or no unit so long that its block would outlast the others by much.
template <int D, int BITS, int NT>
int64_t few_bytes(const AttendParams& a) {
  using T = Tile<D, BITS>;
  int64_t tokens = (int64_t)a.c.max_pages << a.c.page_shift;
  if (a.window > 0) tokens = std::min<int64_t>(tokens, (int64_t)a.window + a.c.max_q + a.sinks + 2 * T::kTokens);
  const int64_t whole = (int64_t)a.c.batch * a.c.n_kv_heads >= kSms ? kWholeMany<BITS> : kWholeFew<BITS>;
  return tokens <= whole * T::kTokens ? 0 : part_bytes(kWave<D, BITS, NT>, a.part_rows, D);
}

template <int D, int BITS, int NT>
cudaError_t few_rows(AttendParams a, int64_t* bytes, cudaStream_t st) {
  using T = Tile<D, BITS>;
  const int64_t need = few_bytes<D, BITS, NT>(a);
  if (bytes) {
    *bytes = need;
    return cudaSuccess;
  }
  if (need == 0 || need > a.part_bytes) a.part = nullptr;
  PageMaps maps;
  if (make_page_maps(a.c, D, BITS, std::min(a.c.page_size, T::kTokens), &maps)) return cudaErrorInvalidValue;
  const int64_t units = (int64_t)a.c.batch * a.c.n_kv_heads;
  auto run = [&](auto per_sm) {
    auto* f = k_attend_few<D, BITS, NT, decltype(per_sm)::value>;
    static std::atomic<uint64_t> prepared{0};
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(f), T::kSmem, &prepared);
    if (e != cudaSuccess) return e;
    f<<<a.part ? dim3(kWave<D, BITS, NT>) : dim3(a.c.batch, a.c.n_kv_heads), kThreads, T::kSmem, st>>>(a, maps);
    return cudaGetLastError();
  };
  if constexpr (kThirdBlock<D, BITS, NT>) {
    if (!a.part && third_block_pays(units)) return run(std::integral_constant<int, 3>{});
  }
  const cudaError_t e = run(std::integral_constant<int, kPerSm<D, BITS, NT>>{});
  if (e != cudaSuccess || !a.part) return e;
  return launch_after(k_attend_join<D, BITS, NT>, dim3(std::min<int64_t>(units, kWave<D, BITS, NT>), a.part_rows), kJoinThreads, st, a);
}

// Runs the call, or (bytes) says what workspace it takes.
template <int BITS>
cudaError_t few(const AttendParams& a, int head_dim, int64_t* bytes, cudaStream_t st) {
  if (head_dim == 128) return a.part_rows <= 8 ? few_rows<128, BITS, 1>(a, bytes, st) : few_rows<128, BITS, 2>(a, bytes, st);
  if constexpr (BITS == 4) {
    if (a.part_rows > 16) return few_rows<64, BITS, 3>(a, bytes, st);
  }
  return a.part_rows <= 8 ? few_rows<64, BITS, 1>(a, bytes, st) : few_rows<64, BITS, 2>(a, bytes, st);
}

}  // namespace

}  // namespace clo
