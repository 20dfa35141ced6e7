// Attention of many rows per kv head over a paged cache: prompts, chunks of prompts, several drafted tokens.
//
// A unit is one or two tiles of 128 rows of one (sequence, kv head) - consecutive query tokens times the group's
// heads, so that a K or V tile of 128 tokens serves every head of the group - with the tiles of tokens that its rows see.
// Both products run on tcgen05: S = Q K^T from shared memory into TMEM, O += P V with P in TMEM (over the
// columns of S that it came from) and O in TMEM.  One thread owns a row of S: its maximum and sum need no exchange.
//
// The grid is one block per SM.  All units' token tiles, laid end to end (a unit counts kUnitCost more), are cut into equal shares, so
// that ragged batches and causal prompts load the SMs alike and the fill of a block's next unit hides behind the current one's
// end.  Units that a cut meets leave their sums in the caller's workspace and are joined by a second kernel; without a workspace, or
// where a share would be short, units stay whole.
//
// Two lanes of work run against each other, so that one's products fill the time of the other's softmax: with two row
// tiles, a lane is a row tile; with one (at most 128 rows), lane 0 takes the even token tiles and lane 1 the odd ones, and
// their sums are joined at the end.
//
//   warps 0-3, 4-7   softmax of lane 0, 1 (TMEM rows are tied to a warp's place in its group of four)
//   warps 8, 11      TMA of K and of V: pages -> ring of operand tiles, K(0) K(1) V(0) K(2) V(1) ...
//   warp 9           MMA issue: P V of a token tile, then S of the lane's next one, the lanes in turn
//   warp 10          bf16 pages: V behind the last token that any row sees is cleared
//   warps 12-15      8-bit pages only: codes -> fp16 operand tiles
//
// The accumulator is rescaled only when a row's maximum has grown by more than 2^8 (weights stay below 2^8 times
// the largest so far; exact in the end, as sum and accumulator share the reference).
//
// A masked weight is zero, but zero times NaN is not.  V behind the last visible token (a page's end, where memory may never
// have been written) is cleared in the operand tile.  Rows that end with an infinity or NaN all the same are computed again, one
// by one, if V has one where they do not look (spoilt_rows looks V over once); what comes from tokens that they see stays.
//
// 8192 tokens, 32 over 8 heads of 128, causal, bf16: 404 to 416 us, 1.34 PFLOP/s, 70 % of a library product's rate: a token tile takes
// both lanes 2770 cycles, of which the products 2048, and the diagonal's tiles count half.  2048 tokens over 32,768 of 8-bit
// pages: 848 us, 1.26 PFLOP/s; there the softmax and the conversions share the issue slots (3700 cycles a tile).
#include <cuda_runtime.h>

#include <algorithm>

#include "clo_paged_attend.cuh"

namespace clo {
namespace {

constexpr int kTok = 128;    // tokens per tile
constexpr int kRows = 128;   // rows per row tile
constexpr float kGrow = 8.f;
constexpr int kUnitCost = 4;   // what a unit costs beside its token tiles, in tiles (11,000 cycles of 2,800)
// Units are cut where every block's share is kMinShare or more, as joining costs about as much as four tiles; in smaller calls only where a
// unit costs twice that, into shares of kLongShare, and otherwise units stay whole, spread over the SMs.  Shares of 8 / 5, us: 30 rows
// over 2000 tokens 19.8 / 17.5, of 8-bit pages 24.3 / 20.7; cutting down to 5 everywhere: a prompt of 600 tokens 17.7 / 20.7.
constexpr int kMinShare = 8, kLongShare = 5;

// ---------------------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(leader)
      : "memory");
}
#define CLO_R4(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3])
#define CLO_I4(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3])
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : CLO_R4(x, 0), CLO_R4(x, 4), CLO_R4(x, 8), CLO_R4(x, 12), CLO_R4(x, 16), CLO_R4(x, 20), CLO_R4(x, 24), CLO_R4(x, 28)
      : "r"(addr));
}
#define CLO_RW4(x, i) "+r"(x[i]), "+r"(x[i + 1]), "+r"(x[i + 2]), "+r"(x[i + 3])
// Ties 32 loaded registers to this point of the program: nothing that uses them moves above it.
__device__ __forceinline__ void tie32(uint32_t* x) {
  asm volatile("" : CLO_RW4(x, 0), CLO_RW4(x, 4), CLO_RW4(x, 8), CLO_RW4(x, 12), CLO_RW4(x, 16), CLO_RW4(x, 20), CLO_RW4(x, 24), CLO_RW4(x, 28));
}
// Waits for this thread's TMEM loads, of which x[0 .. 32 * N) are the results.
template <int N>
__device__ __forceinline__ void tc_wait_ld(uint32_t* x) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) tie32(x + 32 * i);
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::CLO_I4(x, 0),
      CLO_I4(x, 4), CLO_I4(x, 8), CLO_I4(x, 12), CLO_I4(x, 16), CLO_I4(x, 20), CLO_I4(x, 24), CLO_I4(x, 28), "r"(addr)
      : "memory");
}

// Operand tiles are [span of 64 elements][128 rows][128 bytes] with the 128-byte swizzle.  K-major (Q, K): rows are rows, 8-row
// groups 1024 bytes apart.  MN-major (V): a row is a token (the K side), its 64 elements the N side; spans 16 KB apart.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t leading, uint32_t stride) {
  return (uint64_t)((addr >> 4) & 0x3fffu) | (uint64_t)(leading >> 4) << 16 | (uint64_t)(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
__host__ __device__ constexpr uint32_t mma_shape(bool bf16, int n, bool mn_major_b) {
  return 1u << 4 | (bf16 ? 1u : 0u) << 7 | (bf16 ? 1u : 0u) << 10 | (mn_major_b ? 1u : 0u) << 16 | (uint32_t)(n / 8) << 17 | (uint32_t)(kRows / 16) << 24;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <int D, int BITS, int TILES>
struct Cfg {
  static constexpr int kTileBytes = kTok * D * 2;             // an operand tile
  static constexpr int kQBytes = kRows * D * 2;
  // operand tiles of the ring, and 8-bit tiles on their way into it: what fits next to Q
  static constexpr int kSlots = BITS == 16 ? (D == 64 ? 8 : TILES == 2 ? 4 : 5) : (D == 64 ? 6 : 4);
  static constexpr int kRawSide = BITS == 16 ? 0 : D == 64 ? 6 : TILES == 2 ? 2 : 3;  // halves of 64 tokens, for K and for V
  static constexpr int kRaw = 2 * kRawSide;
  static constexpr int kRawBytes = BITS == 16 ? 0 : kTok * D / 2;
  static constexpr int kMeta = D == 64 ? 16 : 8;  // token tiles whose page data is kept: more than the ring runs ahead
  static constexpr int kThreads = BITS == 16 ? 384 : 512;
  static constexpr int kBytes = TILES * kQBytes + kSlots * kTileBytes + kRaw * kRawBytes + 1024;
};

template <int META, int TILES>
struct Shared {
  uint64_t full[8], empty[8];      // operand tiles: filled (TMA or converters), products done
  uint64_t tail[8], q_ready[2];      // bf16: a V tile whose end is yet to be cleared; Q
  uint64_t raw_full[12], raw_empty[12];  // 8-bit pages: halves of tiles on their way
  uint64_t s_full[2], p_half[2], p_ready[2];  // per lane: scores; weights of the first 64 tokens, of all
  uint64_t meta[META];
  float scale[META][3][8];        // K scale, log2 of the V scale, its reciprocal
  uint32_t there[META];
  uint32_t tmem;
  int failed;
  int odd;                         // a row of the block ended as no finite number
  int64_t first, last, total;      // the block's share of the units' costs, [first, last) of total
  int64_t base;                    // where the first unit of the share begins
  PartRecord record;               // of the unit that the share leaves unfinished
  int blocks, cuts;                // blocks that take a share; whether units are cut
  int start[3];                    // that unit: sequence, block of rows, kv head
  float join_m[TILES == 1 ? kRows : 1], join_l[TILES == 1 ? kRows : 1];  // lane 1's maxima and sums
  int8_t q_exp[2][kRows];          // 8-bit pages: q rows are scaled by 2^-q_exp
};

// Bounded wait (two seconds, see mbar_wait_limited); once one has given up, the others follow.
template <typename S>
__device__ __forceinline__ bool wait(S& sh, uint64_t* bar, uint32_t parity) {
  if (mbar_test(bar, parity)) return true;
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait_long(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (*reinterpret_cast<volatile int*>(&sh.failed) == 0) {
    if (mbar_try_wait_long(bar, parity)) return true;
    if (global_timer_ns() - t0 > 2000000000ull) *reinterpret_cast<volatile int*>(&sh.failed) = 1;
  }
  return false;
}

// Steps a pointer through a unit's rows, head by head and token by token.
template <typename T>
struct RowPtr {
  T* p;
  int h, group;
  int64_t head, wrap;
  __device__ __forceinline__ RowPtr(const AttendParams& a, T* base, int first, int kvh, int row, int64_t stride_token, int64_t stride_head) {
    group = a.group;
    head = stride_head;
    wrap = stride_token - (int64_t)(group - 1) * stride_head;
    const int t = token_of_row(a, row);
    h = row - t * group;
    p = base + (int64_t)(first + t) * stride_token + (int64_t)(kvh * group + h) * stride_head;
  }
  __device__ __forceinline__ void next() {
    const bool last = ++h == group;
    p += last ? wrap : head;
    if (last) h = 0;
  }
};

// A unit and the block's part of it.
struct Unit {
  SeqRows s;
  int b, qb, kvh;
  int rows, row0, row_end;  // the sequence's rows, and the unit's [row0, row_end) of them
  int pos_first, pos_last;
  TileList tl;
  int all;                  // token tiles of the unit
  int t_begin, n;           // the block's part
};

template <int TILES>
__device__ __forceinline__ void set_rows(const AttendParams& a, Unit* u) {
  u->row0 = u->qb * TILES * kRows;
  u->row_end = min(u->rows, u->row0 + TILES * kRows);
  u->pos_first = u->s.pos0 + token_of_row(a, u->row0);
  u->pos_last = u->s.pos0 + token_of_row(a, u->row_end - 1);
  u->tl = tiles_of(u->pos_first, u->pos_last, u->s.kv_len, a.window, a.sinks, kTok);
  u->all = u->tl.count();
}
template <int TILES>
__device__ __forceinline__ bool set_seq(const AttendParams& a, int b, Unit* u) {
  u->b = b;
  u->s = seq_rows(a.c, b);
  u->rows = u->s.n * a.group;
  u->qb = (u->rows + TILES * kRows - 1) / (TILES * kRows) - 1;  // the last rows first: they see the most tokens
  u->kvh = 0;
  if (u->rows == 0) return false;
  set_rows<TILES>(a, u);
  return true;
}
// The next unit in the order sequence, block of rows from the last, kv head; false past the last one.
template <int TILES>
__device__ __forceinline__ bool next_unit(const AttendParams& a, Unit* u) {
  if (++u->kvh < a.c.n_kv_heads) return true;
  u->kvh = 0;
  if (u->qb > 0) {
    --u->qb;
    set_rows<TILES>(a, u);
    return true;
  }
  for (int b = u->b + 1; b < a.c.batch; ++b)
    if (set_seq<TILES>(a, b, u)) return true;
  return false;
}

// Cost of a sequence's units for one kv head: by one lane, or by a warp's lanes over its blocks of rows.
template <int TILES>
__device__ __forceinline__ int64_t seq_cost(const AttendParams& a, const SeqRows& s, int lane, int lanes, int* most) {
  Unit u;
  u.s = s;
  u.rows = s.n * a.group;
  const int blocks = (u.rows + TILES * kRows - 1) / (TILES * kRows);
  int64_t c = 0;
  for (u.qb = lane; u.qb < blocks; u.qb += lanes) {
    set_rows<TILES>(a, &u);
    c += u.all + kUnitCost;
    *most = max(*most, u.all + kUnitCost);
  }
  return c;
}
// The block whose share holds the cost before `end`, where block i of n takes [total i / n, total (i + 1) / n).
__device__ __forceinline__ int last_block(int64_t total, int blocks, int64_t end) {
  int c = (int)min(end * blocks / total, (int64_t)blocks - 1);
  while (total * c / blocks >= end) --c;
  while (total * (c + 1) / blocks < end) ++c;
  return c;
}
__device__ __forceinline__ SeqRows shfl_seq(const SeqRows& s, int from) {
  SeqRows r;
  r.first = __shfl_sync(0xffffffffu, s.first, from);
  r.n = __shfl_sync(0xffffffffu, s.n, from);
  r.pos0 = __shfl_sync(0xffffffffu, s.pos0, from);
  r.kv_len = __shfl_sync(0xffffffffu, s.kv_len, from);
  return r;
}

// The block's share and the unit that it begins in, by one warp.
template <int TILES, typename S>
__device__ void find_share(const AttendParams& a, int lane, S& sh) {
  const PagedParams& p = a.c;
  const int heads = p.n_kv_heads;
  int64_t total = 0, share = 0;
  int most = 0;  // the largest unit's cost
  // pass 0 adds everything up, pass 1 stops at the sequence that holds the share's begin
  for (int pass = 0; pass < 2; ++pass) {
    int64_t before = 0;
    int found = -1;
    for (int c = 0; c < p.batch && found < 0; c += 32) {
      SeqRows mine{};
      if (c + lane < p.batch) mine = seq_rows(p, c + lane);
      const int count = min(32, p.batch - c), blocks = (mine.n * a.group + TILES * kRows - 1) / (TILES * kRows);
      const bool many = __any_sync(0xffffffffu, blocks > 8);
      int64_t cost = 0;  // of this lane's sequence
      if (many) {
        for (int i = 0; i < count; ++i) {
          const int64_t x = warp_sum64(seq_cost<TILES>(a, shfl_seq(mine, i), lane, 32, &most));
          if (lane == i) cost = x;
        }
      } else {
        cost = seq_cost<TILES>(a, mine, 0, 1, &most);
      }
      cost *= heads;
      if (pass == 0) {
        total += warp_sum64(cost);
        continue;
      }
      int64_t incl = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned m = __ballot_sync(0xffffffffu, before + incl > share);
      if (m) {
        const int l = __ffs(m) - 1;
        found = c + l;
        before += __shfl_sync(0xffffffffu, incl - cost, l);
        // the block of rows: the lanes step through them from the last
        const SeqRows s = shfl_seq(mine, l);
        Unit u;
        u.s = s;
        u.rows = s.n * a.group;
        const int nb = (u.rows + TILES * kRows - 1) / (TILES * kRows);
        for (int q = 0; q < nb; q += 32) {
          int64_t x = 0;
          if (q + lane < nb) {
            u.qb = nb - 1 - q - lane;
            set_rows<TILES>(a, &u);
            x = (int64_t)(u.all + kUnitCost) * heads;
          }
          int64_t upto = x;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
          }
          const unsigned w = __ballot_sync(0xffffffffu, before + upto > share);
          if (w) {
            const int k = __ffs(w) - 1;
            const int64_t each = __shfl_sync(0xffffffffu, x, k) / heads;
            before += __shfl_sync(0xffffffffu, upto - x, k);
            if (lane == 0) {
              const int64_t h = (share - before) / each;
              sh.start[0] = found;
              sh.start[1] = nb - 1 - q - k;
              sh.start[2] = (int)h;
              sh.base = before + h * each;
            }
            break;
          }
          before += __shfl_sync(0xffffffffu, upto, 31);
        }
      } else {
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (pass == 0) {
      most = __reduce_max_sync(0xffffffffu, most);
      const bool large = total >= (int64_t)kMinShare * gridDim.x, cuts = a.part && (large || most >= 2 * kMinShare);
      const int blocks = cuts && !large ? min(max((int)(total / kLongShare), 1), (int)gridDim.x) : (int)gridDim.x;
      share = total * min((int)blockIdx.x, blocks) / blocks;
      const int64_t last = total * min((int)blockIdx.x + 1, blocks) / blocks;
      if (lane == 0) {
        sh.first = share;
        sh.last = last;
        sh.total = total;
        sh.base = total;  // an empty share finds nothing
        sh.blocks = blocks;
        sh.cuts = cuts;
      }
      __syncwarp();
      if (last == share) return;
    }
  }
}

// The block's walk over its units; every role takes it by itself.  `visit` is called with each unit that the block has a part of.
template <int TILES, typename S, typename F>
__device__ __forceinline__ void walk_units(const AttendParams& a, const S& sh, bool cuts, F&& visit) {
  int64_t base = sh.base;
  const int64_t first = sh.first, last = sh.last;
  if (base >= last) return;
  Unit u;
  set_seq<TILES>(a, sh.start[0], &u);
  u.qb = sh.start[1];
  u.kvh = sh.start[2];
  set_rows<TILES>(a, &u);
  while (true) {
    const int64_t end = base + u.all + kUnitCost;
    bool part = base >= first;  // the unit begins in the share: whole units, and those without a token, go by that alone
    u.t_begin = 0;
    u.n = u.all;
    if (cuts && u.all > 0) {
      u.t_begin = base >= first ? 0 : max((int)(first - base) - kUnitCost, 0);
      u.n = (end <= last ? u.all : max((int)(last - base) - kUnitCost, 0)) - u.t_begin;
      part = u.n > 0;
    }
    if (part && !visit(u, base)) return;
    base = end;
    if (base >= last || !next_unit<TILES>(a, &u)) return;
  }
}

// Rows that ended as no finite numbers: rightly, or to be computed again?  At the block's end, over its units once more and out of line, so
// that the tiles' loops keep their registers (among them it cost 2 to 3 % with 8-bit pages).  A prompt of 8192 tokens, 8 over 2 heads, with
// a NaN in one head's first V: 1.0 ms for 0.13 without; every such row computed again took 100 ms.
template <int D, int BITS, int TILES, typename S>
__device__ __noinline__ void look_again(const AttendParams a, const S& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  walk_units<TILES>(a, sh, sh.cuts, [&](const Unit& u, int64_t) {
    const bool full = u.n == u.all;
    for (int r0 = warp * 32; r0 < TILES * kRows && u.row0 + r0 < u.rows; r0 += blockDim.x) {
      const int row = u.row0 + r0 + lane;
      bool spoilt = false, nan = false;
      float* part = nullptr;
      if (row < u.rows) {
        if (full) {
          const uint16_t* o = a.out + row_offset(a, u.s.first, u.kvh, row, a.o_token, a.o_head);
#pragma unroll 1
          for (int e = 0; e < D; e += 8) {
            float y[8];
            unpack8(*reinterpret_cast<const uint4*>(o + e), y);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              nan |= isnan(y[k]);
              spoilt |= !isfinite(y[k]);
            }
          }
        } else {
          part = part_of(a, blockIdx.x, u.t_begin == 0 ? 1 : 0, TILES * kRows, D) + (int64_t)(r0 + lane) * (D + 4);
          spoilt = !isfinite(part[D + 1]);
#pragma unroll 1
          for (int e = 0; e < D; ++e) {
            nan |= isnan(part[e]);
            spoilt |= !isfinite(part[e]);
          }
        }
      }
      if (!__any_sync(0xffffffffu, spoilt)) continue;
      if (spoilt && !full) part[D + 2] = kPartSeen;
      spoilt = spoilt_rows<D, BITS>(a, u.b, u.kvh, u.s, u.tl, u.t_begin, u.t_begin + u.n, kTok, visible_of(u.pos_last, u.s.kv_len, a.window, a.sinks).hi,
                                    spoilt, u.s.pos0 + token_of_row(a, min(row, u.rows - 1)), nan, lane);
      if (!full) {
        if (spoilt) part[D + 2] = kPartSpoilt;
        continue;
      }
      for (unsigned again = __ballot_sync(0xffffffffu, row_end(sh.failed != 0, spoilt) == RowEnd::again); again; again &= again - 1) {
        const int gr = u.row0 + r0 + __ffs(again) - 1;
        attend_row<D, BITS>(a, u.b, u.s, gr / a.group, u.kvh * a.group + gr % a.group, lane);
      }
    }
    return true;
  });
}

template <int D, int BITS, int TILES>
__global__ void __launch_bounds__(Cfg<D, BITS, TILES>::kThreads, 1) k_attend_many(const AttendParams a, const __grid_constant__ PageMaps maps) {
  using C = Cfg<D, BITS, TILES>;
  constexpr int SLOTS = C::kSlots;
  extern __shared__ uint8_t smem_raw[];
  constexpr int kMeta = C::kMeta;
  __shared__ __align__(16) Shared<kMeta, TILES> sh;

  const PagedParams& p = a.c;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_smem = smem, ring = smem + TILES * C::kQBytes, raw = ring + SLOTS * C::kTileBytes;
  uint8_t* const generic = smem_raw + (smem - smem_u32(smem_raw));

  if (tid == 32) {
    prefetch_map(&maps.side[0]);
    prefetch_map(&maps.side[1]);
  }
  if (tid == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(&sh.full[i], BITS == 16 ? 1 : 2 * 128);
      mbar_init(&sh.empty[i], 1);
      mbar_init(&sh.tail[i], 1);
    }
    for (int i = 0; i < 12; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_empty[i], 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_half[i], 128);
      mbar_init(&sh.p_ready[i], 128);
    }
    for (int i = 0; i < TILES; ++i) mbar_init(&sh.q_ready[i], 256 / TILES);
    for (int i = 0; i < kMeta; ++i) mbar_init(&sh.meta[i], 1);
    sh.failed = sh.odd = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  if (warp == 0) find_share<TILES>(a, lane, sh);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  constexpr uint32_t kS[2] = {0, 128}, kO[2] = {256, 384};

  const bool cuts = sh.cuts;
  auto walk = [&](auto&& visit) { walk_units<TILES>(a, sh, cuts, visit); };

  // Operand tiles of a unit in ring order: e = 0 is K(0), e = 2 j + 1 is K(j + 1), e = 2 j + 2 is V(j), without K(n); the ring's count
  // runs on from unit to unit.  Lane t takes token tiles first_of(t), + kStep, ...
  auto at_k = [](int j) { return j == 0 ? 0 : 2 * j - 1; };
  auto at_v = [](int j, int n) { return 2 * j + 2 - (j + 1 >= n ? 1 : 0); };
  constexpr int kStep = TILES == 2 ? 1 : 2;
  auto first_of = [](int t) { return TILES == 2 ? 0 : t; };
  auto count_of = [](int t, int n) { return TILES == 2 ? n : (n + 1 - t) / 2; };
  // the unit's last tile, if the part has it, holds tokens that no row sees
  auto tail_of = [&](const Unit& u) {
    return u.n > 0 && (u.tl.at(u.t_begin + u.n - 1) + 1) * kTok > visible_of(u.pos_last, u.s.kv_len, a.window, a.sinks).hi;
  };

  if (warp < 8) {
    // ------------------------------------------------------------------------ softmax
    constexpr float kOff = BITS == 16 ? 0.f : 7.f;  // weights of 8-bit pages: up to 2^15 with kGrow, fp16 down to 2^-31
    const int t = warp >> 2, my_tile = TILES == 2 ? t : 0;
    const uint32_t lane_off = (uint32_t)(warp & 3) * 32u << 16;
    const uint32_t s_addr = tmem + lane_off + kS[t], o_addr = tmem + lane_off + kO[t];
    uint32_t q_phase = 0, s_phase = 0;
    int tiles_done = 0;
    bool ok = true;
    if (tid == 0) sh.record.valid = 0;
    walk([&](const Unit& u, int64_t base) {
    const SeqRows& s = u.s;
    const int n = u.n, row0 = u.row0, rows = u.rows, kvh = u.kvh, mine = count_of(t, n);
    const bool full = n == u.all;
    if (tid == 0 && !full && u.t_begin == 0) sh.record = {1, u.b, u.qb, kvh, last_block(sh.total, sh.blocks, base + u.all + kUnitCost), (int)blockIdx.x};
    // Q rows into operand tiles, D / 8 threads per row.  8-bit pages: fp16, each row scaled by a power of two that puts its
    // largest finite element into [2^14, 2^15).
    // Two row tiles: each lane loads its own, so that it need not wait for the other's end.
    constexpr int kLoaders = TILES == 2 ? 128 : 256;
    if (n > 0) asm volatile("bar.sync %0, %1;" ::"r"(1 + my_tile), "n"(kLoaders) : "memory");  // all have left the last unit's Q
    if (n > 0 && ok) {
      // a thread takes one 16-byte chunk of kIters rows that follow one another
      constexpr int kLanes = D / 8, kIters = kRows * kLanes / kLoaders;
      const int c = tid % kLanes, r0 = my_tile * kRows + tid % kLoaders / kLanes * kIters;
      RowPtr<const uint16_t> src(a, a.q + c * 8, s.first, kvh, row0 + r0, a.q_token, a.q_head);
      uint8_t* const to = generic + (r0 / kRows * C::kQBytes + c / 8 * kRows * 128 + r0 % kRows * 128);
#pragma unroll 2
      for (int i = 0; i < kIters; ++i) {
        uint4* at = reinterpret_cast<uint4*>(to + i * 128 + ((c ^ (r0 + i)) & 7) * 16);
        if (row0 + r0 + i < rows)
          cp_async16(at, src.p);
        else
          *at = make_uint4(0, 0, 0, 0);
        src.next();
      }
      cp_async_commit();
      cp_async_wait<0>();
      if (BITS == 8) {
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < kIters; ++i) {
          const int r = r0 + i;
          uint4* at = reinterpret_cast<uint4*>(to + i * 128 + ((c ^ r) & 7) * 16);
          float x[8], mx = 0.f;
          unpack8(*at, x);
#pragma unroll
          for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(x[k]) < INFINITY ? fabsf(x[k]) : 0.f);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127 - 14, -100), 112);
          const float down = __uint_as_float((uint32_t)(127 - e) << 23);
          if (c == 0) sh.q_exp[r / kRows][r % kRows] = (int8_t)e;
          *at = make_uint4(pack_f16(x[0] * down, x[1] * down), pack_f16(x[2] * down, x[3] * down), pack_f16(x[4] * down, x[5] * down), pack_f16(x[6] * down, x[7] * down));
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&sh.q_ready[my_tile]);
    }
    float ref = -INFINITY, l = 0.f;
    const int my_row = row0 + my_tile * kRows + (tid & 127);
    const bool row_ok = my_row < rows;
    if (n > 0) {
      ok = ok && __all_sync(0xffffffffu, wait(sh, &sh.q_ready[my_tile], q_phase));
      q_phase ^= 1u;
    }
    const float fac = BITS == 8 ? a.scale_log2 * __uint_as_float((uint32_t)(127 + sh.q_exp[my_tile][tid & 127]) << 23) : a.scale_log2;
    {
      // the tile's first and last row bound what "every row sees" means; rows past the end follow the last one
      const int rf = min(row0 + my_tile * kRows, rows - 1), rl = min(row0 + my_tile * kRows + kRows - 1, rows - 1);
      const Visible vf = visible_of(s.pos0 + rf / a.group, s.kv_len, a.window, a.sinks);
      const Visible vl = visible_of(s.pos0 + rl / a.group, s.kv_len, a.window, a.sinks);
      const Visible v = visible_of(s.pos0 + min(my_row, rows - 1) / a.group, s.kv_len, a.window, a.sinks);
      for (int i = 0; i < mine && ok; ++i) {
        const int j = first_of(t) + i * kStep, j0 = u.tl.at(u.t_begin + j) * kTok;
        const int slot = (tiles_done + j) % kMeta;
        ok = wait(sh, &sh.meta[slot], ((tiles_done + j) / kMeta) & 1) && wait(sh, &sh.s_full[t], s_phase);
        s_phase ^= 1u;
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t there = sh.there[slot];
        const bool whole = there == 0xffu && j0 + kTok <= vf.hi && (j0 >= vl.lo || j0 + kTok <= (a.window > 0 ? a.sinks : 0));
        // Scores stay in TMEM and pass through registers by halves, twice: for the maximum, then for the weights, which go over
        // columns already read.  (Code of a whole row's 128 scores does not fit the instruction cache beside the other roles'.)
        uint32_t x[64];
        float mx = -INFINITY;
#pragma unroll 1
        for (int half = 1; half >= 0; --half) {  // the first half last: it stays in registers for its weights
          tc_ld32(s_addr + 64 * half, x);
          tc_ld32(s_addr + 64 * half + 32, x + 32);
          tc_wait_ld<2>(x);
          if (!whole) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              // bits of 32 columns that this row sees
              const int base = j0 + 64 * half + 32 * c;
              auto below = [&](int end) { return end - base >= 32 ? 0xffffffffu : end <= base ? 0u : (1u << (end - base)) - 1u; };
              uint32_t see = (below(v.hi) & ~below(v.lo)) | below(v.sink_end);
              const uint32_t pages = there >> (4 * half + 2 * c);
              if (!(pages & 1u)) see &= 0xffff0000u;
              if (!(pages & 2u)) see &= 0x0000ffffu;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(see >> k & 1u)) x[32 * c + k] = 0xff800000u;
              tc_st32(s_addr + 64 * half + 32 * c, x + 32 * c);
            }
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // per 16 tokens, which share a page's scales
#pragma unroll
          for (int k = 0; k < 16; k += 2)
#pragma unroll
            for (int h = 0; h < 4; ++h) m4[h] = fmaxf(m4[h], fmaxf(__uint_as_float(x[16 * h + k]), __uint_as_float(x[16 * h + k + 1])));
          if (BITS == 8) {
#pragma unroll
            for (int h = 0; h < 4; ++h) m4[h] = fmaf(m4[h], fmaxf(sh.scale[slot][0][4 * half + h] * fac, 1e-37f), sh.scale[slot][1][4 * half + h]);
          }
          mx = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
        }
        if (BITS == 16) mx *= fac;
        if (!whole) tc_wait_st();
        const bool grow = mx > ref + kGrow;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? (ref == -INFINITY ? 0.f : exp2_fast(ref - mx)) : 1.f;
          if (grow) ref = mx;
          l *= f;
          if (i > 0) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tc_ld32(o_addr + 32 * c, o);
              tc_wait_ld<1>(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tc_st32(o_addr + 32 * c, o);
            }
          }
        }
        const float sub = ref == -INFINITY ? 0.f : kOff - ref;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint32_t w[32];
          uint64_t sum2[2] = {0, 0};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            // 16 tokens: one page, one set of scales
            const int at = 4 * half + h;
            const float mul = BITS == 8 ? fmaxf(sh.scale[slot][0][at] * fac, 1e-37f) : fac, add = BITS == 8 ? sh.scale[slot][1][at] + sub : sub;
            const uint64_t mul2 = pack2(mul, mul), add_2 = pack2(add, add);
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              float2 y = unpack2(fma2(pack2(__uint_as_float(x[16 * h + k]), __uint_as_float(x[16 * h + k + 1])), mul2, add_2));
              y.x = exp2_fast(y.x);
              y.y = exp2_fast(y.y);
              sum2[(k >> 1) & 1] = add2(sum2[(k >> 1) & 1], pack2(y.x, y.y));
              // weights in the products' type: bf16 next to bf16 V, fp16 next to 8-bit V
              w[8 * h + k / 2] = BITS == 16 ? pack_bf16(y.x, y.y) : pack_f16(y.x, y.y);
            }
            if (BITS == 8 || h == 3) {
              const float2 q = unpack2(add2(sum2[0], sum2[1]));
              l = BITS == 8 ? fmaf(q.x + q.y, sh.scale[slot][2][at], l) : l + (q.x + q.y);
              sum2[0] = sum2[1] = 0;
            }
          }
          tc_st32(s_addr + 32 * half, w);
          if (half == 0) {
            tc_ld32(s_addr + 64, x);
            tc_ld32(s_addr + 96, x + 32);
          }
          tc_wait_st();
          tc_fence_before();
          mbar_arrive(half == 0 ? &sh.p_half[t] : &sh.p_ready[t]);
          if (half == 0) tc_wait_ld<2>(x);
        }
      }
      // the lane's last product
      if (mine > 0) {
        ok = ok && __all_sync(0xffffffffu, wait(sh, &sh.s_full[t], s_phase));
        s_phase ^= 1u;
      }
      tc_fence_after();
      if (TILES == 1 && n > 0) {
        // Lane 1's sums join lane 0's: its accumulator lies in the same TMEM rows.  Barrier 1 at the begin of the next unit with tiles
        // holds lane 1 back until lane 0 has read them; a unit without tiles has neither that barrier nor sums.
        if (t == 1) {
          sh.join_m[tid & 127] = ref;
          sh.join_l[tid & 127] = l;
          tc_fence_before();
        }
        asm volatile("bar.sync 3, 256;" ::: "memory");
        tc_fence_after();
      }
      if (TILES == 2 || t == 0) {
        float f0 = 1.f, f1 = 0.f;
        const bool both = TILES == 1 && count_of(1, n) > 0;
        if (both) {
          const float m1 = sh.join_m[tid & 127], mx = fmaxf(ref, m1);
          f0 = ref == mx ? 1.f : exp2_fast(ref - mx);
          f1 = m1 == mx ? 1.f : exp2_fast(m1 - mx);
          l = l * f0 + sh.join_l[tid & 127] * f1;
          ref = mx;
        }
        // a wait gave up anywhere in the block: this unit's rows and the rest of the share are NaN
        const bool lost = *reinterpret_cast<volatile int*>(&sh.failed) != 0;
        if (lost) l = __int_as_float(0x7fffffff);
        const float inv = full ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        float* part = nullptr;
        if (!full) {
          part = part_of(a, blockIdx.x, u.t_begin == 0 ? 1 : 0, TILES * kRows, D) + (int64_t)(my_tile * kRows + (tid & 127)) * (D + 4);
          *reinterpret_cast<float4*>(part + D) = make_float4(ref, l, part_mark(row_end(lost, false)), 0.f);
        }
        float odd = l * 0.f;  // NaN if anything in the row is no finite number
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (mine > 0) {
            tc_ld32(o_addr + 32 * c, o);
            tc_wait_ld<1>(o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          if (both) {
            uint32_t o1[32];
            tc_ld32(o_addr + 128 + 32 * c, o1);
            tc_wait_ld<1>(o1);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f0 + __uint_as_float(o1[i]) * f1);
          }
          if (!full) {
#pragma unroll
            for (int i = 0; i < 32; ++i) odd = fmaf(__uint_as_float(o[i]), 0.f, odd);
#pragma unroll
            for (int i = 0; i < 32; i += 4) *reinterpret_cast<uint4*>(part + 32 * c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          } else {
            // through the row tile's Q, which is done with, so that rows leave in whole lines
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                odd = fmaf(__uint_as_float(o[i + e]), 0.f, odd);
                y[e] = l == 0.f ? 0.f : __uint_as_float(o[i + e]) * inv;
              }
              *reinterpret_cast<uint4*>(generic + (swizzled<128>(q_smem + my_tile * C::kQBytes, kRows, tid & 127, 4 * c + i / 8) - smem)) = pack8(y);
            }
          }
        }
        if (__any_sync(0xffffffffu, row_ok && odd != 0.f) && lane == 0) sh.odd = 1;
        if (full) {
          __syncwarp();
          constexpr int kLanes = D / 8;
          const int r0 = (warp & 3) * 32 + lane / kLanes * kLanes, c = lane % kLanes;  // kLanes rows that follow one another
          const uint8_t* from = generic + (my_tile * C::kQBytes + c / 8 * kRows * 128 + r0 * 128);
          RowPtr<uint16_t> dst(a, a.out + c * 8, s.first, kvh, row0 + my_tile * kRows + r0, a.o_token, a.o_head);
#pragma unroll 2
          for (int i = 0; i < kLanes; ++i) {
            if (row0 + my_tile * kRows + r0 + i < rows)
              *reinterpret_cast<uint4*>(dst.p) = *reinterpret_cast<const uint4*>(from + i * 128 + ((c ^ (r0 + i)) & 7) * 16);
            dst.next();
          }
          if (BITS == 8) {
            // a sum of weights past fp32's range (scales near 2^-100)
            __syncwarp();
            unsigned again = __ballot_sync(0xffffffffu, row_ok && row_end(lost, l == INFINITY) == RowEnd::again);
            for (; again; again &= again - 1) {
              const int gr = row0 + my_tile * kRows + (warp & 3) * 32 + __ffs(again) - 1;
              attend_row<D, BITS>(a, u.b, s, gr / a.group, kvh * a.group + gr % a.group, lane);
            }
          }
        }
      }
      tc_fence_before();
      tiles_done += n;
    }
    return true;
    });
    if (tid == 0 && a.part) *(reinterpret_cast<PartRecord*>(a.part) + blockIdx.x) = sh.record;
  } else {
    if (warp == 8 || warp == 11) {
      // ---------------------------------------------------------------------- TMA: K and page data; V
      const int side = warp == 8 ? 0 : 1;
      constexpr int kSpan = BITS == 16 ? 128 : (D < 128 ? D : 128);  // bytes of a page row in one box
      constexpr int kBoxSpans = D * BITS / 8 / kSpan;
      // The ring of operand tiles (16 bits), or the side's own ring of half tiles.  Two warps may fill one ring in turns only if it holds
      // three elements or more: the parity of an earlier use than the one waited for must not be met (K jumps three places from
      // unit to unit).
      static_assert(C::kSlots >= 3, "see above");
      constexpr int kBuf = BITS == 16 ? C::kSlots : C::kRawSide;
      constexpr int kParts = BITS == 16 ? 1 : 2, kPartTok = kTok / kParts;
      const int box = min(p.page_size, kPartTok);
      int e_base = 0, tiles_done = 0;
      bool ok = true;
      walk([&](const Unit& u, int64_t) {
      const int n = u.n, b = u.b, kvh = u.kvh;
      const bool tail = tail_of(u);
      // Pages of four tiles at a time, a lane per 16 tokens, looked up two batches ahead and their scales one, so that no load waits for
      // another.
      auto pages_of = [&](int batch) {
        const int j = 4 * batch + (lane >> 3);
        return j < n ? page_of(p, b, (u.tl.at(u.t_begin + j) * kTok + (lane & 7) * 16) >> p.page_shift) : -1;
      };
      auto scales_of = [&](int page) {
        float2 sc = make_float2(1.f, 1.f);
        if (BITS == 8 && side == 0 && page >= 0) {
          const int64_t at = (int64_t)page * p.n_kv_heads + kvh;
          sc = make_float2(__ldg(p.side[0].scales + at), __ldg(p.side[1].scales + at));
        }
        return sc;
      };
      int page0 = pages_of(0), page1 = pages_of(1), page2 = pages_of(2);
      float2 scale0 = scales_of(page0), scale1 = scales_of(page1);
      for (int j = 0; j < n && ok; ++j) {
        const int q = j & 3, e = e_base + (side == 0 ? at_k(j) : at_v(j, n));
        if (q == 0 && j > 0) {
          page0 = page1;
          page1 = page2;
          page2 = pages_of((j >> 2) + 2);
          scale0 = scale1;
          scale1 = scales_of(page1);
        }
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
          const int x = BITS == 16 ? e : 2 * (tiles_done + j) + h, use = x / kBuf, buf = BITS == 16 ? x % kBuf : side * kBuf + x % kBuf;
          uint64_t* full = BITS == 16 ? (tail && side == 1 && j == n - 1 ? &sh.tail[buf] : &sh.full[buf]) : &sh.raw_full[buf];
          uint64_t* empty = BITS == 16 ? &sh.empty[buf] : &sh.raw_empty[buf];
          int id[kPartTok / 16];
#pragma unroll
          for (int g = 0; g < kPartTok / 16; ++g) id[g] = __shfl_sync(0xffffffffu, page0, 8 * q + h * (kPartTok / 16) + g);
          if (use > 0) ok = wait(sh, empty, (use - 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (elect_one()) {
            const uint32_t dst = BITS == 16 ? ring + buf * C::kTileBytes : raw + buf * C::kRawBytes, bar = smem_u32(full);
            const int slot0 = u.tl.at(u.t_begin + j) * kTok + h * kPartTok;
            mbar_arrive_expect_tx(full, BITS == 16 ? C::kTileBytes : C::kRawBytes);
#pragma unroll
            for (int g = 0; g < kPartTok / 16; ++g)
              if (g * 16 % box == 0) {
#pragma unroll
                for (int w = 0; w < kBoxSpans; ++w)
                  tma_box(dst + g * 16 * kSpan + w * kTok * kSpan, &maps.side[side], w * (kSpan * 8 / BITS), (slot0 + g * 16) & (p.page_size - 1), kvh, id[g], bar);
              }
          }
          __syncwarp();
        }
        if (ok && side == 0) {  // which 16-token groups are there, and their scales
          const int slot = (tiles_done + j) % kMeta;
          const unsigned there = __ballot_sync(0xffffffffu, page0 >= 0) >> (8 * q) & 0xffu;
          if (lane == 0) sh.there[slot] = there;
          if (BITS == 8 && lane >> 3 == q) {
            const float vs = fmaxf(scale0.y, kMinScale);
            sh.scale[slot][0][lane & 7] = fmaxf(scale0.x, kMinScale);
            sh.scale[slot][1][lane & 7] = __log2f(vs);
            sh.scale[slot][2][lane & 7] = __frcp_rn(vs);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.meta[slot]);
        }
      }
      e_base += 2 * n;
      tiles_done += n;
      return ok;
      });
      if (!ok) {  // copies in flight land before the block leaves
        for (int i = 0; i < kBuf; ++i)
          for (int ph = 0; ph < 2; ++ph) mbar_wait_limited(BITS == 16 ? &sh.full[i] : &sh.raw_full[side * kBuf + i], ph);
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------------------- MMA issue
      constexpr uint32_t kShapeS = mma_shape(BITS == 16, kTok, false), kShapeO = mma_shape(BITS == 16, D, true);
      const uint32_t leader = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t q_desc = operand(__shfl_sync(0xffffffffu, q_smem, 0), 16, 1024);
      const uint32_t ring_u = __shfl_sync(0xffffffffu, ring, 0);
      auto score = [&](int t, int slot) {
        const uint64_t qd = q_desc + (TILES == 2 ? t * (C::kQBytes >> 4) : 0);
        const uint64_t kd = operand(__shfl_sync(0xffffffffu, ring_u + slot * C::kTileBytes, 0), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          constexpr int kHalf = kTok * 128 >> 4;
          const int off = kk / 4 * kHalf + kk % 4 * 2;
          tc_mma_ss(tm + 128 * t, qd + off, kd + off, kShapeS, kk > 0, leader);
        }
      };
      auto values = [&](int t, int slot, bool add, int from) {
        const uint64_t vd = operand(__shfl_sync(0xffffffffu, ring_u + slot * C::kTileBytes, 0), kTok * 128, 1024);
#pragma unroll
        for (int kk = from; kk < from + kTok / 32; ++kk)
          tc_mma_ts(tm + 256 + 128 * t, tm + 128 * t + kk * 8, vd + kk * (2048 >> 4), kShapeO, add || kk > 0, leader);
      };
      auto ready = [&](int e) { return wait(sh, &sh.full[e % SLOTS], (e / SLOTS) & 1); };
      auto seen = [&](int e) { return mbar_test(&sh.full[e % SLOTS], (e / SLOTS) & 1); };
      uint32_t q_phase = 0, p_phase = 0;  // p_phase: a bit per lane
      int e_base = 0;
      walk([&](const Unit& u, int64_t) {
        const int n = u.n;
        if (n == 0) return true;
        bool ok = true;
        for (int t = 0; t < 2 && ok; ++t) {
          if (TILES == 2 || t == 0) ok = wait(sh, &sh.q_ready[t], q_phase);
          if (count_of(t, n) == 0) break;
          const int e = e_base + at_k(first_of(t));
          ok = ok && ready(e);
          if (!ok) break;
          tc_fence_after();
          score(t, e % SLOTS);
          tc_commit(&sh.s_full[t], leader);
          if (TILES == 1 || t == 1) tc_commit(&sh.empty[e % SLOTS], leader);
        }
        q_phase ^= 1u;
        // V of tile j and K of the lane's next tile; looked at ahead of time, between two products' issue, where a wait
        // costs nothing
        bool ahead = false;
        for (int j = 0; j < n && ok; ++j) {
          const int ev = e_base + at_v(j, n), vslot = ev % SLOTS;
          const bool next = j + kStep < n;
          const int ek = next ? e_base + at_k(j + kStep) : 0, kslot = ek % SLOTS;
          if (!ahead) ok = ready(ev) && (!next || ready(ek));
#pragma unroll
          for (int v = 0; v < TILES; ++v) {
            const int t = TILES == 2 ? v : j & 1;
            const uint32_t phase = p_phase >> t & 1u;
            p_phase ^= 1u << t;
            ok = ok && wait(sh, &sh.p_half[t], phase);
            if (!ok) break;
            tc_fence_after();
            values(t, vslot, TILES == 2 ? j > 0 : j > 1, 0);
            ok = wait(sh, &sh.p_ready[t], phase);
            if (!ok) break;
            tc_fence_after();
            values(t, vslot, true, kTok / 32);
            if (v == TILES - 1) {
              tc_commit(&sh.empty[vslot], leader);
              ahead = __all_sync(0xffffffffu, j + 1 < n && seen(e_base + at_v(j + 1, n)) && (j + 1 + kStep >= n || seen(e_base + at_k(j + 1 + kStep))));
            }
            if (next) score(t, kslot);
            tc_commit(&sh.s_full[t], leader);
          }
          if (ok && next) tc_commit(&sh.empty[kslot], leader);
        }
        e_base += 2 * n;
        return ok;
      });
      __syncwarp();
    } else if (BITS == 16 ? warp == 10 : warp >= 12) {
      if constexpr (BITS == 16) {
        // ------------------------------------------------------------------ the last V tile's end
        uint32_t phase = 0;  // a bit per slot
        int e_base = 0;
        walk([&](const Unit& u, int64_t) {
          const int n = u.n;
          if (tail_of(u)) {
            const int slot = (e_base + 2 * n - 1) % SLOTS;
            // from the first token that no row sees
            const int from = visible_of(u.pos_last, u.s.kv_len, a.window, a.sinks).hi - u.tl.at(u.t_begin + n - 1) * kTok;
            const bool ok = wait(sh, &sh.tail[slot], phase >> slot & 1u);
            phase ^= 1u << slot;
            if (ok) {
              for (int h = 0; h < D / 64; ++h)
                for (int i = from * 8 + lane; i < kTok * 8; i += 32)
                  *(reinterpret_cast<uint4*>(generic + (ring - smem) + slot * C::kTileBytes + h * kTok * 128) + i) = make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.full[slot]);
            if (!ok) return false;
          }
          e_base += 2 * n;
          return true;
        });
      } else {
        // ------------------------------------------------------------------ 8-bit codes -> fp16
        // A warp takes 16 rows of a half tile, a quarter of it 4 neighbouring chunks of two rows that differ in bits 0 and 2: then
        // neither the reads nor the writes of the swizzled tiles meet in a bank.
        constexpr int kHalves = D / 64, kPer = 2 * kHalves;  // 16-byte chunks of codes per thread and half tile
        const int w4 = warp - 12, pair = lane >> 3, r8 = lane & 4 ? pair ^ 5 : pair;
        uint32_t from[kPer], to[kPer];  // offsets in the half tile and in the operand tile's half
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int r = w4 * 16 + i / kHalves * 8 + r8, h = i % kHalves, c = h * 4 + (lane & 3);
          from[i] = swizzled<(D < 128 ? 64 : 128)>(0, kTok, r, c);
          to[i] = h * kTok * 128 + r * 128 + (((2 * (lane & 3)) ^ (r & 7)) << 4);
        }
        int e_base = 0;
        walk([&](const Unit& u, int64_t) {
        const int n = u.n, blk_hi = visible_of(u.pos_last, u.s.kv_len, a.window, a.sinks).hi;
        bool ok = true;
        for (int i = 0; i < 2 * n && ok; ++i) {
          const int e = e_base + i, slot = e % SLOTS;
          if (e >= SLOTS) ok = wait(sh, &sh.empty[slot], (e / SLOTS - 1) & 1);
          const bool is_v = i > 0 && ((i & 1) == 0 || i == 2 * n - 1);
          const int j = !is_v ? (i + 1) / 2 : i == 2 * n - 1 ? n - 1 : i / 2 - 1;           // its token tile
          const int seen = is_v ? blk_hi - u.tl.at(u.t_begin + j) * kTok : kTok;            // tokens that some row sees
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            const int x = 2 * (e_base / 2 + j) + half, buf = (is_v ? C::kRawSide : 0) + x % C::kRawSide;
            ok = ok && wait(sh, &sh.raw_full[buf], (x / C::kRawSide) & 1);
            if (!ok) break;
            const uint8_t* src = generic + (raw - smem) + buf * C::kRawBytes;
            uint8_t* dst = generic + (ring - smem) + slot * C::kTileBytes + half * 64 * 128;
            uint4 w[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) w[i] = *reinterpret_cast<const uint4*>(src + from[i]);
            if (seen < kTok) {
#pragma unroll
              for (int i = 0; i < kPer; ++i)
                if (half * 64 + w4 * 16 + i / kHalves * 8 + r8 >= seen) w[i] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              uint4 lo, hi;
              e4m3_to_f16x4(w[i].x, &lo.x, &lo.y);
              e4m3_to_f16x4(w[i].y, &lo.z, &lo.w);
              e4m3_to_f16x4(w[i].z, &hi.x, &hi.y);
              e4m3_to_f16x4(w[i].w, &hi.z, &hi.w);
              *reinterpret_cast<uint4*>(dst + to[i]) = lo;
              *reinterpret_cast<uint4*>(dst + (to[i] ^ 16)) = hi;
            }
            fence_proxy_async_smem();
            mbar_arrive(&sh.full[slot]);
            mbar_arrive(&sh.raw_empty[buf]);  // not before the stores, which wait for the loads' values: the next copy overwrites them
          }
        }
        e_base += 2 * n;
        return ok;
        });
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }

  if (sh.odd != 0 && sh.failed == 0) look_again<D, BITS, TILES>(a, sh);
}

// Joins the parts of the units that the cuts met: a block per record and eight rows, a warp per row.
template <int D, int BITS, int TILES>
__global__ void __launch_bounds__(256) k_attend_many_join(const AttendParams a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PartRecord rec = *(reinterpret_cast<const PartRecord*>(a.part) + blockIdx.x);
  if (!rec.valid) return;
  const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
  const SeqRows s = seq_rows(a.c, rec.b);
  const int gr = rec.qb * TILES * kRows + r;
  if (gr >= s.n * a.group) return;
  constexpr int E = D / 32;
  const int64_t row = (int64_t)r * (D + 4);
  auto part = [&](int c) { return part_of(a, c, c == (int)blockIdx.x ? 1 : 0, TILES * kRows, D) + row; };
  float mx = -INFINITY;
  for (int c = blockIdx.x + lane; c <= rec.last; c += 32) mx = fmaxf(mx, part(c)[D]);
  mx = warp_max(mx);
  float l = 0.f, o[E];
  bool lost = false, spoilt = false, seen = false;
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.f;
#pragma unroll 4
  for (int c = blockIdx.x; c <= rec.last; ++c) {
    const float* q = part(c);
    const float4 ml = *reinterpret_cast<const float4*>(q + D);
    lost |= ml.z == kPartLost;
    spoilt |= ml.z == kPartSpoilt;
    seen |= ml.z == kPartSeen;
    const float f = ml.x == mx ? 1.f : exp2_fast(ml.x - mx);
    l = fmaf(ml.y, f, l);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 v = *reinterpret_cast<const float2*>(q + lane * E + i);
      o[i] = fmaf(v.x, f, o[i]);
      o[i + 1] = fmaf(v.y, f, o[i + 1]);
    }
  }
  float odd = l * 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) odd = fmaf(o[i], 0.f, odd);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (__any_sync(0xffffffffu, odd != 0.f)) {
    // no part says so: the join itself passed fp32's range; NaN out of parts without one: an infinity met a weight of zero, or its opposite
    bool nan = false, had_nan = false;
#pragma unroll
    for (int i = 0; i < E; ++i) nan |= isnan(o[i] * inv);
    for (int c = blockIdx.x; c <= rec.last; ++c) {
      const float* q = part(c);
      had_nan |= isnan(q[D + 1]);
#pragma unroll
      for (int i = 0; i < E; ++i) had_nan |= isnan(q[lane * E + i]);
    }
    spoilt |= !seen || (__any_sync(0xffffffffu, nan) && !__any_sync(0xffffffffu, had_nan));
    if (row_end(lost, spoilt) == RowEnd::again) {
      attend_row<D, BITS>(a, rec.b, s, gr / a.group, rec.kvh * a.group + gr % a.group, lane);
      return;
    }
  }
  uint16_t* dst = a.out + row_offset(a, s.first, rec.kvh, gr, a.o_token, a.o_head) + lane * E;
#pragma unroll
  for (int i = 0; i < E; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = l == 0.f ? 0u : pack_bf16(o[i] * inv, o[i + 1] * inv);
}

// Bytes of workspace: where the longest lengths that the sizes allow would have units cut.
template <int D, int TILES>
int64_t many_bytes(const AttendParams& a) {
  const int64_t blocks = ((int64_t)a.part_rows + TILES * kRows - 1) / (TILES * kRows) * a.c.n_kv_heads * a.c.batch;
  int64_t tokens = (int64_t)a.c.max_pages << a.c.page_shift;
  if (a.window > 0) tokens = std::min<int64_t>(tokens, (int64_t)a.window + TILES * kRows / a.group + a.sinks + 2 * kTok);
  const int64_t most = tokens / kTok + 1 + kUnitCost;
  if (most < 2 * kMinShare && blocks * most < (int64_t)kMinShare * kSms) return 0;
  return part_bytes(kSms, TILES * kRows, D);
}

template <int D, int BITS, int TILES>
cudaError_t launch(AttendParams a, cudaStream_t st) {
  using C = Cfg<D, BITS, TILES>;
  PageMaps maps;
  if (make_page_maps(a.c, D, BITS, std::min(a.c.page_size, BITS == 16 ? kTok : kTok / 2), &maps)) return cudaErrorInvalidValue;
  auto* f = k_attend_many<D, BITS, TILES>;
  static std::atomic<uint64_t> prepared{0};
  cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(f), C::kBytes, &prepared);
  if (e != cudaSuccess) return e;
  const int64_t bytes = many_bytes<D, TILES>(a);
  if (bytes == 0 || bytes > a.part_bytes) a.part = nullptr;
  f<<<kSms, C::kThreads, C::kBytes, st>>>(a, maps);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.part) return e;
  return launch_after(k_attend_many_join<D, BITS, TILES>, dim3(kSms, TILES * kRows / 8), 256, st, a);
}

template <int D, int BITS>
cudaError_t launch_rows(const AttendParams& a, cudaStream_t st) {
  return a.part_rows <= kRows ? launch<D, BITS, 1>(a, st) : launch<D, BITS, 2>(a, st);
}

}  // namespace

cudaError_t launch_attend_many(const AttendParams& a, int head_dim, int kv_bits, cudaStream_t st) {
  if (head_dim == 128) return kv_bits == 16 ? launch_rows<128, 16>(a, st) : launch_rows<128, 8>(a, st);
  return kv_bits == 16 ? launch_rows<64, 16>(a, st) : launch_rows<64, 8>(a, st);
}

int64_t attend_many_bytes(const AttendParams& a, int head_dim) {
  if (head_dim == 128) return a.part_rows <= kRows ? many_bytes<128, 1>(a) : many_bytes<128, 2>(a);
  return a.part_rows <= kRows ? many_bytes<64, 1>(a) : many_bytes<64, 2>(a);
}

}  // namespace clo
