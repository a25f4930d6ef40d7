// sv_attn_i4.cuh -- tree attention over a paged cache of 4 bits on the tensor cores
// (tcgen05), for head dimensions 64 and 128.
//
// Rows.  The n new tokens and the G query heads that share a KV head form one
// matrix of n * G rows; a unit is up to 64 of them, whatever tokens they belong to.
//
// Keys stand where a product's 128 rows are: S^T = K Q^T and O^T = V^T P^T, with
// 128 keys and 128 (64) dimensions in tensor-memory lanes and N = 16 .. 64 query
// rows in columns.  With queries in the lanes a chain of six tokens and eight heads
// fills 48 of 128, and 128 keys take 1024 cycles of the tensor cores; so they take
// 8 N, 384 for that chain and 128 for a token.
//
// Widening.  Both cache operands go from shared memory through registers into
// tensor memory, as the products' A operand: nothing is written back to shared
// memory, whose bandwidth (136 KB for 128 keys otherwise, 1060 cycles; HBM delivers
// them in 760) would be the bound.  A code's four bits are a 16-bit number's
// fraction, 16 + c or 64 + c, and one multiply-add makes them (c - 8) f for two
// codes, exactly (7 bits).  Pairs of codes:
//   K: one key's elements i and i + 4 of eight lie 16 bits apart, so that a
//      thread (lane = key) unpacks its row in place; the queries' elements
//      are put in the same order, 0 4 1 5 2 6 3 7, on their way into shared memory;
//   V: the lanes are dimensions and the pairs two keys.  ldmatrix transposes units
//      of 16 bits, four codes of a key: a thread gets those of two adjacent keys,
//      16 bits apart again, and tcgen05.st with 16x128b puts each of the
//      four dimensions into its lane.  Lane 32 q + 8 i + g holds dimension 32 q +
//      4 g + i, whose scale is q's.
// fp16 numbers are kept at 1/16 of their value: 72 f is then a number of the type.
//
// Softmax.  A thread has one key and every second eight rows: two groups of four warps.  The
// rows' references m are shared by the 128 keys and live in shared memory; P is
// 2^(x - m), and only when a score exceeds its reference by more than 2^8 (a vote of
// the group, once a tile) are the references raised and O^T's columns rescaled; that
// path also does the first tile of a unit.  A thread's parts of the rows' sums are
// columns of tensor memory, not registers: then every loop over rows has one copy of
// its body.  (Unrolled, the code of all roles together missed the instruction cache:
// 642 us for 128 requests, where the loops then took 382.)
// P has the type of the queries, as both operands of a product have one type: half a
// step of 2^-8 in bf16, whose range keeps what lies far below the largest, 2^-11 in fp16.
// The sums take the fp32 values.  Results are off from 64 bits by 0.0023 for trees (one
// rounding to bf16: 0.0017), 0.00026 in fp16 (0.00021), in the mean relative to them.
//
// Roles.  K, V, their products and the softmax are pipelined through two places each
// (P: three) in tensor or shared memory; even and odd tiles have producers and widening
// warps of their own, for each is a chain of latencies.  (One producer for K and one for
// V took 1800 cycles a tile and bound the kernel; copies by the widening warps
// themselves, without producers, were no faster: 384 us for 128 requests, 364 with them.)
//
// Work, ranges, cut units, marked units and the second kernel are those of
// sv_attn_tc.cuh, with one range for a thread block.
//
// Measured, both kernels together:
//   128 x 6 tokens, 64 heads on 8 of 128, 500-8000 keys  358 us, 1.7 TB/s: a softmax
//                                                warp's chain, about 1300 cycles a tile
//                                                (wait, vote, fence) and 400 per 8 rows
//   16 trees of 64, 32 on 8, 1000-8000 keys      215 us, 260 TFLOP/s: the same; units of
//                                                64 rows take the keys four times (e4m3:
//                                                108 us, each key widened once)
//   131071 keys, 1 token, 64 on 8                57 us, 2.5 TB/s: the same chain, in one
//                                                group: 8 rows leave the other none
//   500 keys, 1 token, 14 on 2 of 64             10 us: start, first data, join
#pragma once

#include "sv_attn_tc.cuh"

namespace svp {
namespace i4 {

constexpr int kT = 128;          // keys of a tile
constexpr int kPlaces = 3;       // of P
constexpr int kRows = 64;        // query rows of a unit, at most
constexpr int kUnit = 16;        // N is a multiple of it
constexpr int kChunk = 8;        // rows in registers at once
constexpr int kThreads = 992;
// Warps: 0 - 7 softmax, 8 - 15 widen K and 16 - 23 V, four for the even and four for
// the odd tiles; the producers of K's even and odd tiles, and of V's; the products
// Q K^T and P V; the queries.
constexpr int kWarpK = 8, kWarpV = 16, kWarpLoad = 24, kWarpS = 28, kWarpO = 29, kWarpQ = 30;

template <int D>
struct Shape {
  static constexpr int kRow = D / 2, kSRow = D / SV_KV_GROUP;     // bytes of a key's codes and scales
  static constexpr int kData = kT * kRow, kScale = kT * kSRow;
  static constexpr int kStages = D == 128 ? 4 : 8;                // of each of the four rings: K, V, even, odd
  static constexpr int kQHalf = kRows * 128;                      // 64 columns of the queries
  static constexpr int kQBytes = D / 64 * kQHalf, kPBytes = kT * 128;
  static constexpr int kSmem = 2 * kQBytes + kPlaces * kPBytes + 4 * kStages * (kData + kScale);
  static constexpr int kGroups = D / SV_KV_GROUP;                 // warps that widen a tile's V
  // TMEM columns: two of K, V and S, O and the sums.
  static constexpr uint32_t kColK = 0, kColV = 128, kColS = 256, kColO = 384, kColL = 448;
};

template <int N>
struct BarSet {
  uint64_t raw[4][N], empty[4][N];  // the rings: K even, K odd, V even, V odd
  uint64_t k_ready[2], k_free[2], v_ready[2], v_free[2], s_full[2], p_ready[4], o_done[4], q_full[2], q_empty[2], drain[2];
};

// Rows' references, shared by the softmax warps.
struct Refs {
  alignas(16) float minus[kRows];   // -m, or the largest float where nothing was seen
  alignas(16) float factor[kRows];
  float m[kRows], top[4][kRows];    // top: of a warp's keys; in the end its part of the sums
  int dead[2];                      // a wait of the group gave up
};

__device__ __forceinline__ void tc_ld8(uint32_t addr, uint32_t *r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : SVP_R8(r, 0)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tc_st8(uint32_t addr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), SVP_W8(r, 0)
               : "memory");
}
// 16 lanes of 16 columns: registers 2 j and 2 j + 1 of thread t go to lanes t / 4 and
// t / 4 + 8, column 4 j + t % 4.
__device__ __forceinline__ void tc_st_16x128b_x4(uint32_t addr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), SVP_W8(r, 0)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Whether any of a softmax group's four warps says so.
__device__ __forceinline__ bool vote(int group, bool x) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %2, 0; barrier.cta.red.or.aligned.pred q, %1, 128, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"(group + 1), "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(group + 1) : "memory");
}
__device__ __forceinline__ float warp_top(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// wait_warp with few instructions: five roles share a scheduler, and waiting took a
// quarter of what it issued.
__device__ __forceinline__ bool wait_for(const uint64_t *bar, uint32_t parity, uint32_t *err) {
  const uint32_t at = sv::smem_addr(bar);
  uint32_t done;
  asm volatile(
      "{ .reg .pred p, q; .reg .u32 n;\n\t"
      "mov.u32 n, 64;\n"
      "W%=: mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra D%=;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra W%=;\n"
      "D%=: selp.u32 %0, 1, 0, p; }"
      : "=r"(done)
      : "r"(at), "r"(parity & 1u)
      : "memory");
  return __all_sync(kFull, done) || wait_long(at, parity & 1u, err);
}

template <typename Q>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (Q::kIsBf16) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename Q>
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  if constexpr (Q::kIsBf16) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// Two scale bytes (in the low halves of 16 bits) as f, or f / 16 in fp16 (a subnormal
// number holds it too); not those that are NaN.
template <typename Q>
__device__ __forceinline__ uint32_t scale2(uint32_t s) {
  if constexpr (Q::kIsBf16) return s * 0x10u + 0x38803880u;                        // exponent + 113
  else return mul2<F16>(s * 0x80u + 0x04000400u, 0x2c002c00u);
}
// Not 0 where one of the two bytes is NaN.
__device__ __forceinline__ uint32_t odd2(uint32_t s) {
  constexpr uint32_t up = 255u - SV_KV_I4_MAX_SCALE;
  return (s + (up | up << 16)) & 0x01000100u;
}
// What takes (16 + c) f (bf16) or (64 + c) f (fp16) to (c - 8) f.
template <typename Q>
__device__ __forceinline__ uint32_t offset2(uint32_t f) {
  return mul2<Q>(f, Q::kIsBf16 ? 0xc1c0c1c0u : 0xd480d480u);                       // -24, -72
}
// (x & mask) | base as one instruction (written as C++ it became two: a mask and a
// base are two constants).
template <uint32_t mask>
__device__ __forceinline__ uint32_t pick(uint32_t x, uint32_t base) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "n"(mask), "r"(base));
  return r;
}
// Codes i and i + 4 of a word's eight, i = 0 .. 3, times their scales f (two,
// for the codes' places).  A multiplication by 8 or 16 is a shift on the other pipe
// than the masks': of the two, half an instruction a cycle each, 6 take a product or
// a shift and 5 (bf16: 7) a mask or a permutation.
template <typename Q>
__device__ __forceinline__ void wide8(uint32_t w, uint32_t f, uint32_t off, uint32_t &o0, uint32_t &o1, uint32_t &o2,
                                      uint32_t &o3) {
  const uint32_t x = __byte_perm(w, 0, 0x2301);   // codes 2, 3 (6, 7) in the places of 0, 1
  if constexpr (Q::kIsBf16) {
    constexpr uint32_t m = 0x00780078u, b = 0x41804180u;
    const uint32_t w1 = w >> 1, x1 = __byte_perm(w1, 0, 0x2301);
    o0 = fma2<Q>(pick<m>(w * 8u, b), f, off);
    o1 = fma2<Q>(pick<m>(w1, b), f, off);
    o2 = fma2<Q>(pick<m>(x * 8u, b), f, off);
    o3 = fma2<Q>(pick<m>(x1, b), f, off);
  } else {
    constexpr uint32_t m = 0x00f000f0u, b = 0x54005400u;
    o0 = fma2<Q>(pick<m>(w * 16u, b), f, off);
    o1 = fma2<Q>(pick<m>(w, b), f, off);
    o2 = fma2<Q>(pick<m>(x * 16u, b), f, off);
    o3 = fma2<Q>(pick<m>(x, b), f, off);
  }
}
template <typename Q>
constexpr float kUndo = Q::kIsBf16 ? 1.f : 16.f;   // a widened number's value, in units of itself

// Byte offset of 16-byte column c of a row of the raw tile, as TMA swizzles rows of
// 64 (32) bytes.
template <int D>
__device__ __forceinline__ int raw_at(int row, int c) {
  return row * (D / 2) + ((D == 128 ? c ^ (row >> 1 & 3) : c ^ (row >> 2 & 1)) << 4);
}

template <typename Q, int D>
__global__ void __launch_bounds__(kThreads, 1) sv_attn_i4_kernel(const __grid_constant__ TcParams p) {
  using S = Shape<D>;
  constexpr int R = S::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ BarSet<R> bars;
  __shared__ Refs refs;
  __shared__ uint32_t tmem_slot;
  __shared__ Walk sh_walk;
  __shared__ int seg_bad[kSegRing];                 // holds 1 + a marked segment's number
  __shared__ uint32_t marks[kMarkBits / 32];        // whole units to recompute
  __shared__ int4 v_meta[2][R];                     // of a stage of V: live and fresh keys, the segment
  __shared__ alignas(16) uint32_t v_scale[8][kT / 2];  // a V warp's scales: those of keys 8 m + 2 j and + 1 at 16 j + m

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t *const sq = smem, *const sp = sq + 2 * S::kQBytes, *const raw = sp + kPlaces * S::kPBytes;
  uint8_t *const scales = raw + 4 * R * S::kData;   // of the rings' stages, like the data
  const AttnParams &a = p.a;

  if (sv::smem_addr(smem) & 1023u) {                // never: the swizzle would not match
    report(p.err, SV_FAULT_TIMEOUT);
    return;
  }
  if (warp == kWarpS) tc_alloc(sv::smem_addr(&tmem_slot), 512);
  if (tid == 0) {
    for (int r = 0; r < 4; ++r)
      for (int i = 0; i < R; ++i) {
        sv::mbar_init(sv::smem_addr(&bars.raw[r][i]), 33);    // 32 lanes' scales, the data
        sv::mbar_init(sv::smem_addr(&bars.empty[r][i]), r < 2 ? 4 : S::kGroups);
      }
    for (int i = 0; i < 2; ++i) {
      sv::mbar_init(sv::smem_addr(&bars.k_ready[i]), 4);
      sv::mbar_init(sv::smem_addr(&bars.k_free[i]), 1);
      sv::mbar_init(sv::smem_addr(&bars.v_ready[i]), S::kGroups);
      sv::mbar_init(sv::smem_addr(&bars.v_free[i]), 1);
      sv::mbar_init(sv::smem_addr(&bars.s_full[i]), 1);
      // P is up to three tiles ahead of its products: with barriers for two of them a
      // phase could end twice before the products' warp looks at it.
      for (int k = i; k < 4; k += 2) {
        sv::mbar_init(sv::smem_addr(&bars.p_ready[k]), 8);
        sv::mbar_init(sv::smem_addr(&bars.o_done[k]), 1);
      }
      sv::mbar_init(sv::smem_addr(&bars.q_full[i]), 1);
      sv::mbar_init(sv::smem_addr(&bars.q_empty[i]), 1);
    }
    sv::mbar_init(sv::smem_addr(&bars.drain[0]), 1);
    sv::mbar_init(sv::smem_addr(&bars.drain[1]), 1);
    for (int i = 0; i < kSegRing; ++i) seg_bad[i] = 0;
    refs.dead[0] = refs.dead[1] = 0;
    sv::fence_mbar_init();
  }
  if (warp == 3)
    for (int i = lane; i < kMarkBits / 32; i += 32) marks[i] = 0;
  if (tid == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.vmap) : "memory");
  }
  if (warp == 2) {  // addresses only: the values may still be written
    const int at = lane * 32 < a.bt.B ? lane * 32 : 0;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.bt.seq_lens + at));
    if (a.bt.new_lens) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.bt.new_lens + at));
    if (a.c.max_blocks > 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.c.tables));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  sv::pdl_wait();
  sv::pdl_launch_dependents();

  const RowUnits unit{p.unit_rows};
  uint32_t *const err = p.err;
  bool ok = true, marked = false;
  if (warp == kWarpQ) {
    Walk w;
    int total;
    begin_walk(a, unit, static_cast<int>(blockIdx.x), p.ranges, w, total);
    if (lane == 0) {
      sh_walk = w;
      // Range 0 is written even if there are no tiles: its total says so.
      if (w.on || blockIdx.x == 0) p.cuts[blockIdx.x] = Cut{w.b, w.h, w.mp, w.r.n, w.t0, w.r.kt, total, 0};
    }
  }
  __syncthreads();

  Walk walk = sh_walk;
  const int wq = warp & 3;                          // TMEM lanes 32 wq ..
  const uint32_t lanes = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  const auto rows_of = [&](const Walk &w) { return min(w.r.n * a.G - w.mp * p.unit_rows, p.unit_rows); };
  if (warp < kWarpK) {
    // ---------------------------------------------------------- softmax ----
    const int grp = warp >> 2, my = tid & 127;      // key of the tile; in the end a lane's dimension
    constexpr float kHead = Q::kIsBf16 ? 0.f : 7.f;   // fp16 probabilities begin at 2^7
    constexpr float kUp = kHead + 8.f;
    const float c = p.c * kUndo<Q>;
    const uint64_t c2 = f2_pack(c, c);
    uint32_t tiles = 0;
    const int swizzle = (my & 7) << 4;
    uint8_t *prow = sp + my * 128;                  // this key's place in the tile's P
    const int mine = (my / kChunk * 2 + grp) * kChunk + my % kChunk;   // the row that the thread looks after
#pragma unroll 1
    while (walk.on) {
      const Walk sg = walk;
      const Req &r = sg.r;
      const int nt = sg.t1 - sg.t0, seg = sg.seg;
      const int row0 = sg.mp * p.unit_rows, rows = rows_of(sg);
      // The group's rows of the unit: every second eight, from g0 on, whatever the unit's
      // size: a group may be done with a unit before the other one, and what it then
      // writes (references, sums) must not be the other's.  There may be none.
      const int g0 = grp * kChunk, g1 = (rows + kChunk - 1) / kChunk * kChunk;
      const int full_end = sg.new0();               // every row sees these
      const uint32_t col_o = lanes + S::kColO, col_l = lanes + S::kColL;
#pragma unroll 1
      for (int j = 0; j < nt; ++j, ++tiles) {
        const uint32_t buf = tiles & 1, round = tiles >> 1;
        const uint32_t col_s = lanes + S::kColS + 64u * buf;
        const int k0 = (sg.t0 + j) * kT;
        const bool masked = k0 + kT > full_end, fast = j > 0;
        const auto put = [&](int row, const uint32_t (&pk)[kChunk / 2]) {
          *reinterpret_cast<uint4 *>(prow + ((row / kChunk * 16) ^ swizzle)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        };
        // Which rows see the thread's key, while S is being computed.
        uint64_t vis = ~0ull;
        if (masked) {
          const int pos = k0 + my, cn = pos - r.L;
          if (pos >= r.kv_end) {
            vis = 0;
          } else if (cn >= 0) {
            if (a.mask) {
              vis = 0;
              const uint8_t *col = a.mask + sg.b * a.msb + cn;
              const int t0 = row0 / a.G, t1 = (row0 + rows - 1) / a.G;
#pragma unroll 4
              for (int t = t0; t <= t1; ++t) {
                const int lo = max(t * a.G - row0, 0), hi = min((t + 1) * a.G - row0, rows);   // hi - lo in 1 .. 64
                if (ld8(col + static_cast<int64_t>(t) * a.bt.T)) vis |= (~0ull >> (64 - (hi - lo))) << lo;
              }
            } else {
              const int64_t lo = static_cast<int64_t>(cn) * a.G - row0;
              vis = lo >= 64 ? 0 : lo > 0 ? ~0ull << lo : ~0ull;
            }
          }
        }
        if (g0 >= rows) {                           // no row: in step with the other group, no more
          if (ok && !(ok = wait_for(&bars.s_full[buf], round, err))) refs.dead[grp] = 1;   // seen below by all
          if (ok && lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.p_ready[tiles & 3]));
          prow += S::kPBytes;
          if (prow >= raw) prow -= kPlaces * S::kPBytes;
          continue;
        }
        const bool good = wait_for(&bars.s_full[buf], round, err);   // and P's place is free
        tc_fence_after();
        float top = -INFINITY;
        const auto hide = [&](int row, uint32_t (&x)[kChunk]) {
          const uint32_t bits = static_cast<uint32_t>(vis >> row);
#pragma unroll
          for (int k = 0; k < kChunk; ++k)
            if (!(bits >> k & 1u)) x[k] = 0xff800000u;
        };
        if (fast && good) {
          // A row that has seen nothing yet has the largest float for its -m: any score
          // above -inf then asks for a reference.
#pragma unroll 1
          for (int row = g0; row < g1; row += 2 * kChunk) {
            uint32_t x[kChunk], l[kChunk];
            tc_ld8(col_s + row, x);
            tc_ld8(col_l + row, l);
            const ulonglong2 n0 = *reinterpret_cast<const ulonglong2 *>(&refs.minus[row]);
            const ulonglong2 n1 = *reinterpret_cast<const ulonglong2 *>(&refs.minus[row + 4]);
            const uint64_t nm[4] = {n0.x, n0.y, n1.x, n1.y};
            tc_wait_ld(x);
            tc_wait_ld(l);
            if (masked) hide(row, x);
            uint32_t pk[kChunk / 2];
#pragma unroll
            for (int k = 0; k < kChunk; k += 2) {
              float y0, y1, s0, s1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), c2, nm[k / 2]), y0, y1);
              top = fmaxf(top, fmaxf(y0, y1));
              y0 = sv::ex2(y0);
              y1 = sv::ex2(y1);
              f2_unpack(f2_add(f2_pack(__uint_as_float(l[k]), __uint_as_float(l[k + 1])), f2_pack(y0, y1)), s0, s1);
              l[k] = __float_as_uint(s0);
              l[k + 1] = __float_as_uint(s1);
              pk[k / 2] = pack2<Q>(y0, y1);
            }
            tc_st8(col_l + row, l);
            put(row, pk);
          }
        }
        if (!good) refs.dead[grp] = 1;
        // A warp whose wait gave up takes part in the others' barriers until all have seen it.
        if (!fast || vote(grp, !good || top > kUp)) {
          tc_wait_st();
          if (good) {
#pragma unroll 1
            for (int row = g0; row < g1; row += 2 * kChunk) {
              uint32_t x[kChunk];
              tc_ld8(col_s + row, x);
              if (fast) {
                // The sums without what was just added; where that exceeds 2^100, what was
                // there before is nothing against what the raised reference brings.
                uint32_t l[kChunk];
                tc_ld8(col_l + row, l);
                tc_wait_ld(x);
                tc_wait_ld(l);
                if (masked) hide(row, x);
#pragma unroll
                for (int k = 0; k < kChunk; ++k) {
                  const float e = sv::ex2(fmaf(__uint_as_float(x[k]), c, refs.minus[row + k]));
                  l[k] = e >= 0x1p100f ? 0u : __float_as_uint(__uint_as_float(l[k]) - e);
                }
                tc_st8(col_l + row, l);
              } else {
                tc_wait_ld(x);
                if (masked) hide(row, x);
              }
              float best = -INFINITY;
#pragma unroll
              for (int k = 0; k < kChunk; ++k) {
                const float t = warp_top(__uint_as_float(x[k]) * c);
                if (lane == k) best = t;
              }
              if (lane < kChunk) refs.top[wq][row + lane] = best;
            }
            // The products of the tile before may still run.
            if (j > 0 && !wait_for(&bars.o_done[(tiles - 1) & 3], (tiles - 1) >> 2, err)) refs.dead[grp] = 1;
          }
          tc_wait_st();
          group_sync(grp);
          if (*const_cast<volatile int *>(&refs.dead[grp])) {
            ok = false;
            break;
          }
          const int row = mine;
          bool up = false;
          if (row < g1) {
            const float mt = fmaxf(fmaxf(refs.top[0][row], refs.top[1][row]), fmaxf(refs.top[2][row], refs.top[3][row]));
            float m = j > 0 ? refs.m[row] : -INFINITY, f = 1.f;
            if (mt - kHead > m && !(mt - m <= kUp)) {
              f = sv::ex2(m - (mt - kHead));
              m = mt - kHead;
              up = j > 0;
            }
            refs.m[row] = m;
            refs.minus[row] = m == -INFINITY ? 3.402823466e38f : -m;
            refs.factor[row] = f;
          }
          up = vote(grp, up);
          tc_fence_after();
#pragma unroll 1
          for (int row = g0; row < g1; row += 2 * kChunk) {
            uint32_t x[kChunk], l[kChunk], pk[kChunk / 2];
            if (j > 0) {
              tc_ld8(col_l + row, l);
              tc_wait_ld(l);
            } else {
#pragma unroll
              for (int k = 0; k < kChunk; ++k) l[k] = 0;
            }
            if (up) {
              uint32_t o[kChunk];
              tc_ld8(col_o + row, o);
              tc_wait_ld(o);
#pragma unroll
              for (int k = 0; k < kChunk; ++k) {
                const float f = refs.factor[row + k];
                o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                l[k] = __float_as_uint(__uint_as_float(l[k]) * f);
              }
              tc_st8(col_o + row, o);
            }
            tc_ld8(col_s + row, x);
            tc_wait_ld(x);
            if (masked) hide(row, x);
#pragma unroll
            for (int k = 0; k < kChunk; k += 2) {
              // Where nothing was seen x is -inf: so is the sum, and P is 0.
              const float e0 = sv::ex2(fmaf(__uint_as_float(x[k]), c, refs.minus[row + k]));
              const float e1 = sv::ex2(fmaf(__uint_as_float(x[k + 1]), c, refs.minus[row + k + 1]));
              l[k] = __float_as_uint(__uint_as_float(l[k]) + e0);
              l[k + 1] = __float_as_uint(__uint_as_float(l[k + 1]) + e1);
              pk[k / 2] = pack2<Q>(e0, e1);
            }
            tc_st8(col_l + row, l);
            put(row, pk);
          }
        }
        fence_async_smem();
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.p_ready[tiles & 3]));
        prow += S::kPBytes;
        if (prow >= raw) prow -= kPlaces * S::kPBytes;
      }
      if (!ok && g0 < rows) break;                   // the whole group
      next_segment(a, unit, walk);

      // The warp's part of the rows' sums: a butterfly whose halves keep half of the rows each.
#pragma unroll 1
      for (int row = g0; row < g1; row += 2 * kChunk) {
        uint32_t l[kChunk];
        tc_ld8(col_l + row, l);
        tc_wait_ld(l);
        float v[kChunk];
#pragma unroll
        for (int k = 0; k < kChunk; ++k) v[k] = __uint_as_float(l[k]);
#pragma unroll
        for (int o = 16, h = kChunk / 2; h > 0; o >>= 1, h >>= 1) {
          const bool up = lane & o;
#pragma unroll
          for (int k = 0; k < h; ++k) {
            const float keep = up ? v[k + h] : v[k], send = up ? v[k] : v[k + h];
            v[k] = keep + __shfl_xor_sync(kFull, send, o);
          }
        }
        v[0] += __shfl_xor_sync(kFull, v[0], 2);
        v[0] += __shfl_xor_sync(kFull, v[0], 1);
        if (!(lane & 3)) refs.top[wq][row + (lane >> 2)] = v[0];
      }
      const uint32_t last = tiles - 1;
      if (!wait_for(&bars.o_done[last & 3], last >> 2, err)) refs.dead[grp] = 1;
      group_sync(grp);
      if (*const_cast<volatile int *>(&refs.dead[grp])) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool bad = seg_bad[seg % kSegRing] == seg + 1;
      const bool whole = sg.t0 == 0 && sg.t1 == r.kt;
      float *slot = nullptr;
      if (!whole)  // slot 0 of the range where the segment starts it, else slot 1
        slot = p.slots + (static_cast<size_t>(blockIdx.x) * 2 + (seg == 0 ? 0 : 1)) * p.slot_floats;
      const auto out_row = [&](int row) {
        const int t = (row0 + row) / a.G, g = row0 + row - t * a.G;
        return (static_cast<int64_t>(sg.b) * a.bt.T + t) * a.Hq + sg.h * a.G + g;
      };
      if (mine < rows) {
        const int row = mine;
        const float l = (refs.top[0][row] + refs.top[1][row]) + (refs.top[2][row] + refs.top[3][row]);
        const float m = l == 0.f ? -INFINITY : refs.m[row];
        // What O is multiplied by; 0 where the row has seen nothing.
        refs.factor[row] = whole ? (l == 0.f ? 0.f : kUndo<Q> / l) : kUndo<Q>;
        if (!whole) {
          slot[D * p.slot_rows + row] = m;
          slot[(D + 1) * p.slot_rows + row] = l;
        } else if (a.lse && !bad) {
          a.lse[out_row(row)] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
        }
      }
      if (tid == 0) {
        if (!whole) reinterpret_cast<int *>(slot)[(D + 2) * p.slot_rows] = bad ? 1 : 0;
        else if (bad) marks[seg / 32 % (kMarkBits / 32)] |= 1u << (seg % 32);
      }
      if (bad && whole) marked = true;
      group_sync(grp);
      const int dim = 32 * wq + 4 * (lane & 7) + (lane >> 3);
      if (!bad && wq < S::kGroups && g0 < rows) {
        float *const part = whole ? nullptr : slot + static_cast<size_t>(dim >> 2) * p.slot_rows * 4 + (dim & 3);
#pragma unroll 1
        for (int row = g0; row < rows; row += 2 * kChunk) {
          uint32_t o[kChunk];
          tc_ld8(col_o + row, o);
          tc_wait_ld(o);
          const float4 f0 = *reinterpret_cast<const float4 *>(&refs.factor[row]);
          const float4 f1 = *reinterpret_cast<const float4 *>(&refs.factor[row + 4]);
          const float fs[kChunk] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
          uint8_t *to = a.out + (out_row(row) * D + dim) * 2;
          int head = (row0 + row) % a.G;
#pragma unroll
          for (int k = 0; k < kChunk; ++k) {
            if (row + k < rows) {
              const float y = fs[k] == 0.f ? 0.f : __uint_as_float(o[k]) * fs[k];   // not 0 * O: it may be NaN
              if (whole) {
                store1<Q>(to, y);
                to += D * 2;
                if (++head == a.G) {
                  head = 0;
                  to += static_cast<int64_t>(a.Hq - a.G) * (D * 2);
                }
              } else {
                part[(row + k) * 4] = y;
              }
            }
          }
        }
      }
      tc_fence_before();   // O is read before the next P is announced
      group_sync(grp);     // and the factors before the next unit's
    }
  } else if (warp < kWarpV) {
    // ----------------------------------------------------------- K wideners ----
    const int my = wq * 32 + lane;                  // key of the tile
    const int n = count_of(walk), par = warp >> 2 & 1;
    const uint8_t *const ring = raw + par * R * S::kData, *const ring_s = scales + par * R * S::kScale;
    int st = 0;
    uint32_t round = 0, turn = 0;                   // of the ring, of the buffer
#pragma unroll 1
    for (int i = par; i < n; i += 2, ++turn) {
      if (!wait_for(&bars.raw[par][st], round, err)) break;
      const uint8_t *src = ring + st * S::kData, *sc = ring_s + st * S::kScale + my * S::kSRow;
      uint4 w = *reinterpret_cast<const uint4 *>(src + raw_at<D>(my, 0));
      uint32_t f4 = D == 128 ? *reinterpret_cast<const uint32_t *>(sc) : *reinterpret_cast<const uint16_t *>(sc);
      const bool nan = __any_sync(kFull, odd2(f4 & 0x00ff00ffu) | odd2(f4 >> 8 & 0x00ff00ffu));
      if (turn > 0 && !wait_for(&bars.k_free[par], turn - 1, err)) break;
      tc_fence_after();
      const uint32_t col = lanes + S::kColK + 64u * par;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        const uint4 next = *reinterpret_cast<const uint4 *>(src + raw_at<D>(my, ch + 1 & (D / 32 - 1)));
        const uint32_t s2 = __byte_perm(f4, 0, 0x4040);
        uint32_t f = scale2<Q>(s2);
        if (nan) f = odd2(s2) ? 0x7fff7fffu : f;
        f4 >>= 8;
        const uint32_t off = offset2<Q>(f);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) wide8<Q>(u[k], f, off, o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        tc_st16(col + 16 * ch, o);
        w = next;
      }
      __syncwarp();
      if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.empty[par][st]));
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.k_ready[par]));
      if (++st == R) {
        st = 0;
        ++round;
      }
    }
  } else if (warp < kWarpLoad) {
    // ----------------------------------------------------------- V wideners ----
    const int n = wq < S::kGroups ? count_of(walk) : 0, par = warp >> 2 & 1;
    const uint8_t *const ring = raw + (2 + par) * R * S::kData, *const ring_s = scales + (2 + par) * R * S::kScale;
    uint32_t *const mine = v_scale[warp - kWarpV];
    int st = 0;
    uint32_t round = 0, turn = 0;
#pragma unroll 1
    for (int i = par; i < n; i += 2, ++turn) {
      if (!wait_for(&bars.raw[2 + par][st], round, err)) break;
      const uint32_t src = sv::smem_addr(ring + st * S::kData);
      // The scales of this lane's keys 4 lane .. + 3, in pairs; 0 behind the last token.
      const int4 m = v_meta[par][st];
      const int live = m.x;
      uint32_t s01, s23;
      if constexpr (D == 128) {
        const uint4 v = *reinterpret_cast<const uint4 *>(ring_s + st * S::kScale + lane * 16);
        const uint32_t pick = wq * 0x1111u + 0x4400u;
        s01 = __byte_perm(v.x, v.y, pick) & 0x00ff00ffu;
        s23 = __byte_perm(v.z, v.w, pick) & 0x00ff00ffu;
      } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(ring_s + st * S::kScale + lane * 8);
        const uint32_t pick = wq * 0x1111u + 0x2200u;
        s01 = __byte_perm(v.x, 0, pick) & 0x00ff00ffu;
        s23 = __byte_perm(v.y, 0, pick) & 0x00ff00ffu;
      }
      uint32_t f01 = scale2<Q>(s01), f23 = scale2<Q>(s23);
      if (live < kT || __any_sync(kFull, odd2(s01) | odd2(s23))) {
        const int fresh = m.y, key = lane * 4;
        const auto put_right = [&](uint32_t &f, uint32_t s, int k) {
          uint32_t lo = f & 0xffffu, hi = f >> 16;
          if ((s & 255u) > SV_KV_I4_MAX_SCALE) {
            lo = 0x7fffu;
            // NaN among the new tokens: a row that does not see it must not meet it.
            if (k >= fresh && k < live) seg_bad[m.z % kSegRing] = m.z + 1;
          }
          if (s >> 16 > SV_KV_I4_MAX_SCALE) {
            hi = 0x7fffu;
            if (k + 1 >= fresh && k + 1 < live) seg_bad[m.z % kSegRing] = m.z + 1;
          }
          f = (k < live ? lo : 0u) | (k + 1 < live ? hi << 16 : 0u);
        };
        put_right(f01, s01, key);
        put_right(f23, s23, key + 2);
      }
      mine[(lane & 1) * 32 + (lane >> 1)] = f01;    // j = 0 or 2, m = lane / 2
      mine[(lane & 1) * 32 + 16 + (lane >> 1)] = f23;
      __syncwarp();
      if (turn > 0 && !wait_for(&bars.v_free[par], turn - 1, err)) break;
      tc_fence_after();
      const uint32_t col = lanes + S::kColV + 64u * par;
      uint32_t x[4];
      ldmatrix_x4_trans(src + raw_at<D>(lane, wq), x);
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {                 // 32 keys
        uint32_t next[4], lo[8], hi[8];
        ldmatrix_x4_trans(src + raw_at<D>((g + 1 & 3) * 32 + lane, wq), next);
        const uint4 f4 = *reinterpret_cast<const uint4 *>(&mine[(lane & 3) * 16 + 4 * g]);
        const uint32_t f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          wide8<Q>(x[m], f[m], offset2<Q>(f[m]), lo[2 * m], lo[2 * m + 1], hi[2 * m], hi[2 * m + 1]);
          x[m] = next[m];
        }
        tc_st_16x128b_x4(col + 16 * g, lo);
        tc_st_16x128b_x4(col + 16 * g + (16u << 16), hi);
      }
      __syncwarp();
      if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.empty[2 + par][st]));
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.v_ready[par]));
      if (++st == R) {
        st = 0;
        ++round;
      }
    }
  } else if (warp < kWarpS) {
    // ------------------------------------------------------------ producers ----
    // Of every second tile of K or V.  Lane i looks up keys 4 i .. of a tile (one block:
    // its size is a multiple of 8) and fetches their scales, an elected lane issues the
    // boxes.
    const int ring = warp - kWarpLoad, par = ring & 1;
    const bool is_v = ring >= 2;
    const uint32_t data0 = sv::smem_addr(raw) + ring * R * S::kData;
    const uint32_t scale0 = sv::smem_addr(scales) + ring * R * S::kScale + lane * 4 * S::kSRow;
    const CUtensorMap *map = is_v ? &p.vmap : &p.kmap;
    const uint8_t *from = is_v ? a.c.vs : a.c.ks;
    const int box = p.box, per = box / 4;           // keys of a box, lanes of it
    const int step_block = 2 * kT / a.c.bs, step_row = 2 * kT - step_block * a.c.bs;
    Tile w = tile_of(walk);
    int left = count_of(walk);                      // tiles of the range from w on
    const int32_t *table = nullptr;
    int block = 0, row = 0, id = 0;
    bool in = false;
    const auto step = [&] {
      if (--left > 0) next_tile(a, unit, walk, w);
    };
    const auto look = [&](bool fresh) {
      const int pos = w.t * kT + lane * 4;
      if (fresh) {
        table = a.c.tables + static_cast<size_t>(w.b) * a.c.max_blocks;
        block = pos / a.c.bs;
        row = pos - block * a.c.bs;
      }
      in = left > 0 && pos < w.kv_end;
      if (in) id = ld32(table + block);
    };
    if (par) step();
    look(true);
    int st = 0, round = 0, issued = 0;
#pragma unroll 1
    for (; left > 0; ++issued) {
      if (!is_v && lane == 0 && w.cut) report(a.bt.status, SV_KV_TABLE_SHORT);
      // A block that is not there marks the segment, whose unit is recomputed; any
      // block is loaded in its place.
      if (in && static_cast<uint32_t>(id) >= static_cast<uint32_t>(a.c.num_blocks)) {
        if (!is_v) {
          report(a.bt.status, id == -1 ? SV_KV_MISSING_BLOCK : SV_KV_BAD_BLOCK);
          seg_bad[w.seg % kSegRing] = w.seg + 1;
        }
        id = 0;
      }
      const int boxes = (__popc(__ballot_sync(kFull, in)) + per - 1) / per;
      if (round > 0 && !wait_for(&bars.empty[ring][st], round - 1, err)) {
        ok = false;
        break;
      }
      const uint32_t bar = sv::smem_addr(&bars.raw[ring][st]), dst = data0 + st * S::kData;
      if (in) {
        const uint8_t *src = from + id * a.c.sblock_bytes + (w.h * a.c.bs + row) * S::kSRow;
        const uint32_t to = scale0 + st * S::kScale;
        if constexpr (D == 128) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(src) : "memory");
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
      if (is_v && lane == 0) v_meta[par][st] = make_int4(w.kv_end - w.t * kT, w.new0 - w.t * kT, w.seg, 0);
      __syncwarp();
      if (elect_one()) sv::mbar_arrive_expect_tx(bar, boxes * box * S::kRow);   // no box: a table without blocks
      __syncwarp();
#pragma unroll 1
      for (int k = 0; k < boxes; k += 2) {          // two at a time: their look-ups overlap
        const int id0 = __shfl_sync(kFull, id, k * per), row0 = __shfl_sync(kFull, row, k * per);
        const int id1 = __shfl_sync(kFull, id, (k + 1) * per), row1 = __shfl_sync(kFull, row, (k + 1) * per);
        if (elect_one()) {
          tma_4d(dst + k * box * S::kRow, map, 0, row0, w.h, id0, bar);
          if (k + 1 < boxes) tma_4d(dst + (k + 1) * box * S::kRow, map, 0, row1, w.h, id1, bar);
        }
        __syncwarp();
      }
      const int seg = w.seg;
      step();
      step();
      block += step_block;
      row += step_row;
      if (row >= a.c.bs) {
        row -= a.c.bs;
        ++block;
      }
      look(w.seg != seg);
      if (++st == R) {
        st = 0;
        ++round;
      }
    }
    // Copies in flight land before the block ends (a stage not widened: the wait gives up).
    if (!ok)
#pragma unroll 1
      for (int k = max(0, issued - R); k < issued; ++k) wait_for(&bars.raw[ring][k % R], k / R, err);
  } else if (warp < kWarpQ) {
    // ------------------------------------------------------------- products ----
    // One warp for Q K^T, one for P V.  What a product needs is in uniform registers
    // (a reduction leaves it there).
    const bool is_o = warp == kWarpO;
    Tile w = tile_of(walk);
    const int n = __reduce_max_sync(kFull, count_of(walk));
    const uint32_t tm = __reduce_or_sync(kFull, tmem);
    // A tile's N (the unit's rows, padded), in its place of the descriptor, and below it
    // whether it is a segment's first (1) or last (2), and the segment's parity (4).
    uint32_t width = 0;
    const auto look = [&] {
      if (w.first()) {
        const int rows = min(walk.r.n * a.G - w.mp * p.unit_rows, p.unit_rows);
        width = static_cast<uint32_t>(rows + kUnit - 1) / kUnit * (kUnit / 8) << 17;
      }
      return __reduce_or_sync(kFull, width | (w.first() ? 1u : 0u) | (w.last() ? 2u : 0u) | (w.seg & 1) << 2);
    };
    constexpr uint32_t kN = 63u << 17;
    const uint64_t desc = smem_desc(sv::smem_addr(is_o ? sp : sq), 16);
    const uint32_t kind = is_o ? mma_desc<Q>(0, true) : mma_desc<Q>(0, false) | (p.negate ? kNegateA : 0u);
    uint32_t now = 0, place = 0;
    if (n > 0) now = look();
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const uint32_t buf = i & 1, round = i >> 1, id = kind | (now & kN);
      if (is_o) {
        if (!(ok = wait_for(&bars.v_ready[buf], round, err) && wait_for(&bars.p_ready[i & 3], i >> 2, err))) break;
        tc_fence_after();
        const uint32_t d = tm + S::kColO, va = tm + S::kColV + 64u * buf, more = ~now & 1u;
        const uint64_t pd = desc + (place * S::kPBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kT / 16; ++k) tc_mma_ts(d, va + 8u * k, pd + k * (2048 >> 4), id, k > 0 ? 1u : more);
          tc_commit(sv::smem_addr(&bars.o_done[i & 3]));
          tc_commit(sv::smem_addr(&bars.v_free[buf]));
        }
        if (++place == kPlaces) place = 0;
      } else {
        // The keys, the queries, S's place, free when the second tile before is P, and P's,
        // free when the third tile's products are done.
        if (!(ok = (!(now & 1u) || wait_for(&bars.q_full[now >> 2 & 1u], w.seg >> 1, err)) &&
                   wait_for(&bars.k_ready[buf], round, err) && (i < 2 || wait_for(&bars.p_ready[i - 2 & 3], (i - 2) >> 2, err)) &&
                   (i < 3 || wait_for(&bars.o_done[i - 3 & 3], (i - 3) >> 2, err))))
          break;
        tc_fence_after();
        const uint32_t d = tm + S::kColS + 64u * buf, ka = tm + S::kColK + 64u * buf;
        const uint64_t qd = desc + (now & 4u ? S::kQBytes >> 4 : 0);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc_mma_ts(d, ka + 8u * k, qd + (((k >> 2) * S::kQHalf + (k & 3) * 32) >> 4), id, k > 0);
          tc_commit(sv::smem_addr(&bars.s_full[buf]));
          tc_commit(sv::smem_addr(&bars.k_free[buf]));
          if (now & 2u) tc_commit(sv::smem_addr(&bars.q_empty[now >> 2 & 1u]));
        }
      }
      __syncwarp();
      if (i + 1 < n) {
        next_tile(a, unit, walk, w);
        now = look();
      }
    }
    if (!ok) {  // issued products end before TMEM is freed
      if (elect_one()) tc_commit(sv::smem_addr(&bars.drain[is_o]));
      __syncwarp();
      wait_for(&bars.drain[is_o], 0, err);
    }
  } else if (warp == kWarpQ) {
    // -------------------------------------------------------------- queries ----
    // A segment's rows, a segment ahead, each eight elements in the order of the
    // widened keys.
#pragma unroll 1
    for (; walk.on; next_segment(a, unit, walk)) {
      const int seg = walk.seg, qb = seg & 1, row0 = walk.mp * p.unit_rows, rows = rows_of(walk);
      if (seg >= 2 && !wait_for(&bars.q_empty[qb], (seg >> 1) - 1, err)) break;
      uint8_t *const dst = sq + qb * S::kQBytes;
      const int chunks = (rows + kUnit - 1) / kUnit * kUnit * (D / 8);
      const uint8_t *base = a.q + walk.b * a.qsb;
#pragma unroll 8
      for (int i = lane; i < chunks; i += 32) {
        const int row = i / (D / 8), ch = i % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < rows) {
          const int t = (row0 + row) / a.G, g = row0 + row - t * a.G;
          v = ld128(base + t * a.qst + (walk.h * a.G + g) * a.qsh + ch * 16);
        }
        const uint4 o = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                   __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
        *reinterpret_cast<uint4 *>(dst + (ch >> 3) * S::kQHalf + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) = o;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.q_full[qb]));
    }
  }

  tc_fence_before();
  const bool some = __syncthreads_or(marked);
  tc_fence_after();
  if (warp == kWarpS) tc_dealloc(tmem, 512);
  if (some) recompute_marked<Q, I4, D>(a, unit, sh_walk, marks, warp, kThreads / 32);
}

}  // namespace i4
}  // namespace svp
