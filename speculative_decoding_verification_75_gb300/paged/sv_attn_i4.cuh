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
// 24 N, 384 for that chain and 128 for a token.
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
// Softmax.  A thread has one key and half of the rows: two groups of four warps.  The
// rows' references m are shared by the 128 keys and live in shared memory; P is
// 2^(x - m), and only when a score exceeds its reference by more than 2^8 (a vote of
// the group, once a tile) are the references raised and O^T's columns rescaled; that
// path also does the first tile of a unit and the tiles that hold new tokens, with
// their masks.  A thread's parts of the rows' sums are columns of tensor memory, not
// registers: then every loop over rows has one copy of its body.  (Unrolled, the
// code of all roles together missed the instruction cache: 642 us for 128 requests.)
//
// Work, ranges, cut units, marked units and the second kernel are those of
// sv_attn_tc.cuh, with one range for a thread block.
#pragma once

#include "sv_attn_tc.cuh"

namespace svp {
namespace i4 {

constexpr int kT = 128;          // keys of a tile
constexpr int kRows = 64;        // query rows of a unit, at most
constexpr int kUnit = 16;        // N is a multiple of it
constexpr int kChunk = 8;        // rows in registers at once
constexpr int kThreads = 640;
// Warps: 0 - 7 softmax, 8 - 11 widen K, 12 - 15 V, then K's and V's producer, the
// products, the queries.
constexpr int kWarpK = 8, kWarpV = 12, kWarpLoadK = 16, kWarpLoadV = 17, kWarpMma = 18, kWarpQ = 19;

template <int D>
struct Shape {
  static constexpr int kRow = D / 2, kSRow = D / SV_KV_GROUP;     // bytes of a key's codes and scales
  static constexpr int kData = kT * kRow, kScale = kT * kSRow;
  static constexpr int kStages = D == 128 ? 8 : 16;               // of K, and of V
  static constexpr int kQHalf = kRows * 128;                      // 64 columns of the queries
  static constexpr int kQBytes = D / 64 * kQHalf, kPBytes = kT * 128;
  static constexpr int kSmem = 2 * kQBytes + 2 * kPBytes + 2 * kStages * (kData + kScale);
  static constexpr int kGroups = D / SV_KV_GROUP;                 // warps that widen V
  // TMEM columns: two of K, V and S, O and the sums.
  static constexpr uint32_t kColK = 0, kColV = 128, kColS = 256, kColO = 384, kColL = 448;
};

template <int N>
struct BarSet {
  uint64_t k_raw[N], v_raw[N], k_empty[N], v_empty[N];
  uint64_t k_ready[2], k_free[2], v_ready[2], v_free[2], s_full[2], p_ready[2], o_done[2], q_full[2], q_empty[2], drain;
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
// A scale byte twice: f, or f / 16 in fp16 (a subnormal number holds it too).
template <typename Q>
__device__ __forceinline__ uint32_t scale2(uint32_t s) {
  if constexpr (Q::kIsBf16) {
    return s > SV_KV_I4_MAX_SCALE ? 0x7fff7fffu : s * 0x00100010u + 0x38803880u;   // exponent + 113
  } else {
    return mul2<F16>(s > SV_KV_I4_MAX_SCALE ? 0x7fff7fffu : s * 0x00800080u + 0x04000400u, 0x2c002c00u);
  }
}
// What takes (16 + c) f (bf16) or (64 + c) f (fp16) to (c - 8) f.
template <typename Q>
__device__ __forceinline__ uint32_t offset2(uint32_t f) {
  return mul2<Q>(f, Q::kIsBf16 ? 0xc1c0c1c0u : 0xd480d480u);                       // -24, -72
}
// Codes i and i + 4 of a word's eight, i = 0 .. 3, times their scales f (two,
// for the codes' places).  A multiplication by 8 or 16 is a shift on the other pipe
// than the masks'.
template <typename Q>
__device__ __forceinline__ void wide8(uint32_t w, uint32_t f, uint32_t off, uint32_t &o0, uint32_t &o1, uint32_t &o2,
                                      uint32_t &o3) {
  const uint32_t x = __byte_perm(w, 0, 0x2301);   // codes 2, 3 (6, 7) in the places of 0, 1
  if constexpr (Q::kIsBf16) {
    constexpr uint32_t m = 0x00780078u, b = 0x41804180u;
    const uint32_t w1 = w >> 1, x1 = __byte_perm(w1, 0, 0x2301);
    o0 = fma2<Q>((w * 8u & m) | b, f, off);
    o1 = fma2<Q>((w1 & m) | b, f, off);
    o2 = fma2<Q>((x * 8u & m) | b, f, off);
    o3 = fma2<Q>((x1 & m) | b, f, off);
  } else {
    constexpr uint32_t m = 0x00f000f0u, b = 0x54005400u;
    o0 = fma2<Q>((w * 16u & m) | b, f, off);
    o1 = fma2<Q>((w & m) | b, f, off);
    o2 = fma2<Q>((x * 16u & m) | b, f, off);
    o3 = fma2<Q>((x & m) | b, f, off);
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
  __shared__ alignas(16) uint32_t v_scale[4][kT / 2];  // a V warp's scales: pair m of keys 8 m + 2 j at 16 j + m

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t *const sq = smem, *const sp = sq + 2 * S::kQBytes, *const raw = sp + 2 * S::kPBytes;
  uint8_t *const scales = raw + 2 * R * S::kData;   // stages of K, then of V, like the data
  const AttnParams &a = p.a;

  if (sv::smem_addr(smem) & 1023u) {                // never: the swizzle would not match
    report(p.err, SV_FAULT_TIMEOUT);
    return;
  }
  if (warp == kWarpMma) tc_alloc(sv::smem_addr(&tmem_slot), 512);
  if (tid == 0) {
    for (int i = 0; i < R; ++i) {
      sv::mbar_init(sv::smem_addr(&bars.k_raw[i]), 33);       // 32 lanes' scales, the data
      sv::mbar_init(sv::smem_addr(&bars.v_raw[i]), 33);
      sv::mbar_init(sv::smem_addr(&bars.k_empty[i]), 4);
      sv::mbar_init(sv::smem_addr(&bars.v_empty[i]), S::kGroups);
    }
    for (int i = 0; i < 2; ++i) {
      sv::mbar_init(sv::smem_addr(&bars.k_ready[i]), 4);
      sv::mbar_init(sv::smem_addr(&bars.k_free[i]), 1);
      sv::mbar_init(sv::smem_addr(&bars.v_ready[i]), S::kGroups);
      sv::mbar_init(sv::smem_addr(&bars.v_free[i]), 1);
      sv::mbar_init(sv::smem_addr(&bars.s_full[i]), 1);
      sv::mbar_init(sv::smem_addr(&bars.p_ready[i]), 8);
      sv::mbar_init(sv::smem_addr(&bars.o_done[i]), 1);
      sv::mbar_init(sv::smem_addr(&bars.q_full[i]), 1);
      sv::mbar_init(sv::smem_addr(&bars.q_empty[i]), 1);
    }
    sv::mbar_init(sv::smem_addr(&bars.drain), 1);
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
  if (warp == kWarpLoadK) {
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
#pragma unroll 1
    while (walk.on) {
      const Walk sg = walk;
      const Req &r = sg.r;
      const int nt = sg.t1 - sg.t0, seg = sg.seg;
      const int row0 = sg.mp * p.unit_rows, rows = rows_of(sg);
      // The group's rows [g0, g1) of the unit; none of them may be real.
      const int half = (rows + kUnit - 1) / kUnit * (kUnit / 2), g0 = grp * half;
      const int g1 = g0 < rows ? g0 + half : g0;
      const int full_end = sg.new0();               // every row sees these
      const uint32_t col_o = lanes + S::kColO, col_l = lanes + S::kColL;
#pragma unroll 1
      for (int j = 0; j < nt; ++j, ++tiles) {
        const uint32_t buf = tiles & 1, round = tiles >> 1;
        const uint32_t col_s = lanes + S::kColS + 64u * buf;
        const int k0 = (sg.t0 + j) * kT;
        const bool masked = k0 + kT > full_end, fast = j > 0 && !masked;
        uint8_t *const prow = sp + buf * S::kPBytes + my * 128;
        const auto put = [&](int row, const uint32_t (&pk)[kChunk / 2]) {
          *reinterpret_cast<uint4 *>(prow + ((row / kChunk ^ (my & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        };
        bool good = wait_warp(&bars.s_full[buf], round, err);
        if (good && tiles >= 2) good = wait_warp(&bars.o_done[buf], round - 1, err);
        __syncwarp();
        tc_fence_after();
        float top = -INFINITY;
        if (fast && good) {
#pragma unroll 1
          for (int row = g0; row < g1; row += kChunk) {
            uint32_t x[kChunk], l[kChunk];
            tc_ld8(col_s + row, x);
            tc_ld8(col_l + row, l);
            const ulonglong2 n0 = *reinterpret_cast<const ulonglong2 *>(&refs.minus[row]);
            const ulonglong2 n1 = *reinterpret_cast<const ulonglong2 *>(&refs.minus[row + 4]);
            const uint64_t nm[4] = {n0.x, n0.y, n1.x, n1.y};
            tc_wait_ld(x);
            tc_wait_ld(l);
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
          // Which rows see the thread's key.
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
          const auto hide = [&](int row, uint32_t (&x)[kChunk]) {
            const uint32_t bits = static_cast<uint32_t>(vis >> row);
#pragma unroll
            for (int k = 0; k < kChunk; ++k)
              if (!(bits >> k & 1u)) x[k] = 0xff800000u;
          };
          if (good) {
#pragma unroll 1
            for (int row = g0; row < g1; row += kChunk) {
              uint32_t x[kChunk];
              tc_ld8(col_s + row, x);
              if (fast) {
                // The sums without what was just added; where that exceeds 2^100, what was
                // there before is nothing against what the raised reference brings.
                uint32_t l[kChunk];
                tc_ld8(col_l + row, l);
                tc_wait_ld(x);
                tc_wait_ld(l);
#pragma unroll
                for (int k = 0; k < kChunk; ++k) {
                  const float e = sv::ex2(fmaf(__uint_as_float(x[k]), c, refs.minus[row + k]));
                  l[k] = e >= 0x1p100f ? 0u : __float_as_uint(__uint_as_float(l[k]) - e);
                }
                tc_st8(col_l + row, l);
              } else {
                tc_wait_ld(x);
              }
              hide(row, x);
              float best = -INFINITY;
#pragma unroll
              for (int k = 0; k < kChunk; ++k) {
                const float t = warp_top(__uint_as_float(x[k]) * c);
                if (lane == k) best = t;
              }
              if (lane < kChunk) refs.top[wq][row + lane] = best;
            }
            // The products of the tile before may still run.
            if (j > 0 && !wait_warp(&bars.o_done[buf ^ 1], (tiles - 1) >> 1, err)) refs.dead[grp] = 1;
          }
          tc_wait_st();
          group_sync(grp);
          if (*const_cast<volatile int *>(&refs.dead[grp])) {
            ok = false;
            break;
          }
          const int row = g0 + my;
          if (row < g1) {
            const float mt = fmaxf(fmaxf(refs.top[0][row], refs.top[1][row]), fmaxf(refs.top[2][row], refs.top[3][row]));
            float m = j > 0 ? refs.m[row] : -INFINITY, f = 1.f;
            if (mt - kHead > m && !(mt - m <= kUp)) {
              f = sv::ex2(m - (mt - kHead));
              m = mt - kHead;
            }
            refs.m[row] = m;
            refs.minus[row] = m == -INFINITY ? 3.402823466e38f : -m;
            refs.factor[row] = f;
          }
          group_sync(grp);
          tc_fence_after();
#pragma unroll 1
          for (int row = g0; row < g1; row += kChunk) {
            uint32_t x[kChunk], l[kChunk], pk[kChunk / 2];
            if (j > 0) {
              uint32_t o[kChunk];
              tc_ld8(col_o + row, o);
              tc_ld8(col_l + row, l);
              tc_wait_ld(o);
              tc_wait_ld(l);
#pragma unroll
              for (int k = 0; k < kChunk; ++k) {
                const float f = refs.factor[row + k];
                o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                l[k] = __float_as_uint(__uint_as_float(l[k]) * f);
              }
              tc_st8(col_o + row, o);
            } else {
#pragma unroll
              for (int k = 0; k < kChunk; ++k) l[k] = 0;
            }
            tc_ld8(col_s + row, x);
            tc_wait_ld(x);
            hide(row, x);
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
        if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.p_ready[buf]));
      }
      if (!ok) break;
      next_segment(a, unit, walk);

      // The warp's part of the rows' sums: a butterfly whose halves keep half of the rows each.
#pragma unroll 1
      for (int row = g0; row < g1; row += kChunk) {
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
      if (!wait_warp(&bars.o_done[last & 1], last >> 1, err)) refs.dead[grp] = 1;
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
      const int end = min(g1, rows);                // of the group's real rows
      if (g0 + my < end) {
        const int row = g0 + my;
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
      if (!bad && wq < S::kGroups) {
#pragma unroll 1
        for (int row = g0; row < end; row += kChunk) {
          uint32_t o[kChunk];
          tc_ld8(col_o + row, o);
          tc_wait_ld(o);
#pragma unroll
          for (int k = 0; k < kChunk; ++k) {
            if (row + k < end) {
              const float f = refs.factor[row + k];
              const float y = f == 0.f ? 0.f : __uint_as_float(o[k]) * f;   // not 0 * O: it may be NaN
              if (whole) store1<Q>(a.out + (out_row(row + k) * D + dim) * 2, y);
              else slot[(static_cast<size_t>(dim >> 2) * p.slot_rows + row + k) * 4 + (dim & 3)] = y;
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
    const int n = count_of(walk);
    int st = 0, round = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const uint32_t buf = i & 1;
      if (!wait_warp(&bars.k_raw[st], round, err)) break;
      const uint8_t *src = raw + st * S::kData, *sc = scales + st * S::kScale + my * S::kSRow;
      uint4 w = *reinterpret_cast<const uint4 *>(src + raw_at<D>(my, 0));
      uint32_t f4 = D == 128 ? *reinterpret_cast<const uint32_t *>(sc) : *reinterpret_cast<const uint16_t *>(sc);
      if (i >= 2 && !wait_warp(&bars.k_free[buf], (i >> 1) - 1, err)) break;
      tc_fence_after();
      const uint32_t col = lanes + S::kColK + 64u * buf;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        const uint4 next = *reinterpret_cast<const uint4 *>(src + raw_at<D>(my, ch + 1 & (D / 32 - 1)));
        const uint32_t f = scale2<Q>(f4 & 255u), off = offset2<Q>(f);
        f4 >>= 8;
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) wide8<Q>(u[k], f, off, o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        tc_st16(col + 16 * ch, o);
        w = next;
      }
      __syncwarp();
      if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.k_empty[st]));
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.k_ready[buf]));
      if (++st == R) {
        st = 0;
        ++round;
      }
    }
  } else if (warp < kWarpV + S::kGroups) {
    // ----------------------------------------------------------- V wideners ----
    Tile w = tile_of(walk);
    const int n = count_of(walk);
    int st = 0, round = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const uint32_t buf = i & 1;
      if (!wait_warp(&bars.v_raw[st], round, err)) break;
      const uint32_t src = sv::smem_addr(raw + (R + st) * S::kData);
      const uint8_t *sc = scales + (R + st) * S::kScale + wq;
      // This lane's keys lane, lane + 32, ..: their scales, 0 behind the last token.
      const int k0 = w.t * kT, live = w.kv_end - k0, fresh = w.new0 - k0;
      bool found = false;
      uint16_t *const mine = reinterpret_cast<uint16_t *>(v_scale[wq]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = lane + 32 * k;
        const uint32_t s = sc[key * S::kSRow];
        found = found || (key >= fresh && key < live && s > SV_KV_I4_MAX_SCALE);
        mine[((key >> 1 & 3) * 16 + (key >> 3)) * 2 + (key & 1)] =
            static_cast<uint16_t>(key < live ? scale2<Q>(s) : 0u);
      }
      // NaN among the new tokens: a row that does not see it must not meet it.
      if (found) seg_bad[w.seg % kSegRing] = w.seg + 1;
      __syncwarp();
      if (i >= 2 && !wait_warp(&bars.v_free[buf], (i >> 1) - 1, err)) break;
      tc_fence_after();
      const uint32_t col = lanes + S::kColV + 64u * buf;
      uint32_t x[4];
      ldmatrix_x4_trans(src + raw_at<D>(lane, wq), x);
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {                 // 32 keys
        uint32_t next[4], lo[8], hi[8];
        ldmatrix_x4_trans(src + raw_at<D>((g + 1 & 3) * 32 + lane, wq), next);
        const uint4 f4 = *reinterpret_cast<const uint4 *>(&v_scale[wq][(lane & 3) * 16 + 4 * g]);
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
      if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.v_empty[st]));
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.v_ready[buf]));
      next_tile(a, unit, walk, w);
      if (++st == R) {
        st = 0;
        ++round;
      }
    }
  } else if (warp == kWarpLoadK || warp == kWarpLoadV) {
    // ------------------------------------------------------------ producers ----
    // One warp for K, one for V.  Lane i looks up keys 4 i .. of a tile (one block:
    // its size is a multiple of 8) and fetches their scales, an elected lane
    // issues the boxes.
    const bool is_v = warp == kWarpLoadV;
    uint64_t *const fullb = is_v ? bars.v_raw : bars.k_raw, *const emptyb = is_v ? bars.v_empty : bars.k_empty;
    const uint32_t data0 = sv::smem_addr(raw) + (is_v ? R * S::kData : 0);
    const uint32_t scale0 = sv::smem_addr(scales) + (is_v ? R * S::kScale : 0) + lane * 4 * S::kSRow;
    const CUtensorMap *map = is_v ? &p.vmap : &p.kmap;
    const uint8_t *from = is_v ? a.c.vs : a.c.ks;
    const int box = p.box, per = box / 4;           // keys of a box, lanes of it
    const int step_block = kT / a.c.bs, step_row = kT - step_block * a.c.bs;
    Tile w = tile_of(walk);
    const int n = count_of(walk);
    const int32_t *table = nullptr;
    int block = 0, row = 0, id = 0;
    bool in = false;
    const auto fetch = [&] {
      const int pos = w.t * kT + lane * 4;
      if (w.first()) {
        table = a.c.tables + static_cast<size_t>(w.b) * a.c.max_blocks;
        block = pos / a.c.bs;
        row = pos - block * a.c.bs;
      } else {
        block += step_block;
        row += step_row;
        if (row >= a.c.bs) {
          row -= a.c.bs;
          ++block;
        }
      }
      in = w.on && pos < w.kv_end;
      id = in ? ld32(table + block) : 0;
    };
    fetch();
    int st = 0, round = 0, issued = -1;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      if (!is_v && lane == 0 && w.first() && w.cut) report(a.bt.status, SV_KV_TABLE_SHORT);
      // A block that is not there marks the segment, whose unit is recomputed; any
      // block is loaded in its place.
      if (in && static_cast<uint32_t>(id) >= static_cast<uint32_t>(a.c.num_blocks)) {
        if (!is_v) {
          report(a.bt.status, id == -1 ? SV_KV_MISSING_BLOCK : SV_KV_BAD_BLOCK);
          seg_bad[w.seg % kSegRing] = w.seg + 1;
        }
        id = 0;
      }
      const int h = w.h, now = id, at_row = row, boxes = (__popc(__ballot_sync(kFull, in)) + per - 1) / per;
      const bool put = in;
      next_tile(a, unit, walk, w);
      fetch();                                      // on its way while the stage is waited for
      if (round > 0 && !wait_warp(&emptyb[st], round - 1, err)) {
        ok = false;
        break;
      }
      const uint32_t bar = sv::smem_addr(fullb) + 8u * st;
      if (put) {
        const uint8_t *src = from + static_cast<int64_t>(now) * a.c.sblock_bytes +
                             (static_cast<int64_t>(h) * a.c.bs + at_row) * S::kSRow;
        const uint32_t dst = scale0 + st * S::kScale;
        if constexpr (D == 128) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
      const uint32_t dst = data0 + st * S::kData;
      if (elect_one()) sv::mbar_arrive_expect_tx(bar, boxes * box * S::kRow);   // no box: a table without blocks
      __syncwarp();
#pragma unroll 1
      for (int k = 0; k < boxes; ++k) {
        const int b_id = __shfl_sync(kFull, now, k * per), b_row = __shfl_sync(kFull, at_row, k * per);
        if (elect_one()) tma_4d(dst + k * box * S::kRow, map, 0, b_row, h, b_id, bar);
        __syncwarp();
      }
      issued = i;
      if (++st == R) {
        st = 0;
        ++round;
      }
    }
    // Copies in flight land before the block ends (a stage not widened: the wait gives up).
    if (!ok)
#pragma unroll 1
      for (int k = max(0, issued - R + 1); k <= issued; ++k) wait_warp(&fullb[k % R], k / R, err);
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------- products ----
    Tile w = tile_of(walk), behind = w;
    const int n = count_of(walk);
    const uint64_t q_desc = smem_desc(sv::smem_addr(sq), 16), p_desc = smem_desc(sv::smem_addr(sp), 16);
    const uint32_t kQK = mma_desc<Q>(0, false) | (p.negate ? kNegateA : 0u);
    constexpr uint32_t kPV = mma_desc<Q>(0, true);
    const auto width = [&](const Tile &x, int total) {   // of the products: the unit's rows, padded
      return static_cast<uint32_t>(min(total - x.mp * p.unit_rows, p.unit_rows) + kUnit - 1) / kUnit * (kUnit / 8) << 17;
    };
    int tokens = walk.r.n, tokens_behind = tokens;
#pragma unroll 1
    for (int i = 0; ok && i <= n && n > 0; ++i) {
      if (i < n) {
        const uint32_t buf = i & 1, qb = w.seg & 1;
        ok = (!w.first() || wait_warp(&bars.q_full[qb], w.seg >> 1, err)) && wait_warp(&bars.k_ready[buf], i >> 1, err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + S::kColS + 64u * buf, ka = tmem + S::kColK + 64u * buf;
        const uint64_t qd = q_desc + (qb * S::kQBytes >> 4);
        const uint32_t id = kQK | width(w, tokens * a.G);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc_mma_ts(d, ka + 8u * k, qd + (((k >> 2) * S::kQHalf + (k & 3) * 32) >> 4), id, k > 0);
          tc_commit(sv::smem_addr(&bars.k_free[buf]));
          tc_commit(sv::smem_addr(&bars.s_full[buf]));
          if (w.last()) tc_commit(sv::smem_addr(&bars.q_empty[qb]));
        }
        __syncwarp();
      }
      if (i > 0) {
        const uint32_t t = i - 1, buf = t & 1;
        ok = wait_warp(&bars.v_ready[buf], t >> 1, err) && wait_warp(&bars.p_ready[buf], t >> 1, err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + S::kColO, va = tmem + S::kColV + 64u * buf;
        const uint64_t pd = p_desc + (buf * S::kPBytes >> 4);
        const uint32_t id = kPV | width(behind, tokens_behind * a.G), first = behind.first();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kT / 16; ++k) tc_mma_ts(d, va + 8u * k, pd + k * (2048 >> 4), id, !(first && k == 0));
          tc_commit(sv::smem_addr(&bars.v_free[buf]));
          tc_commit(sv::smem_addr(&bars.o_done[buf]));
        }
        __syncwarp();
      }
      behind = w;
      tokens_behind = tokens;
      if (i < n) {
        next_tile(a, unit, walk, w);
        tokens = walk.r.n;
      }
    }
    if (!ok) {  // issued products end before TMEM is freed
      if (elect_one()) tc_commit(sv::smem_addr(&bars.drain));
      __syncwarp();
      wait_warp(&bars.drain, 0, err);
    }
  } else if (warp == kWarpQ) {
    // -------------------------------------------------------------- queries ----
    // A segment's rows, a segment ahead, each eight elements in the order of the
    // widened keys.
#pragma unroll 1
    for (; walk.on; next_segment(a, unit, walk)) {
      const int seg = walk.seg, qb = seg & 1, row0 = walk.mp * p.unit_rows, rows = rows_of(walk);
      if (seg >= 2 && !wait_warp(&bars.q_empty[qb], (seg >> 1) - 1, err)) break;
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
  if (warp == kWarpMma) tc_dealloc(tmem, 512);
  if (some) recompute_marked<Q, I4, D>(a, unit, sh_walk, marks, warp, kThreads / 32);
}

}  // namespace i4
}  // namespace svp
