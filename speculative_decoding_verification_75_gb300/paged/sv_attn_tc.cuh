// sv_attn_tc.cuh -- tree attention over the paged cache on the tensor cores
// (tcgen05), for head dimensions 64 and 128.
//
// Rows.  All n new tokens and the G query heads that share a KV head form one
// matrix of n * G rows, row r = token r / G, head r % G, so that a key is read
// once for all of them; a tile takes as many whole tokens as fit 128 rows.
// S = Q K^T and O = P V run as M = 128 row tiles with 64 keys a step; S and O
// live in tensor memory (TMEM: lane = row, one thread per row), P overwrites
// half of its S as the 16-bit A operand.
//
// Two streams of such steps alternate in a thread block, each with a softmax
// warpgroup of its own and two S, so that the tensor cores work on one stream
// while the other takes exponentials, and on the next scores of a stream while
// it works on these.  With at most 128 rows the streams are independent, each
// with a range of work of its own (kPair = false): one goes on while the other
// stores its rows and begins the next unit.  With more rows each has 128 of
// the unit's and both use every key tile (kPair = true).
//
// Work.  The key tiles of all units (request, KV head, row tiles) form one
// sequence that is cut into equal ranges, one per stream or pair of streams of
// one block per SM: ragged lengths are balanced to within a tile.  A unit cut
// by a range's end leaves partial results (unnormalised O, row maximum and
// sum) in the workspace, joined by the second kernel in range order, so
// results do not depend on timing.  The lengths are read on the device; the
// host never waits.
//
// Softmax.  One pass: a row keeps a reference m and sums 2^(x - m) in fp32.
// O is rescaled only when a tile's maximum exceeds the one that set m by more
// than 2^8 (bf16 and fp16 hold 2^8 as exactly as 1, fp32 sums lose nothing),
// which after the first tiles is rare.  fp16 probabilities begin at 2^7, so that
// small ones keep their bits: what is lost is 2^-32 of the largest, at most.
//
// Data.  TMA boxes of one page's rows (a power of two of them that divides the
// block size) fill 128-byte swizzled tiles through an mbarrier ring; e4m3 tiles
// arrive raw with their scale bytes and are widened to fp16 by eight warps.
// Rows of V behind the last token are zeroed in shared memory, because
// 0 * garbage may be NaN; a value that is not finite among the new tokens, or a
// missing block, marks the unit, which is recomputed row by row
// (sv_attn_general.cuh): by the second kernel if it is cut, else when the
// block's ranges are done.
//
// Measured, both kernels together:
//   131071 keys, 1 token, 64 heads on 8 of 128   92 us, 5.8 TB/s: HBM; 8 us are
//                                                the join and the first tiles
//   32 x 9 tokens, 32 heads on 32, 200-2000 keys 114 us, 5.1 TB/s: HBM, and the
//                                                ends of units of few tiles
//   8 x 6 tokens, 64 on 8, 1000-4000 keys        29 us, 2.9 TB/s: start, first
//                                                data and join, 15 us together
//   16 trees of 64, 32 on 8, 1000-8000 keys      102 us, 547 TFLOP/s: unit ends,
//                                                join; a step takes twice its
//                                                products' time, with 64 keys a
//                                                step and with 128
//   128 x 6 tokens, e4m3, 500-8000 keys          363 us, 3.2 TB/s: instructions
//                                                of the wideners and the softmax
// The kernel's code is fetched by five roles at once: with the loops unrolled
// further they missed the instruction cache (90 % hits, 423 us for the last case
// against 379 at 96 %), so each role's loop has one copy of its body.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "sv_attn_general.cuh"

namespace svp {

constexpr int kMaxGrid = 152;   // thread blocks, one per SM
constexpr int kTile = 128;      // rows of a tile
// Keys of a step, and of a stage.  A stream has two S of 64 keys, so that Q K^T
// is a step ahead of the softmax.  (With one S of 128 keys Q K^T, softmax and P V
// were a chain: 413 us for 128 e4m3 requests, 393 with two.  Pairs of row tiles,
// bound by the tensor cores, take the same time with either.)
constexpr int kKeys = 64, kBufs = 2;
constexpr int kScaleRing = 16;  // K tiles that are widened and not yet used, at most 7
constexpr int kSegRing = 32;    // more segments than any role is ahead of another
constexpr int kMarkBits = 1024; // of a range's marked segments, by number modulo this

// The first segment of a range: its unit, the tile of the unit it begins at,
// and the unit's tiles; `total` tiles of all ranges.
struct alignas(16) Cut {
  int b, h, mp, n, t0, kt, total, pad;
};

struct TcParams {
  CUtensorMap kmap, vmap, qmap;
  AttnParams a;
  uint32_t *err;       // SV_FAULT_TIMEOUT goes here
  Cut *cuts;           // [ranges] where each range begins
  float *slots;        // [ranges * 2] partial results
  int ranges, grid;    // of the tiles; thread blocks at most
  int slot_rows;       // rows of a slot
  int slot_floats;
  int box;             // rows of a TMA box of the cache
  int TT;              // tokens of a row tile: its rows are TT * G <= 128
  int qbox;            // tokens of a TMA box of the queries
  int mvec;            // mask rows are whole 4-byte words
  float c;             // |scale| * log2(e), not 0
  int negate;          // scale < 0: S is computed with Q's signs flipped
};

// ------------------------------------------------------------- tcgen05 ----

__device__ __forceinline__ void tc_alloc(uint32_t smem_dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_dealloc(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// One lane of a converged warp, the same one each time.  (Selected this way the
// descriptors stay in uniform registers; under `lane == 0` every product took
// ~120 cycles to issue, twice its execution time.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred P; elect.sync _|P, 0xffffffff; selp.u32 %0, 1, 0, P; }" : "=r"(p));
  return p != 0;
}
// Completion of every tcgen05.mma this thread has issued, on an mbarrier.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

#define SVP_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), \
                     "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define SVP_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), \
                     "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of this warp's 32 lanes: one lane per thread.
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : SVP_R8(r, 0), SVP_R8(r, 8), SVP_R8(r, 16), SVP_R8(r, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      SVP_W8(r, 0), SVP_W8(r, 8), SVP_W8(r, 16), SVP_W8(r, 24)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      SVP_W8(r, 0), SVP_W8(r, 8)
      : "memory");
}
// The loaded registers are tied to the wait, so that no use moves before it.
template <int N>
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Shared-memory operand descriptor: 128-byte swizzle, 8-row groups 1024 bytes
// apart; `lead`: distance of the next 64 elements along the contiguous
// dimension where the operand is not K-major.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

// Instruction descriptor: fp32 accumulators, M = 128; b_mn: B's N runs
// contiguously.  kNegateA: A's signs are flipped.
constexpr uint32_t kNegateA = 1u << 13;
template <typename Q>
__device__ constexpr uint32_t mma_desc(int n, bool b_mn) {
  const uint32_t fmt = sizeof(Q) && Q::kBytes == 2 && Q::kIsBf16 ? 1u : 0u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                       int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void bulk_1d(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Two fp32 at once.
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <typename Q>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (Q::kIsBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}

// Whether one of the two 16-bit values is an infinity or NaN.
template <typename Q>
__device__ __forceinline__ bool odd16(uint32_t u) {
  constexpr uint32_t e = Q::kIsBf16 ? 0x7f80u : 0x7c00u;
  return (u & e) == e || ((u >> 16) & e) == e;
}

// ---------------------------------------------------------------- shape ----

template <typename Q, typename C, int D, bool kPair>
struct Shape {
  static constexpr bool kRaw = C::kBytes == 1;      // e4m3: widened on chip
  using M = typename std::conditional<kRaw, F16, Q>::type;   // what the tensor cores multiply
  static constexpr int kHalves = D / 64;
  static constexpr int kStreams = kPair ? 1 : 2;    // ranges of a block
  static constexpr int kQTile = kTile * D * 2;
  static constexpr int kQBytes = 2 * kQTile;        // a Q tile per stream
  // Each range has a ring of its own, with one order of loads: a parity tells
  // two phases of a barrier apart only if no one is a whole round ahead.
  static constexpr int kStageBytes = kKeys * D * 2;
  static constexpr int kHalf = kKeys * 128;                 // bytes of a stage's 64 columns
  static constexpr int kRawData = kKeys * D, kRawScale = kKeys * (D / SV_KV_GROUP);
  static constexpr int kRawBytes = kRawData + kRawScale;
  // Stages of a ring: as many as 227 KB hold (about 200 KB where tiles are
  // small); raw stages first, they are what is in flight.
  static constexpr int kStages = (kRaw ? 3 : D == 128 ? 5 : 11) * (kPair ? 2 : 1);
  static constexpr int kRawStages = kRaw ? (D == 128 ? 3 : 10) * (kPair ? 2 : 1) : 0;
  static constexpr int kChunk = kRaw ? 32 : 64;     // S columns in registers at once
  static constexpr int kTilesPerUnit = kPair ? 2 : 1;
  // Warps: 8 softmax, 2 producers, 2 for the products, and 8 that widen: 3 or 5
  // on each scheduler (4 wideners were bound by their latencies).
  static constexpr int kWideners = kRaw ? 8 : 0;
  static constexpr int kWarps = 12 + kWideners;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRingWideners = kWideners / kStreams;
  static constexpr int kSmem = kQBytes + kStreams * (kStages * kStageBytes + kRawStages * kRawBytes);
};

// Least factor of a score: with 0, -inf would become NaN.  Nothing that a finite
// product of it reaches 2^-20.
constexpr float kLeast = 1.4e-45f;

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// TMEM columns.
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 * stream (S: + 64 * buffer)
constexpr uint32_t kPOff = kKeys / 2;       // P in the upper half of its S

template <int N, int R>
struct RingBars {
  uint64_t full[N], empty[N], fixed[N], rfull[R], rempty[R];
};
// One barrier of s_full, p_ready and o_done per S buffer: of the tile two before,
// all three are done when a tile's S is, and none of the tile two behind can be.
struct Bars {
  uint64_t s_full[2][2], p_ready[2][2], o_done[2][2], q_full[2], q_ready[2], q_empty[2], drain[2];
};

// ----------------------------------------------------------------- work ----

struct Req {
  int L, n, mp, kv_end, kt, weight;
};

// Tiles of a request: its units (KV head, group of row tiles) times its key
// tiles.  upt: new tokens of a unit.
__device__ __forceinline__ Req request(const AttnParams &p, int upt, int b, uint32_t &st) {
  Req r;
  lengths(p.bt, b, r.L, r.n, st);
  r.mp = (r.n + upt - 1) / upt;
  r.kv_end = min(r.L + r.n, p.c.max_blocks * p.c.bs);
  r.kt = max(1, (r.kv_end + kKeys - 1) / kKeys);
  r.weight = p.c.heads * r.mp * r.kt;
  return r;
}

__device__ __forceinline__ int weight_of(const AttnParams &p, int upt, int b, uint32_t &st) {
  return b < p.bt.B ? request(p, upt, b, st).weight : 0;
}

// Range i of N <= total over `total` tiles is [start(i), start(i + 1)): none is
// empty.  Range i belongs to stream i / gridDim.x of block i % gridDim.x, so
// that few tiles spread over many blocks.
struct Ranges {
  int N, q, rest;
  float inv;

  __device__ __forceinline__ Ranges(int n, int total) : N(max(n, 1)), q(total / N), rest(total - q * N), inv(1.f / N) {}
  // i * q + i * rest / N.  i, rest < N <= 304: the quotient is an integer or at
  // least 1 / 304 from the next, the product with the reciprocal off by less
  // than 2^-14.
  __device__ __forceinline__ int start(int i) const {
    return i * q + static_cast<int>((static_cast<float>(i * rest) + 0.5f) * inv);
  }
};

// A walk over a range's tiles, unit after unit: where it stands, and the
// segment (a run of key tiles of one unit) it is in.
struct Walk {
  int b, unit, left;      // left: tiles of the range behind this segment
  Req r;
  int h, mp, t0, t1, seg;
  bool on;

  __device__ __forceinline__ int new0() const { return min(r.L, r.kv_end); }  // keys every row sees
};

// To the next segment.  Not inlined: every role of the kernel walks, and the
// copies together would crowd the instruction cache.
__device__ __noinline__ void next_segment(const AttnParams &p, int upt, Walk &w) {
  Walk v = w;
  v.on = v.left > 0;
  if (v.on) {
    if (++v.unit == p.c.heads * v.r.mp) {
      v.unit = 0;
      uint32_t st = 0;
      do {
        v.r = request(p, upt, ++v.b, st);
      } while (v.r.weight == 0);
    }
    v.t0 = 0;                                // a later segment begins a unit
    v.t1 = min(v.r.kt, v.left);
    v.left -= v.t1;
    v.h = v.unit / v.r.mp;
    v.mp = v.unit - v.h * v.r.mp;
  }
  ++v.seg;
  w = v;
}

// What the roles ask about the tile they are at, in registers (a Walk lives in
// local memory, for next_segment takes its address).
struct Tile {
  int t, t0, t1, b, h, mp, seg, kv_end, new0;
  bool on, cut;  // cut: the table is too short

  __device__ __forceinline__ bool first() const { return t == t0; }
  __device__ __forceinline__ bool last() const { return t + 1 == t1; }
};

__device__ __forceinline__ Tile tile_of(const Walk &w) {
  return Tile{w.t0, w.t0, w.t1, w.b, w.h, w.mp, w.seg, w.r.kv_end, w.new0(), w.on, w.r.kv_end < w.r.L + w.r.n};
}

__device__ __forceinline__ void next_tile(const AttnParams &p, int upt, Walk &w, Tile &x) {
  if (++x.t < x.t1) return;
  next_segment(p, upt, w);
  x = tile_of(w);
}

// Tiles of a range whose walk begins.  They are loaded, widened and multiplied
// in one order, K a tile ahead: K0 K1 V0 K2 V1 .. at positions 0 .. 2n - 1.  Even
// positions are K0 V0 V1 .., odd ones K1 K2 .. and the last V.
__device__ __forceinline__ int count_of(const Walk &w) { return w.on ? w.left + w.t1 - w.t0 : 0; }

// Range i's first tile, by a whole warp: the requests are spread over the
// lanes, 32 at a time.
__device__ __forceinline__ void begin_walk(const AttnParams &p, int upt, int i, int limit, Walk &w, int &total) {
  const int lane = threadIdx.x & 31, B = p.bt.B;
  uint32_t st = 0;
  const int mine = weight_of(p, upt, lane, st);  // requests 0 .. 31
  total = mine;
#pragma unroll 1
  for (int b = lane + 32; b < B; b += 32) total += weight_of(p, upt, b, st);
  total = __reduce_add_sync(kFull, total);
  if (i == 0) report(p.bt.status, st);
  const int N = min(limit, total);
  w = Walk{};
  if (i >= N) return;
  const Ranges ranges(N, total);
  const int begin = ranges.start(i);
  w.left = ranges.start(i + 1) - begin;
  int base = 0, x = mine, c = 0;
#pragma unroll 1
  for (;;) {
    const int sum = __reduce_add_sync(kFull, x);
    if (begin < base + sum) break;               // begin < total: it ends
    base += sum;
    c += 32;
    x = weight_of(p, upt, c + lane, st);
  }
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  const int excl = base + incl - x;
  const int src = __ffs(__ballot_sync(kFull, begin >= excl && begin < excl + x)) - 1;
  const int rem = begin - __shfl_sync(kFull, excl, src);
  w.b = c + src;
  w.r = request(p, upt, w.b, st);
  w.unit = rem / w.r.kt;
  w.t0 = rem - w.unit * w.r.kt;
  w.t1 = min(w.r.kt, w.t0 + w.left);
  w.left -= w.t1 - w.t0;
  w.h = w.unit / w.r.mp;
  w.mp = w.unit - w.h * w.r.mp;
  w.seg = 0;
  w.on = true;
}

// A converged warp's wait for an mbarrier phase; false when it gives up, after
// about two seconds.  The warp is suspended meanwhile: polling warps took the
// issue slots of those that widen and of the softmax.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, uint32_t *err) {
  const uint64_t t0 = sv::global_timer_ns();
#pragma unroll 1
  for (uint32_t i = 0; i < (1u << 30); ++i) {
    if (__any_sync(kFull, sv::mbar_try_wait_sleep(bar, parity, 20000u))) return true;
    if (__any_sync(kFull, sv::global_timer_ns() - t0 > sv::kWaitLimitNs)) break;
  }
  report(err, SV_FAULT_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool wait_warp(const uint64_t *bar, uint32_t parity, uint32_t *err) {
  const uint32_t at = sv::smem_addr(bar);
  parity &= 1u;
  return __any_sync(kFull, sv::mbar_try_wait(at, parity)) || wait_long(at, parity, err);
}

// The marked units of a range that its ends do not cut, by all warps of the
// block, when no role waits for another any more: the 128 rows of a tile take
// 4 us a key (e4m3: 8.6), seconds over a long context, and bounded waits would
// run out.  Segments whose number is a marked one's modulo kMarkBits are done
// again as well.
template <typename Q, typename C, int D>
__device__ __noinline__ void recompute_marked(const AttnParams &p, int upt, const Walk &begin, const uint32_t *marks,
                                              int warp, int warps) {
#pragma unroll 1
  for (Walk w = begin; w.on; next_segment(p, upt, w)) {
    if (w.t0 > 0 || w.t1 < w.r.kt || !(marks[w.seg / 32 % (kMarkBits / 32)] >> (w.seg % 32) & 1u)) continue;
    const int rows = min(w.r.n - w.mp * upt, upt) * p.G;
#pragma unroll 1
    for (int row = warp; row < rows; row += warps)
      recompute_row<Q, C, D>(p, w.b, w.mp * upt + row / p.G, w.h * p.G + row % p.G);
  }
}

// ------------------------------------------------------------ main kernel ----

template <typename Q, typename C, int D, bool kPair>
__global__ void __launch_bounds__(Shape<Q, C, D, kPair>::kThreads, 1)
    sv_attn_tc_kernel(const __grid_constant__ TcParams p) {
  using S = Shape<Q, C, D, kPair>;
  extern __shared__ __align__(1024) uint8_t smem[];   // swizzle atoms: 1024 bytes
  __shared__ Bars bars;
  using Ring = RingBars<S::kStages, S::kRaw ? S::kRawStages : 1>;
  __shared__ Ring rings[S::kStreams];
  __shared__ uint32_t tmem_slot;
  __shared__ Walk sh_walk[S::kStreams];
  __shared__ int seg_bad[S::kStreams][kSegRing];  // holds 1 + a marked segment's number
  __shared__ uint32_t marks[S::kStreams][kMarkBits / 32];  // whole units to recompute
  // kRaw: scale bytes that a K tile, and (plus 256) a segment's V, refer to.
  __shared__ int k_scale[S::kStreams][kScaleRing], v_scale[S::kStreams][kSegRing];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t *const sq = smem;
  uint8_t *const ring0 = sq + S::kQBytes;
  uint8_t *const raw0 = ring0 + S::kStreams * S::kStages * S::kStageBytes;

  if (sv::smem_addr(smem) & 1023u) {                    // never: the swizzle would not match
    report(p.err, SV_FAULT_TIMEOUT);
    return;
  }
  if (warp == 11) tc_alloc(sv::smem_addr(&tmem_slot), 512);
  if (tid == 0) {
    for (int r = 0; r < S::kStreams; ++r) {
      for (int i = 0; i < S::kStages; ++i) {
        sv::mbar_init(sv::smem_addr(&rings[r].full[i]), S::kRaw ? S::kRingWideners / 2 : 1);
        sv::mbar_init(sv::smem_addr(&rings[r].empty[i]), kPair ? 2 : 1);
        sv::mbar_init(sv::smem_addr(&rings[r].fixed[i]), 1);
      }
      for (int i = 0; i < S::kRawStages; ++i) {
        sv::mbar_init(sv::smem_addr(&rings[r].rfull[i]), 1);
        sv::mbar_init(sv::smem_addr(&rings[r].rempty[i]), S::kRingWideners / 2);
      }
    }
    for (int s = 0; s < 2; ++s) {
      for (int i = 0; i < kBufs; ++i) {
        sv::mbar_init(sv::smem_addr(&bars.s_full[s][i]), 1);
        sv::mbar_init(sv::smem_addr(&bars.o_done[s][i]), 1);
        sv::mbar_init(sv::smem_addr(&bars.p_ready[s][i]), 4);
      }
      sv::mbar_init(sv::smem_addr(&bars.q_full[s]), 1);
      sv::mbar_init(sv::smem_addr(&bars.q_ready[s]), 4);
      sv::mbar_init(sv::smem_addr(&bars.q_empty[s]), 1);
      sv::mbar_init(sv::smem_addr(&bars.drain[s]), 1);
    }
    for (int s = 0; s < S::kStreams; ++s)
      for (int i = 0; i < kSegRing; ++i) seg_bad[s][i] = 0;
    sv::fence_mbar_init();
  }
  if (warp == 3) {
    for (int s = 0; s < S::kStreams; ++s)
      for (int i = lane; i < kMarkBits / 32; i += 32) marks[s][i] = 0;
  }
  if (tid == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.vmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.qmap) : "memory");
  }
  const AttnParams &a = p.a;
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

  // Where this block's ranges begin: one warp each finds out, all start there.
  const int upt = p.TT * S::kTilesPerUnit;
  uint32_t *const err = p.err;
  bool ok = true, marked = false;
  if (warp >= 8 && warp - 8 < S::kStreams) {
    const int i = static_cast<int>(blockIdx.x + (warp - 8) * gridDim.x);
    Walk w;
    int total;
    begin_walk(a, upt, i, p.ranges, w, total);
    if (lane == 0) {
      sh_walk[warp - 8] = w;
      // Range 0 is written even if there are no tiles: its total says so.
      if (w.on || i == 0) p.cuts[i] = Cut{w.b, w.h, w.mp, w.r.n, w.t0, w.r.kt, total, 0};
    }
  }
  __syncthreads();

  if (warp < 8) {
    // ------------------------------------------------ softmax warpgroups ----
    const int s = warp >> 2;                 // stream
    const int wq = warp & 3;                 // TMEM lanes 32 wq ..
    const uint32_t lanes = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t col_s0 = lanes + kColS + 128u * s, col_o = lanes + kColO + 128u * s;
    const int my = wq * 32 + lane;           // row of the 128-row tile
    const int rs = kPair ? 0 : s;            // range of the block
    // kRaw: bf16 Q as fp16, each row times a power of two that brings its largest
    // magnitude to 2^14 .. 2^15 (exact for elements down to 2^-31 of it, and
    // what is lost below is 2^-39 of it); a tile's factor takes 2^q_next back.
    int q_next = 0;
    const auto prepare_q = [&](const Walk &w) {
      const int rows = min(max(w.r.n - (w.mp * upt + (kPair ? s * p.TT : 0)), 0), p.TT) * a.G;
      if (!wait_warp(&bars.q_full[rs], w.seg, err)) return false;
      if (Q::kIsBf16 && my < rows) {
        uint8_t *q = sq + s * S::kQTile + my * 128;
        uint32_t big = 0;
#pragma unroll 4
        for (int ch = 0; ch < D / 8; ++ch) {
          const uint4 v = *reinterpret_cast<const uint4 *>(q + (ch >> 3) * (kTile * 128) + (((ch & 7) ^ (my & 7)) << 4));
          big = __vmaxu2(big, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                       __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
        }
        const int e = max(static_cast<int>(max(big & 0xffffu, big >> 16) >> 7), 14);   // 127 + exponent
        const float m = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);         // 2^(141 - e)
        q_next = e - 141;
#pragma unroll 4
        for (int ch = 0; ch < D / 8; ++ch) {
          uint4 *at = reinterpret_cast<uint4 *>(q + (ch >> 3) * (kTile * 128) + (((ch & 7) ^ (my & 7)) << 4));
          const uint4 v = *at;
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
          uint32_t h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) h[k] = pack2<F16>(sv::bf16_lo(u[k]) * m, sv::bf16_hi(u[k]) * m);
          *at = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.q_ready[s]));
      return true;
    };
    Walk walk = sh_walk[rs];
    if (S::kRaw && walk.on) ok = prepare_q(walk);
    uint32_t tiles = 0;                      // of the range
#pragma unroll 1
    while (ok && walk.on) {
      const Walk sg = walk;
      const int q_exp = q_next;
      const Req &r = sg.r;
      const int nt = sg.t1 - sg.t0, seg = sg.seg;
      // Tokens and rows of this stream's tile.
      const int tok0 = sg.mp * upt + (kPair ? s * p.TT : 0);
      const int tile_rows = min(max(r.n - tok0, 0), p.TT) * a.G;
      const bool active = wq * 32 < tile_rows;               // warp-uniform
      const int t_row = tok0 + min(my, max(tile_rows - 1, 0)) / a.G;
      const int full_end = sg.new0();                        // every row sees these
      const uint8_t *mrow = a.mask ? a.mask + sg.b * a.msb + static_cast<int64_t>(t_row) * a.bt.T : nullptr;
      float m_ref = -INFINITY, mc = 0.f, l = 0.f;            // log2 units; mc: 0 before a key is seen
#pragma unroll 1
      for (int j = 0; j < nt; ++j, ++tiles) {
        // Which of the tile's keys the row sees, while S is being computed.
        const int k0 = (sg.t0 + j) * kKeys;
        const uint32_t buf = tiles % kBufs, round = tiles / kBufs;
        const uint32_t col_s = col_s0 + 64u * buf;
        const bool masked = k0 + kKeys > full_end;
        uint32_t vis[2] = {~0u, ~0u};
        if (masked && active) {
          const int lim = min(r.kv_end, mrow ? r.L : r.L + t_row + 1) - k0;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int n = min(max(lim - 32 * w, 0), 32);
            vis[w] = n == 32 ? ~0u : (1u << n) - 1u;
          }
          if (mrow) {
            // The row's bytes for new tokens [o0, o1), four at a time where
            // rows are whole words; bit c of the tile is new token k0 + c - L.
            const int o0 = max(k0 - r.L, 0), o1 = min(min(r.kv_end, k0 + kKeys) - r.L, r.n);
            uint64_t lo = 0;
            const auto put = [&](uint64_t bits, int c) { lo |= c < 0 ? bits >> -c : bits << c; };
            if (p.mvec) {
#pragma unroll 4
              for (int o = o0 & ~3; o < o1; o += 4) {
                const uint32_t v = static_cast<uint32_t>(ld32(reinterpret_cast<const int32_t *>(mrow + o)));
                const uint32_t nz = (((v & 0x7f7f7f7fu) + 0x7f7f7f7fu) | v) & 0x80808080u;
                uint32_t bits = ((nz >> 7) * 0x10204080u) >> 28;   // byte e to bit e
                if (o1 - o < 4) bits &= (1u << (o1 - o)) - 1u;
                put(bits, o + r.L - k0);
              }
            } else {
#pragma unroll 1
              for (int o = o0; o < o1; ++o) put(ld8(mrow + o) != 0, o + r.L - k0);
            }
            vis[0] |= static_cast<uint32_t>(lo);
            vis[1] |= static_cast<uint32_t>(lo >> 32);
          }
        }
        if (!(ok = wait_warp(&bars.s_full[s][buf], round, err))) break;
        __syncwarp();
        if (active) {
          tc_fence_after();
          if (masked) {  // scores that the row does not see become -inf, in place
#pragma unroll 1
            for (int w = 0; w < 2; ++w) {
              const uint32_t bits = w == 0 ? vis[0] : vis[1];
              if (__all_sync(kFull, bits == ~0u)) continue;
              uint32_t y[32];
              tc_ld32(col_s + 32u * w, y);
              tc_wait_ld(y);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!((bits >> k) & 1u)) y[k] = 0xff800000u;
              tc_st32(col_s + 32u * w, y);
            }
            tc_wait_st();
            __syncwarp();
          }
          // A chunk of S; the last one of the first pass stays in registers.
          constexpr int W = S::kChunk;
          uint32_t x[W];
          const auto load_s = [&](int ch) {
#pragma unroll
            for (int k = 0; k < W; k += 32) tc_ld32(col_s + ch * W + k, x + k);
            tc_wait_ld(x);
          };
          constexpr int kChunks = kKeys / W;
          float mt = -INFINITY, cf = p.c;
          if constexpr (S::kRaw) {
            // The powers of the row's queries and of the tile's keys together, for
            // they may cancel; in two steps, for the sum may not be an exponent.
            const int e = max(q_exp + k_scale[rs][tiles % kScaleRing] - 127, -252), e0 = e >> 1;
            cf = fmaxf(p.c * pow2(e0) * pow2(e - e0), kLeast);
          }
#pragma unroll
          for (int ch = 0; ch < kChunks; ++ch) {
            load_s(ch);
            float q0 = -INFINITY, q1 = -INFINITY, q2 = -INFINITY, q3 = -INFINITY;
#pragma unroll
            for (int k = 0; k < W; k += 4) {
              q0 = fmaxf(q0, __uint_as_float(x[k]));
              q1 = fmaxf(q1, __uint_as_float(x[k + 1]));
              q2 = fmaxf(q2, __uint_as_float(x[k + 2]));
              q3 = fmaxf(q3, __uint_as_float(x[k + 3]));
            }
            mt = fmaxf(mt, fmaxf(fmaxf(q0, q1), fmaxf(q2, q3)) * cf);
          }
          // Raise the reference where the tile's maximum is more than 2^8
          // above it (or nothing was seen before).
          constexpr float kHead = S::M::kIsBf16 ? 0.f : 7.f;   // 2^(7 + 8) is below fp16's largest
          const bool up = mt - kHead > m_ref && !(mt - m_ref <= kHead + 8.f);
          if (__any_sync(kFull, up)) {
            float f = 1.f;
            if (up) {
              mt -= kHead;
              f = sv::ex2(m_ref - mt);
              m_ref = mc = mt;
              l *= f;
            }
            __syncwarp();
            if (j > 0) {
              // The products of the tile before may still run.
              if (!(ok = wait_warp(&bars.o_done[s][(tiles - 1) % kBufs], (tiles - 1) / kBufs, err))) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tc_ld32(col_o + c, o);
                tc_wait_ld(o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tc_st32(col_o + c, o);
              }
            }
          }
          const uint64_t nm2 = f2_pack(-mc, -mc), c2 = f2_pack(cf, cf);
          uint64_t l2a = 0, l2b = 0;
          // The last chunk first: it is in registers, and P's columns are the
          // upper half of S, where a chunk's P covers only S already taken.
#pragma unroll
          for (int ch = kChunks - 1; ch >= 0; --ch) {
            if (ch < kChunks - 1) load_s(ch);
            uint32_t pk[W / 2];
#pragma unroll
            for (int k = 0; k < W; k += 2) {
              const uint64_t y =
                  f2_fma(f2_pack(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), c2, nm2);
              float y0, y1;
              f2_unpack(y, y0, y1);
              y0 = sv::ex2(y0);
              y1 = sv::ex2(y1);
              if (k & 2) l2a = f2_add(l2a, f2_pack(y0, y1));
              else l2b = f2_add(l2b, f2_pack(y0, y1));
              pk[k >> 1] = pack2<typename S::M>(y0, y1);
            }
            if constexpr (W == 64) tc_st32(col_s + kPOff + ch * (W / 2), pk);
            else tc_st16(col_s + kPOff + ch * (W / 2), pk);
          }
          float e0, e1, e2, e3;
          f2_unpack(l2a, e0, e1);
          f2_unpack(l2b, e2, e3);
          l += (e0 + e1) + (e2 + e3);
          tc_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.p_ready[s][buf]));
      }
      if (!ok) break;
      next_segment(a, upt, walk);
      if (S::kRaw && walk.on && !(ok = prepare_q(walk))) break;   // while the last products run
      if (!(ok = wait_warp(&bars.o_done[s][(tiles - 1) % kBufs], (tiles - 1) / kBufs, err))) break;
      tc_fence_after();
      const float vs = S::kRaw ? scale_value(v_scale[rs][seg % kSegRing] & 255) : 1.f;
      const bool bad = seg_bad[rs][seg % kSegRing] == seg + 1;
      const bool whole = sg.t0 == 0 && sg.t1 == r.kt;
      const int base_row = kPair ? s * kTile : 0;            // of the slot
      const float mx = l == 0.f ? -INFINITY : mc;
      const bool mine = my < tile_rows;
      const bool boss = (tid & 127) == 0 && (!kPair || s == 0);
      float *slot = nullptr;
      uint8_t *orow = nullptr;
      float inv = 1.f;
      if (whole) {
        const int t = tok0 + my / a.G, g = my % a.G;
        const int64_t row = (static_cast<int64_t>(sg.b) * a.bt.T + t) * a.Hq + sg.h * a.G + g;
        orow = a.out + row * (D * 2);
        inv = vs / l;
        if (mine && a.lse && !bad) a.lse[row] = l == 0.f ? -INFINITY : mx * kLn2 + logf(l);
      } else {
        // Slot 0 of the range where the segment starts it, else slot 1.
        slot = p.slots + (static_cast<size_t>(blockIdx.x + rs * gridDim.x) * 2 + (seg == 0 ? 0 : 1)) *
                             p.slot_floats;
        if (mine) {
          slot[D * p.slot_rows + base_row + my] = mx;
          slot[(D + 1) * p.slot_rows + base_row + my] = l;
        }
        if (boss) reinterpret_cast<int *>(slot)[(D + 2) * p.slot_rows] = bad ? 1 : 0;
      }
      if (bad && whole && boss) {
        marks[rs][seg / 32 % (kMarkBits / 32)] |= 1u << (seg % 32);
        marked = true;
      }
      __syncwarp();
      if (active && !bad) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tc_ld32(col_o + c, o);
          tc_wait_ld(o);
          if (mine) {
            if (whole) {
#pragma unroll
              for (int k = 0; k < 32; k += 8) {
                uint32_t u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  u[e] = l == 0.f ? 0u   // not 0 * O: it may be NaN
                                  : pack2<Q>(__uint_as_float(o[k + 2 * e]) * inv, __uint_as_float(o[k + 2 * e + 1]) * inv);
                *reinterpret_cast<uint4 *>(orow + (c + k) * 2) = make_uint4(u[0], u[1], u[2], u[3]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 32; k += 4)
                *reinterpret_cast<float4 *>(slot + (static_cast<size_t>((c + k) >> 2) * p.slot_rows + base_row +
                                                    my) * 4) =
                    make_float4(__uint_as_float(o[k]) * vs, __uint_as_float(o[k + 1]) * vs,
                                __uint_as_float(o[k + 2]) * vs, __uint_as_float(o[k + 3]) * vs);
            }
          }
          __syncwarp();  // the warp's loads from TMEM are executed together
        }
      }
      tc_fence_before();   // O is read before the next P is announced
    }
  } else if (warp < 10) {
    // -------------------------------------------------------- producers ----
    // One warp per ring (two were no faster: 122 us for 32 x 32 heads that share
    // nothing, 115 with one), or (kPair) one for its even and one for its odd
    // positions.  Lane i looks up box i of a tile, an elected lane issues the
    // copies (~90 cycles each).
    const int rs = kPair ? 0 : warp - 8, grp = kPair ? warp - 8 : 0;
    const int box = p.box, nb = kKeys / box;               // boxes of a stage, at most 8
    constexpr int kRing = S::kRaw ? S::kRawStages : S::kStages;
    uint64_t *const fullb = S::kRaw ? rings[rs].rfull : rings[rs].full;
    uint64_t *const emptyb = S::kRaw ? rings[rs].rempty : rings[rs].empty;
    const uint32_t stage0 = S::kRaw ? sv::smem_addr(raw0) + rs * (S::kRawStages * S::kRawBytes)
                                    : sv::smem_addr(ring0) + rs * (S::kStages * S::kStageBytes);
    constexpr int kRingBytes = S::kRaw ? S::kRawBytes : S::kStageBytes;
    int issued = -1, q_last = -1;                       // last position, last segment's Q
    // This lane's box of a tile: its block and the row in it (-1: no box).
    struct Box {
      int id, row, h;
    };
    const int32_t *table = nullptr;          // the segment's
    int block = 0, row = 0;                  // of the lane's box in the tile
    const int step_block = kKeys / a.c.bs, step_row = kKeys - step_block * a.c.bs;
    const auto fetch = [&](const Tile &w) {
      const int pos = w.t * kKeys + lane * box;
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
      Box x = {0, -1, w.h};
      if (w.on && lane < nb && pos < w.kv_end) {
        x.row = row;
        x.id = ld32(table + block);
      }
      return x;
    };
    // A block that is not there marks the segment, whose unit is recomputed;
    // any block is loaded in its place.
    const auto settle = [&](Box &x, const Tile &w) {
      if (x.row >= 0 && static_cast<uint32_t>(x.id) >= static_cast<uint32_t>(a.c.num_blocks)) {
        report(a.bt.status, x.id == -1 ? SV_KV_MISSING_BLOCK : SV_KV_BAD_BLOCK);
        seg_bad[rs][w.seg % kSegRing] = w.seg + 1;
        x.id = 0;
      }
      __syncwarp();  // the mark before the elected lane's arrival on the stage's barrier
    };
    // A tile's K or V into the next stage.
    int st = grp, round = 0;                 // of the next position
    const uint32_t sblock = static_cast<uint32_t>(a.c.sblock_bytes);   // < 2^31
    const auto load = [&](const Box &x, bool is_v) {
      const CUtensorMap *map = is_v ? &p.vmap : &p.kmap;
      constexpr int srow = D / SV_KV_GROUP;
      const uint32_t box_bytes = S::kRaw ? box * (D + srow) : S::kHalves * box * 128;
      const int boxes = __popc(__ballot_sync(kFull, x.row >= 0));  // the first ones
      const uint8_t *scales = is_v ? a.c.vs : a.c.ks;
      if (round > 0 && !wait_warp(&emptyb[st], round - 1, err)) return false;
      const uint32_t bar = sv::smem_addr(fullb) + 8u * st, dst = stage0 + st * kRingBytes;
      const auto issue = [&](int i, int id, int row) {
        const int at = i * box;              // row in the stage
        if constexpr (S::kRaw) {
          tma_4d(dst + at * D, map, 0, row, x.h, id, bar);
          bulk_1d(dst + S::kRawData + at * srow,
                  scales + static_cast<uint64_t>(static_cast<uint32_t>(id)) * sblock + (x.h * a.c.bs + row) * srow,
                  box * srow, bar);
        } else {
#pragma unroll
          for (int hf = 0; hf < S::kHalves; ++hf)
            tma_4d(dst + hf * S::kHalf + at * 128, map, hf * 64, row, x.h, id, bar);
        }
      };
      int i = 0;
#pragma unroll 1
      do {                                   // two boxes at a time: their look-ups overlap
        const int id0 = __shfl_sync(kFull, x.id, i), id1 = __shfl_sync(kFull, x.id, i + 1);
        const int row0 = __shfl_sync(kFull, x.row, i), row1 = __shfl_sync(kFull, x.row, i + 1);
        if (elect_one()) {
          if (i == 0) sv::mbar_arrive_expect_tx(bar, boxes * box_bytes);
          if (i < boxes) issue(i, id0, row0);
          if (i + 1 < boxes) issue(i + 1, id1, row1);
        }
        __syncwarp();
      } while ((i += 2) < boxes);
      issued = round * kRing + st;
      st += kPair ? 2 : 1;
      if (st >= kRing) {
        st -= kRing;
        ++round;
      }
      return true;
    };
    // A segment's queries: whole tokens, G heads each, in the swizzled layout.
    const auto load_q = [&](const Tile &w) {
      if (lane == 0 && w.cut) report(a.bt.status, SV_KV_TABLE_SHORT);
      if (w.seg > 0 && !wait_warp(&bars.q_empty[rs], w.seg - 1, err)) return false;
      if (kPair && w.seg > 0 && !wait_warp(&bars.q_empty[1], w.seg - 1, err)) return false;
      const uint32_t bar = sv::smem_addr(&bars.q_full[rs]);
      if (elect_one()) {
        sv::mbar_arrive_expect_tx(bar, S::kTilesPerUnit * S::kHalves * p.qbox * a.G * 128);
#pragma unroll
        for (int i = 0; i < S::kTilesPerUnit; ++i)
#pragma unroll
          for (int hf = 0; hf < S::kHalves; ++hf)
            tma_4d(sv::smem_addr(sq) + (kPair ? i : rs) * S::kQTile + hf * (kTile * 128), &p.qmap,
                   hf * 64, w.h * a.G, w.mp * upt + i * p.TT, w.b, bar);
      }
      __syncwarp();
      q_last = w.seg;
      return true;
    };
    Walk walk = sh_walk[rs];
    Tile w = tile_of(walk);
    Box x = fetch(w);                        // of the next tile
    const int n = count_of(walk);
    if constexpr (kPair) {
      if (grp && n > 1) {
        next_tile(a, upt, walk, w);
        x = fetch(w);
      }
#pragma unroll 1
      for (int i = 0; ok && i < n; ++i) {
        const bool is_v = grp ? i == n - 1 : i > 0;
        const Tile at = w;
        Box now = x;
        settle(now, w);
        if (grp ? i + 2 < n : i > 0) {
          next_tile(a, upt, walk, w);
          x = fetch(w);                      // on its way while the stage is waited for
        }
        ok = load(now, is_v);
        if (ok && !is_v && at.first()) ok = load_q(at);
      }
    } else {
      Box b0 = x, b1 = x;                    // of the two tiles before
#pragma unroll 1
      for (int pos = 0; ok && pos < 2 * n; ++pos) {
        const bool tail = pos + 1 == 2 * n;  // the last V
        if ((pos & 1 || pos == 0) && !tail) {
          b0 = b1;
          settle(x, w);
          b1 = x;
          ok = load(x, false);
          if (ok && w.first()) ok = load_q(w);
          next_tile(a, upt, walk, w);
          x = fetch(w);                      // on its way while a V is loaded
        } else {
          ok = load(tail ? b1 : b0, true);
        }
      }
    }
    if (!ok) {  // copies in flight land before the block ends (a position not issued: the wait gives up)
#pragma unroll 1
      for (int k = max(0, issued - kRing + 1); k <= issued; ++k) wait_warp(&fullb[k % kRing], k / kRing, err);
      if (q_last >= 0) wait_warp(&bars.q_full[rs], q_last, err);
    }
  } else if (warp < 12) {
    // -------------------------------------------------------- products ----
    // One warp per stream issues its Q K^T and P V, in order.
    const int s = warp - 10, rs = kPair ? 0 : s;
    const uint32_t kQK = mma_desc<typename S::M>(kKeys, false) | (p.negate ? kNegateA : 0u);
    constexpr uint32_t kPV = mma_desc<typename S::M>(D, true);
    uint8_t *const ring = ring0 + rs * (S::kStages * S::kStageBytes);
    Ring &rb = rings[rs];
    const uint64_t q_desc = smem_desc(sv::smem_addr(sq) + s * S::kQTile, 16);
    const uint64_t k_desc = smem_desc(sv::smem_addr(ring), 16);
    const uint64_t v_desc = smem_desc(sv::smem_addr(ring), S::kHalf);
    const uint32_t ts = tmem + kColS + 128u * s, to = tmem + kColO + 128u * s;
    uint32_t fix = 0;              // parities of the repairs, per stage
    uint32_t nk = 0, nv = 0;       // tiles multiplied so far
    int st = 0, round = 0;         // of the next position
    const auto take = [&] {
      const bool good = wait_warp(&rb.full[st], round, err);
      tc_fence_after();
      return good;
    };
    const auto next_stage = [&] {
      if (++st == S::kStages) {
        st = 0;
        ++round;
      }
    };
    // Not kRaw: rows of V behind the committed tokens, keys k0 .. of a stage.
    // What lies behind the last token becomes 0, a value that is not finite
    // marks the segment.
    const auto repair = [&](const Tile &w, int k0, int st) {
      uint8_t *base = ring + st * S::kStageBytes;
      const int r0 = max(w.new0 - k0, 0), r1 = w.kv_end - k0;   // new rows [r0, r1)
      constexpr int kCh = S::kHalves * 8;
      bool found = false;
#pragma unroll 2
      for (int i = lane + r0 * kCh; i < kKeys * kCh; i += 32) {
        const int row = i / kCh, ch = i % kCh;
        uint4 *v = reinterpret_cast<uint4 *>(base + (ch >> 3) * S::kHalf + row * 128 + (ch & 7) * 16);
        if (row >= r1) {
          *v = make_uint4(0, 0, 0, 0);
        } else {
          const uint4 y = *v;
          found = found || odd16<Q>(y.x) || odd16<Q>(y.y) || odd16<Q>(y.z) || odd16<Q>(y.w);
        }
      }
      if (found) seg_bad[rs][w.seg % kSegRing] = w.seg + 1;
      fence_async_smem();
      __syncwarp();
    };
    // S of a tile.
    const auto qk = [&](const Tile &w) {
      if (w.first() && !wait_warp(S::kRaw ? &bars.q_ready[s] : &bars.q_full[rs], w.seg, err)) return false;
      if (!take()) return false;
      const uint64_t kd = k_desc + st * (S::kStageBytes >> 4);
      const uint32_t buf = nk % kBufs;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma_ss(ts + 64u * buf, q_desc + (((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4),
                    kd + (((k >> 2) * S::kHalf + (k & 3) * 32) >> 4), kQK, k > 0);
        tc_commit(sv::smem_addr(&rb.empty[st]));
        tc_commit(sv::smem_addr(&bars.s_full[s][buf]));
        if (w.last()) tc_commit(sv::smem_addr(&bars.q_empty[s]));
      }
      __syncwarp();
      next_stage();
      ++nk;
      return true;
    };
    // O += P V.
    const auto pv = [&](const Tile &w) {
      const int k0 = w.t * kKeys;
      if (!take()) return false;
      if (!S::kRaw && k0 + kKeys > w.new0) {
        if (!kPair || s == 0) {
          repair(w, k0, st);
          if (kPair && lane == 0) sv::mbar_arrive(sv::smem_addr(&rb.fixed[st]));
        } else {
          if (!wait_warp(&rb.fixed[st], fix >> st, err)) return false;
          fix ^= 1u << st;
        }
      }
      const uint32_t buf = nv % kBufs;
      if (!wait_warp(&bars.p_ready[s][buf], nv / kBufs, err)) return false;
      tc_fence_after();
      const uint64_t vd = v_desc + st * (S::kStageBytes >> 4);
      const uint32_t first = w.first();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_ts(to, ts + 64u * buf + kPOff + 8u * k, vd + k * (2048 >> 4), kPV, !(first && k == 0));
        tc_commit(sv::smem_addr(&rb.empty[st]));
        tc_commit(sv::smem_addr(&bars.o_done[s][buf]));
      }
      __syncwarp();
      next_stage();
      ++nv;
      return true;
    };
    Walk walk = sh_walk[rs];
    Tile w = tile_of(walk), behind = w;
    const int n = count_of(walk);
#pragma unroll 1
    for (int i = 0; ok && i <= n && n > 0; ++i) {
      if (i < n) ok = qk(w);
      if (ok && i > 0) ok = pv(behind);
      behind = w;
      if (i < n) next_tile(a, upt, walk, w);
    }
    if (!ok) {  // issued products end before TMEM is freed
      if (elect_one()) tc_commit(sv::smem_addr(&bars.drain[s]));
      __syncwarp();
      wait_warp(&bars.drain[s], 0, err);
    }
  } else {
    // ------------------------------------------------------------ wideners ----
    // e4m3 stages as fp16, 16 codes at a time, into the swizzled layout: a code
    // becomes code * 2^(e - E), one conversion and one product for two codes
    // (as bf16 numbers they took six, and the widening bound the kernel).  E is
    // the largest e of the stage for K, that of a segment's first stage for V;
    // S and O are scaled back in fp32.  A code is a multiple of 2^-9, so that the
    // product is exact down to e = E - 15.  A unit whose scales differ by more is
    // recomputed: the key that sets a stage's E may be one that a row does not
    // see, or sees without weight, and must not round those that count (at
    // E - 24 a code is rounded to a whole number).  Zeros at the smallest scale
    // (2^-120, which the cache writes for them) do not count.
    //
    // The wideners of a ring are two groups, of its even and its odd positions:
    // what a stage costs besides its conversions (two waits, the scales, a
    // fence) is latency, and two stages at a time hide each other's.  A group
    // waits for a stage to be empty before it waits for the raw one: by then the
    // stage's last user is done, so that no parity is a round ahead (rings of
    // different sizes: kRawStages is even, and the raw stage's last user is the
    // group itself).
    static_assert(S::kRawStages == S::kStages || S::kRawStages % 2 == 0, "parities");
    constexpr int kGW = S::kRaw ? S::kRingWideners / 2 : 1, kRS = S::kRaw ? S::kRawStages : 1;
    const int rs = kPair ? 0 : (warp - 12) / (2 * kGW), grp = warp & 1;
    const int ht = ((warp - 12 - rs * 2 * kGW) >> 1) * 32 + lane;
    Ring &rb = rings[rs];
    uint8_t *const ring = ring0 + rs * (S::kStages * S::kStageBytes);
    uint8_t *const raw = raw0 + rs * (S::kRawStages * S::kRawBytes);
    int v_ref = 0;
    // This thread's chunks: 16 codes (column group ch) of every kRowStep-th row.
    // Eight lanes write 4 chunks of one row and 4 of the next, whose swizzles
    // differ in the lowest bit: eight different 16-byte columns of the banks.
    constexpr int kCh = D / 16, kRowStep = kGW * 32 / kCh, kRows = kKeys / kRowStep, kTurn = kRows < 4 ? kRows : 4;
    static_assert(kRowStep % 8 == 0 || !S::kRaw, "one swizzle per thread");
    const int ch = (ht & 3) + (kCh == 8 ? (ht >> 3 & 1) * 4 : 0);
    const int row0 = (kCh == 8 ? ht >> 4 : ht >> 3) * 2 + (ht >> 2 & 1);
    const int from = row0 * D + ch * 16;
    const int to_row = (ch >> 2) * S::kHalf + row0 * 128, c0 = (ch & 3) * 2;
    const int to_lo = to_row + ((c0 ^ (row0 & 7)) << 4), to_hi = to_row + (((c0 + 1) ^ (row0 & 7)) << 4);
    // A tile's K (the range's k-th) or V, at the group's next position.
    int st = grp, round = 0, rst = grp, rround = 0;
    const auto widen = [&](const Tile &w, bool is_v, int k) {
      const int k0 = w.t * kKeys;
      if (round > 0 && !wait_warp(&rb.empty[st], round - 1, err)) return false;
      if (!wait_warp(&rb.rfull[rst], rround, err)) return false;
      const uint8_t *src = raw + rst * S::kRawBytes;
      const uint8_t *sc = src + S::kRawData;
      uint8_t *dst = ring + st * S::kStageBytes;
      constexpr int kSc = D / SV_KV_GROUP;            // scale bytes of a row
      const int live = min(w.kv_end - k0, kKeys);  // rows that hold tokens
      int *const vs = &v_scale[rs][w.seg % kSegRing];
      if (is_v) {
        if (w.first()) {
          v_ref = 0;
        } else if (grp) {                             // a range's last V: the other group had the one before
          const int pos = round * S::kStages + st - 1;
          if (!wait_warp(&rb.full[pos % S::kStages], pos / S::kStages, err)) return false;
          const int x = *vs;
          v_ref = x & 256 ? x & 255 : 0;
        }
      }
      int ref = v_ref;
      if (!is_v || v_ref == 0) {
        // The stage's largest scale, over the rows that hold tokens: each warp
        // reads them all.
        int hi = 0;
        if (live == kKeys) {
          uint32_t m = 0;
#pragma unroll
          for (int k = 0; k < kKeys * kSc / 128; ++k) {
            const uint32_t u = *reinterpret_cast<const uint32_t *>(sc + (k * 32 + lane) * 4);
            m = __vmaxu2(m, __vmaxu2(u & 0x00ff00ffu, (u >> 8) & 0x00ff00ffu));
          }
          hi = max(m & 0xffff, m >> 16);
        } else {
#pragma unroll 1
          for (int i = lane; i < live * kSc; i += 32) hi = max(hi, static_cast<int>(sc[i]));
        }
        ref = min(__reduce_max_sync(kFull, hi), 254);
        if (is_v) {
          if (ref > 7) v_ref = ref;                   // the first stage with more than zeros
          else ref = 254;
          __syncwarp();
          if (ht == 0) *vs = v_ref ? 256 + ref : ref;
        } else if (ht == 0) {
          k_scale[rs][k % kScaleRing] = ref;
        }
      }
      // A turn's chunks together, loads first: a chunk alone is a chain of
      // latencies.
      bool found = false;
      const int least = ref - 14;
      const uint32_t span = min(is_v ? 14 + 7 : 14, 254 - least);   // 255: NaN
#pragma unroll 1
      for (int t0 = 0; t0 < kRows; t0 += kTurn) {
        uint4 c[kTurn];
        int x[kTurn];
#pragma unroll
        for (int t = 0; t < kTurn; ++t) {
          c[t] = *reinterpret_cast<const uint4 *>(src + from + (t0 + t) * kRowStep * D);
          x[t] = sc[row0 * kSc + (ch >> 1) + (t0 + t) * kRowStep * kSc];
        }
        // 2^(e - E) as fp16, twice: where it is a normal number, its exponent
        // field; else (rows behind the last token, zeros, scales far apart)
        // rounded as fp32 is, a subnormal number or 0 where it is that small.
        uint32_t far = 0, m[kTurn];
#pragma unroll
        for (int t = 0; t < kTurn; ++t) {
          far = max(far, static_cast<uint32_t>(x[t] - least));
          m[t] = (x[t] - least + 1) * 0x04000400u;
        }
        if (__any_sync(kFull, far > span)) {
          // Scales that the products cannot hold (448 * 2^7 is below fp16's
          // largest), and NaN: the unit is recomputed.
          const int below = ref - 15, above = min(is_v ? ref + 7 : ref, 254);
#pragma unroll
          for (int t = 0; t < kTurn; ++t) {
            const uint32_t any = (c[t].x | c[t].y | c[t].z | c[t].w) & 0x7f7f7f7fu;
            found = found || (row0 + (t0 + t) * kRowStep < live && (x[t] > 7 || any) && (x[t] < below || x[t] > above));
            const float mf = __uint_as_float(static_cast<uint32_t>(min(max(x[t] - ref + 127, 0), 254)) << 23);
            m[t] = pack2<F16>(mf, mf);
          }
        }
#pragma unroll
        for (int t = 0; t < kTurn; ++t) {
          const __half2 mul = *reinterpret_cast<const __half2 *>(&m[t]);
          const uint32_t u[4] = {c[t].x, c[t].y, c[t].z, c[t].w};
          uint32_t o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                static_cast<__nv_fp8x2_storage_t>(u[k >> 1] >> (16 * (k & 1))), __NV_E4M3);
            const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&h), mul);
            o[k] = *reinterpret_cast<const uint32_t *>(&y);
          }
          uint8_t *to = dst + (t0 + t) * kRowStep * 128;
          *reinterpret_cast<uint4 *>(to + to_lo) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4 *>(to + to_hi) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
      if (is_v && k0 + kKeys > w.new0) {  // the last tiles of a unit: the thread's own rows once more
        const int r0 = max(w.new0 - k0, 0), r1 = w.kv_end - k0;
#pragma unroll 1
        for (int t = 0; t < 2 * kRows; ++t) {
          const int row = row0 + (t >> 1) * kRowStep;
          uint4 *at = reinterpret_cast<uint4 *>(dst + (t >> 1) * kRowStep * 128 + (t & 1 ? to_hi : to_lo));
          if (row >= r1) {
            *at = make_uint4(0, 0, 0, 0);
          } else if (row >= r0) {
            const uint4 y = *at;
            found = found || odd16<F16>(y.x) || odd16<F16>(y.y) || odd16<F16>(y.z) || odd16<F16>(y.w);
          }
        }
      }
      if (found) seg_bad[rs][w.seg % kSegRing] = w.seg + 1;
      fence_async_smem();
      __syncwarp();
      if (lane < 2) sv::mbar_arrive(sv::smem_addr(lane ? &rb.rempty[rst] : &rb.full[st]));
      if ((st += 2) >= S::kStages) {
        st -= S::kStages;
        ++round;
      }
      if ((rst += 2) >= kRS) {
        rst -= kRS;
        ++rround;
      }
      return true;
    };
    Walk walk = sh_walk[rs];
    Tile w = tile_of(walk);
    const int n = count_of(walk);
    bool step = grp && n > 1;                // to the next tile
#pragma unroll 1
    for (int i = 0; ok && i < n; ++i) {
      if (step) next_tile(a, upt, walk, w);
      ok = widen(w, grp ? i == n - 1 : i > 0, i + grp);
      step = grp ? i + 2 < n : i > 0;
    }
  }

  tc_fence_before();
  const bool some = __syncthreads_or(marked);
  tc_fence_after();
  if (warp == 11) tc_dealloc(tmem, 512);
  if (some) {
#pragma unroll 1
    for (int rs = 0; rs < S::kStreams; ++rs)
      recompute_marked<Q, C, D>(a, upt, sh_walk[rs], marks[rs], warp, S::kWarps);
  }
}

// ---------------------------------------------------------- second kernel ----

constexpr int kJoinThreads = 256;

// Joins the partial results of a unit that range ends cut: block (x, y) looks
// at the cut where range x + 1 begins and, if it is the unit's first, joins
// part y of the unit's rows x D / 4 columns.  Each thread has E = 4 columns of a
// row, whose loads are in flight together, and the grid is a quarter of what it
// is with one (8 chains of 6 tokens: 28 us of both kernels together, 32.5 with
// one; 16 trees of 64 nodes: 100 and 111), and K threads share them, each with
// every K-th range.
constexpr int kJoinCols = 4;

template <typename Q, typename C, int D, bool kPair>
__global__ void __launch_bounds__(kJoinThreads) sv_attn_join_kernel(const __grid_constant__ TcParams p, const int K) {
  constexpr int E = kJoinCols;
  __shared__ float4 so[E][kJoinThreads];
  __shared__ float sm[kJoinThreads], sl[kJoinThreads];
  const AttnParams &a = p.a;
  const int i = static_cast<int>(blockIdx.x) + 1, tid = threadIdx.x;
  sv::pdl_wait();
  sv::pdl_launch_dependents();
  const int4 *cp = reinterpret_cast<const int4 *>(p.cuts);
  const int4 z = __ldcg(cp + 1), u0 = __ldcg(cp + 2 * i), u1 = __ldcg(cp + 2 * i + 1);
  const int total = z.z, N = min(p.ranges, total);
  if (i >= N || u1.x == 0) return;                    // no such range, or a unit begins with it
  const Ranges ranges(N, total);
  const int b = u0.x, h = u0.y, mp = u0.z, n = u0.w, kt = u1.y;
  const int start = ranges.start(i) - u1.x, c0 = i - 1, before = ranges.start(c0);
  if (before > start) return;                         // cut before as well: another block's
  const int late = before == start ? 0 : 1;
  // The range of the unit's last tile: an estimate, put right.
  const int end = start + kt - 1;
  int c1 = min(N - 1, static_cast<int>(static_cast<float>(end) * N / static_cast<float>(total)));
  while (ranges.start(c1) > end) --c1;
  while (c1 + 1 < N && ranges.start(c1 + 1) <= end) ++c1;
  const int upt = p.TT * (kPair ? 2 : 1), tok0 = mp * upt, rows = min(upt, n - tok0) * a.G;
  const auto slot_of = [&](int c) {
    return p.slots + (static_cast<size_t>(c) * 2 + (c == c0 ? late : 0)) * p.slot_floats;
  };
  int bad = 0;
  for (int c = c0 + tid % 32; c <= c1; c += 32)
    bad |= __ldcg(reinterpret_cast<const int32_t *>(slot_of(c)) + (D + 2) * p.slot_rows);
  constexpr int kCols = D / 4 / E;                    // columns e * kCols + d4, of 4 elements
  const int per = kJoinThreads / K, k = tid / per, o = blockIdx.y * per + tid % per;
  const bool in = o < rows * kCols;
  const int d4 = in ? o / rows : 0, row = in ? o - d4 * rows : 0;
  // Rows of the second tile start at row 128 of a slot.
  const int tile_rows = p.TT * a.G, srow = row < tile_rows ? row : kTile + row - tile_rows;
  float m = -INFINITY, l = 0.f;
  float4 v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  const auto add = [&](float m2, float l2, const float4 (&w)[E]) {
    const float nm = fmaxf(m, m2), nb = nm == -INFINITY ? 0.f : nm;
    const float f = sv::ex2(m - nb), g = sv::ex2(m2 - nb);
    m = nm;
    l = l * f + l2 * g;
#pragma unroll
    for (int e = 0; e < E; ++e)
      v[e] = make_float4(v[e].x * f + w[e].x * g, v[e].y * f + w[e].y * g, v[e].z * f + w[e].z * g,
                         v[e].w * f + w[e].w * g);
  };
  if (in) {
#pragma unroll 2
    for (int c = c0 + k; c <= c1; c += K) {
      const float *s = slot_of(c);
      const float m2 = __ldcg(s + D * p.slot_rows + srow), l2 = __ldcg(s + (D + 1) * p.slot_rows + srow);
      float4 w[E];
#pragma unroll
      for (int e = 0; e < E; ++e)
        w[e] = __ldcg(reinterpret_cast<const float4 *>(s) + static_cast<size_t>(e * kCols + d4) * p.slot_rows + srow);
      add(m2, l2, w);
    }
  }
  if (__any_sync(kFull, bad)) {                       // the same for every warp
    constexpr int warps = kJoinThreads / 32;
    for (int r = blockIdx.y * warps + tid / 32; r < rows; r += gridDim.y * warps)
      recompute_row<Q, C, D>(a, b, tok0 + r / a.G, h * a.G + r % a.G);
    return;
  }
  if (K > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) so[e][tid] = v[e];
    sm[tid] = m;
    sl[tid] = l;
    __syncthreads();
    if (k > 0) return;
    for (int q = 1; q < K; ++q) {
      float4 w[E];
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] = so[e][q * per + tid];
      add(sm[q * per + tid], sl[q * per + tid], w);
    }
  }
  if (!in) return;
  const float inv = 1.f / l;
  const int t = tok0 + row / a.G, g = row % a.G;
  const int64_t orow = (static_cast<int64_t>(b) * a.bt.T + t) * a.Hq + h * a.G + g;
#pragma unroll
  for (int e = 0; e < E; ++e)
    *reinterpret_cast<uint2 *>(a.out + orow * (D * 2) + (e * kCols + d4) * 8) =
        l == 0.f ? make_uint2(0u, 0u)   // not 0 * v: it may be NaN
                 : make_uint2(pack2<Q>(v[e].x * inv, v[e].y * inv), pack2<Q>(v[e].z * inv, v[e].w * inv));
  if (a.lse && d4 == 0) a.lse[orow] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

}  // namespace svp
