// sv_attn_tc.cuh -- tree attention over the paged cache on the tensor cores
// (tcgen05), for head dimensions 64 and 128.
//
// Rows.  All n new tokens and the G query heads that share a KV head form one
// matrix of n * G rows, row r = token r / G, head r % G, so that a key is read
// once for all of them; a tile takes as many whole tokens as fit 128 rows.  S = Q K^T and O = P V run as M = 128 row tiles with
// 128 keys a step; S and O live in tensor memory (TMEM: lane = row, one
// thread per row), P overwrites half of its S as the 16-bit A operand.
//
// Two streams of such steps alternate in a thread block, each with a softmax
// warpgroup of its own, so that the tensor cores work on one while the other
// takes exponentials.  With at most 128 rows the streams are independent, each
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
// O is rescaled only when a tile's maximum exceeds m by more than 2^8 (bf16
// and fp16 hold 2^8 as exactly as 1, fp32 sums lose nothing), which after
// the first tiles is rare.
//
// Data.  TMA boxes of one page's rows (or of gcd(block size, 128) rows) fill
// 128-byte swizzled tiles through an mbarrier ring; e4m3 tiles arrive raw with
// their scale bytes and are widened to 16-bit tiles by four warps (exactly:
// code * 2^e is a bf16 number).  Rows of V behind the last token are zeroed
// in shared memory, because 0 * garbage may be NaN; a value that is not
// finite among the new tokens, or a missing block, marks the unit, and the
// second kernel recomputes it row by row (sv_attn_general.cuh).
#pragma once

#include <cuda.h>

#include "sv_attn_general.cuh"

namespace svp {

constexpr int kMaxGrid = 152;   // thread blocks, one per SM
constexpr int kTile = 128;      // keys per step, rows per tile
constexpr int kSegRing = 8;

struct TcParams {
  CUtensorMap kmap, vmap, qmap;
  AttnParams a;
  uint32_t *err;       // SV_FAULT_TIMEOUT goes here
  int32_t *head;       // [0] tiles of all ranges
  int32_t *pre;        // [B + 1] tiles before each request
  uint8_t *dirty;      // [B * heads * MP] units to recompute (whole ranges)
  float *slots;        // [ranges * 2] partial results
  int ranges;
  int slot_rows;       // rows of a slot
  int slot_floats;
  int MP;              // row-tile groups per (request, head), at most
  int box;             // rows of a TMA box of the cache
  int TT;              // tokens of a row tile: its rows are TT * G <= 128
  int qbox;            // tokens of a TMA box of the queries
  int mvec;            // mask rows are whole 4-byte words
  float c;             // |scale| * log2(e), at least 1e-30
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
  static constexpr int kHalves = D / 64;
  static constexpr int kStageBytes = kTile * D * 2;
  static constexpr int kStreams = kPair ? 1 : 2;    // ranges of a block
  static constexpr int kQBytes = 2 * kStageBytes;
  static constexpr int kRawData = kTile * D, kRawScale = kTile * (D / SV_KV_GROUP);
  static constexpr int kRawBytes = kRawData + kRawScale;
  // Ring sizes: as many stages as 227 KB hold (about 200 KB where tiles are
  // small); raw stages first, they are what is in flight.
  static constexpr int kStages = kRaw ? 3 : D == 128 ? 5 : 11;
  static constexpr int kRawStages = kRaw ? (D == 128 ? 3 : 10) : 0;
  static constexpr int kHelpers = kRaw ? 6 : 2;     // warps: 3 or 4 per scheduler in all
  static constexpr int kWarps = 10 + kHelpers;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kChunk = kRaw ? 32 : 64;     // S columns in registers at once
  static constexpr int kTilesPerUnit = kPair ? 2 : 1;
  static constexpr int kSmem = kQBytes + kStages * kStageBytes + kRawStages * kRawBytes;
};

// TMEM columns.
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 * stream
constexpr uint32_t kPOff = 64;              // P in the upper half of its S

struct Bars {
  uint64_t full[12], empty[12], fixed[12], rfull[10], rempty[10];
  uint64_t s_full[2], p_half[2], p_ready[2], o_done[2], q_full[2], q_empty[2], drain;
};

// ----------------------------------------------------------------- work ----

struct Req {
  int L, n, mp, kv_end, kt, weight;
};

// Tiles of a request: its units (KV head, group of row tiles) times its key
// tiles.  upt: new tokens of a unit.
__device__ __forceinline__ Req make_request(const AttnParams &p, int upt, int L, int n) {
  Req r;
  r.L = L;
  r.n = n;
  r.mp = (n + upt - 1) / upt;
  r.kv_end = min(L + n, p.c.max_blocks * p.c.bs);
  r.kt = max(1, (r.kv_end + kTile - 1) / kTile);
  r.weight = p.c.heads * r.mp * r.kt;
  return r;
}
__device__ __forceinline__ Req request(const AttnParams &p, int upt, int b, uint32_t &st) {
  int L, n;
  lengths(p.bt, b, L, n, st);
  return make_request(p, upt, L, n);
}

// Lengths of the requests from a range's first one on, in shared memory.
constexpr int kReqCache = 32;
struct ReqCache {
  int b0;
  int2 len[kReqCache];
};

// A run of key tiles [t0, t1) of one unit.
struct Seg {
  int b, unit, h, mp, t0, t1;
  Req r;
};

// Walks a range of the tile sequence, unit after unit.
struct Walk {
  int b, unit, tile, left;
  Req r;
};

__device__ __forceinline__ Req fetch_request(const AttnParams &p, int upt, const ReqCache &rc, int b) {
  if (b - rc.b0 < kReqCache) {
    const int2 v = rc.len[b - rc.b0];
    return make_request(p, upt, v.x, v.y);
  }
  uint32_t st = 0;
  return request(p, upt, b, st);
}

// The next segment of a walk, false at its end.  `rem` >= 0 begins the walk:
// tiles of the first request before the range.  Not inlined: every role of the
// kernel walks, and the copies together would not fit the instruction cache.
__device__ __noinline__ bool walk_next(const AttnParams &p, int upt, const ReqCache &rc, Walk &w, Seg &s,
                                       int rem) {
  if (w.left <= 0) return false;
  if (rem >= 0) {
    w.b = rc.b0;
    w.r = fetch_request(p, upt, rc, w.b);
    w.unit = rem / w.r.kt;
    w.tile = rem - w.unit * w.r.kt;
  }
  s.b = w.b;
  s.r = w.r;
  s.unit = w.unit;
  s.h = w.unit / w.r.mp;
  s.mp = w.unit - s.h * w.r.mp;
  s.t0 = w.tile;
  s.t1 = min(w.r.kt, w.tile + w.left);
  w.left -= s.t1 - s.t0;
  w.tile = s.t1;
  if (w.tile == w.r.kt) {
    w.tile = 0;
    if (++w.unit == p.c.heads * w.r.mp) {
      w.unit = 0;
      if (w.left > 0) {
        do {
          ++w.b;
          w.r = fetch_request(p, upt, rc, w.b);
        } while (w.r.weight == 0);
      }
    }
  }
  return true;
}

// Range i of N <= total over `total` tiles is [start(i), start(i + 1)): none is
// empty.  Range i belongs to stream i / gridDim.x of block i % gridDim.x, so
// that few tiles spread over many blocks.
__device__ __forceinline__ int range_start(int i, int N, int total) {
  return static_cast<int>(static_cast<int64_t>(i) * total / N);
}
__device__ __forceinline__ int range_of(int tile, int N, int total) {
  return static_cast<int>(((static_cast<int64_t>(tile) + 1) * N - 1) / total);
}

// A tile step of a walk: where it is and what the roles ask about it.
struct Cursor {
  int b, h, mp, t, t0, t1, seg, new0, kv_end;  // new0: keys that every row sees
  bool on, cut;                                // cut: the table is too short

  __device__ __forceinline__ bool first() const { return t == t0; }
  __device__ __forceinline__ bool last() const { return t + 1 == t1; }
};

// begin: to the range's first tile, `rem` tiles into its first request.
__device__ __forceinline__ void step_to(const AttnParams &p, int upt, const ReqCache &rc, Walk &w, Cursor &c,
                                        bool begin, int rem) {
  if (!begin && ++c.t < c.t1) return;
  Seg s;
  c.on = walk_next(p, upt, rc, w, s, begin ? rem : -1);
  c.seg = begin ? 0 : c.seg + 1;
  if (!c.on) return;
  c.b = s.b;
  c.h = s.h;
  c.mp = s.mp;
  c.t = c.t0 = s.t0;
  c.t1 = s.t1;
  c.kv_end = s.r.kv_end;
  c.new0 = min(s.r.L, s.r.kv_end);
  c.cut = s.r.kv_end < s.r.L + s.r.n;
}

template <typename T>
__device__ __forceinline__ void swap2(T &a, T &b) {
  const T c = a;
  a = b;
  b = c;
}

__device__ __forceinline__ bool wait_warp(const uint64_t *bar, uint32_t parity, uint32_t *err) {
  return sv::mbar_wait_warp(sv::smem_addr(bar), parity & 1u, err);
}

// ------------------------------------------------------------ main kernel ----

template <typename Q, typename C, int D, bool kPair>
__global__ void __launch_bounds__(Shape<Q, C, D, kPair>::kThreads, 1)
    sv_attn_tc_kernel(const __grid_constant__ TcParams p) {
  using S = Shape<Q, C, D, kPair>;
  extern __shared__ __align__(1024) uint8_t smem[];   // swizzle atoms: 1024 bytes
  __shared__ Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ ReqCache rc[S::kStreams];        // b0: the range's first request
  __shared__ int sh_rem[S::kStreams];         // tiles of it before the range
  __shared__ int sh_scan[S::kWarps + 1];
  __shared__ int seg_bad[S::kStreams][kSegRing];  // holds 1 + a marked segment's number

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t *const sq = smem;
  uint8_t *const ring = sq + S::kQBytes;
  uint8_t *const raw = ring + S::kStages * S::kStageBytes;

  if (sv::smem_addr(smem) & 1023u) {                    // never: the swizzle would not match
    report(p.err, SV_FAULT_TIMEOUT);
    return;
  }
  if (warp == 9) tc_alloc(sv::smem_addr(&tmem_slot), 512);
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      sv::mbar_init(sv::smem_addr(&bars.full[i]), S::kRaw ? S::kHelpers : 1);
      sv::mbar_init(sv::smem_addr(&bars.empty[i]), S::kRaw ? 1 : 1 + S::kHelpers);
      sv::mbar_init(sv::smem_addr(&bars.fixed[i]), S::kHelpers);
    }
    for (int i = 0; i < S::kRawStages; ++i) {
      sv::mbar_init(sv::smem_addr(&bars.rfull[i]), 1);
      sv::mbar_init(sv::smem_addr(&bars.rempty[i]), S::kHelpers);
    }
    for (int s = 0; s < 2; ++s) {
      sv::mbar_init(sv::smem_addr(&bars.s_full[s]), 1);
      sv::mbar_init(sv::smem_addr(&bars.p_ready[s]), 4);
      sv::mbar_init(sv::smem_addr(&bars.p_half[s]), 4);
      sv::mbar_init(sv::smem_addr(&bars.o_done[s]), 1);
      sv::mbar_init(sv::smem_addr(&bars.q_full[s]), 1);
      sv::mbar_init(sv::smem_addr(&bars.q_empty[s]), 1);
    }
    sv::mbar_init(sv::smem_addr(&bars.drain), 1);
    for (int s = 0; s < S::kStreams; ++s) {
      for (int i = 0; i < kSegRing; ++i) seg_bad[s][i] = 0;
      sh_rem[s] = 0;   // of a range without tiles
    }
    sv::fence_mbar_init();
  }
  if (tid == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.vmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.qmap) : "memory");
  }
  const AttnParams &a = p.a;
  const int B = a.bt.B;
  if (warp == 2) {  // addresses only: the values may still be written
    const int64_t at = static_cast<int64_t>(lane) * 32 < B ? lane * 32 : 0;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.bt.seq_lens + at));
    if (a.bt.new_lens) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.bt.new_lens + at));
    if (a.c.max_blocks > 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.c.tables));
  }
  sv::pdl_wait();
  sv::pdl_launch_dependents();

  // This block's ranges of the tile sequence: all requests' tiles are summed
  // and scanned by the block, in one go for up to kThreads requests.
  const int upt = p.TT * S::kTilesPerUnit;
  int total = 0, begin[S::kStreams], count[S::kStreams];
  const bool once = B <= S::kThreads;
  for (int pass = once ? 1 : 0; pass < 2; ++pass) {
    int base = 0;
    for (int c = 0; c < B; c += S::kThreads) {
      uint32_t st = 0;
      const int b = c + tid;
      const int w = b < B ? request(a, upt, b, st).weight : 0;
      if (blockIdx.x == 0 && pass == 1) report(a.bt.status, st);
      int incl = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += v;
      }
      __syncthreads();
      if (lane == 31) sh_scan[warp] = incl;
      __syncthreads();
      int before = base, all = 0;
      for (int k = 0; k < S::kWarps; ++k) {
        if (k < warp) before += sh_scan[k];
        all += sh_scan[k];
      }
      base += all;
      if (once) total = all;
      if (pass == 1) {
        const int excl = before + incl - w, N = min(p.ranges, total);
#pragma unroll
        for (int s = 0; s < S::kStreams; ++s) {
          const int i = static_cast<int>(blockIdx.x + s * gridDim.x);
          begin[s] = i < N ? range_start(i, N, total) : total;
          count[s] = i < N ? range_start(i + 1, N, total) - begin[s] : 0;
          if (w > 0 && begin[s] >= excl && begin[s] < excl + w) {
            rc[s].b0 = b;
            sh_rem[s] = begin[s] - excl;
          }
        }
        if (blockIdx.x == 0 && b < B) p.pre[b] = excl;
      }
    }
    if (pass == 0) total = base;
  }
  if (blockIdx.x == 0 && tid == 0) p.head[0] = total;
  __syncthreads();
#pragma unroll
  for (int s = 0; s < S::kStreams; ++s) {
    const int i = tid - s * kReqCache;
    if (count[s] > 0 && i >= 0 && i < kReqCache && rc[s].b0 + i < B) {
      uint32_t st = 0;
      int L, n;
      lengths(a.bt, rc[s].b0 + i, L, n, st);
      rc[s].len[i] = make_int2(L, n);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  uint32_t *const err = p.err;
  bool ok = true;
  Walk walk[S::kStreams];
#pragma unroll
  for (int s = 0; s < S::kStreams; ++s) walk[s].left = count[s];
  // Steps to the next tile of a stream's range, or (begin) to its first.
  const auto advance = [&](Cursor &c, int s, bool begin = false) {
    step_to(a, upt, rc[s], walk[s], c, begin, sh_rem[s]);
  };

  if (warp < 8) {
    // ------------------------------------------------ softmax warpgroups ----
    const int s = warp >> 2;                 // stream
    const int wq = warp & 3;                 // TMEM lanes 32 wq ..
    const uint32_t lanes = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t col_s = lanes + kColS + 128u * s, col_o = lanes + kColO + 128u * s;
    const int my = wq * 32 + lane;           // row of the 128-row tile
    constexpr int kR = S::kStreams - 1;
    const int rs = s & kR;                   // range of the block
    uint32_t ph_s = 0, ph_o = 0;
    int seg = 0;
    for (; ok; ++seg) {
      Seg next_seg;
      if (!walk_next(a, upt, rc[rs], walk[rs], next_seg, seg == 0 ? sh_rem[rs] : -1)) break;
      const Seg sg = next_seg;
      const Req r = sg.r;
      const int nt = sg.t1 - sg.t0;
      // Tokens and rows of this stream's tile.
      const int tok0 = sg.mp * upt + (kPair ? s * p.TT : 0);
      const int tile_rows = min(max(r.n - tok0, 0), p.TT) * a.G;
      const bool active = wq * 32 < tile_rows;               // warp-uniform
      const int t_row = tok0 + min(my, max(tile_rows - 1, 0)) / a.G;
      const int full_end = min(r.L, r.kv_end);               // every row sees these
      const uint8_t *mrow = a.mask ? a.mask + sg.b * a.msb + static_cast<int64_t>(t_row) * a.bt.T : nullptr;
      float m_ref = -INFINITY, mc = 0.f, l = 0.f;            // mc = m_ref * c, 0 before a key is seen
      for (int j = 0; j < nt; ++j) {
        // Which of the tile's keys the row sees, while S is being computed.
        const int k0 = (sg.t0 + j) * kTile;
        const bool masked = k0 + kTile > full_end;
        uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
        if (masked && active) {
          const int lim = min(r.kv_end, mrow ? r.L : r.L + t_row + 1) - k0;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int n = min(max(lim - 32 * w, 0), 32);
            vis[w] = n == 32 ? ~0u : (1u << n) - 1u;
          }
          if (mrow) {
            // The row's bytes for new tokens [o0, o1), four at a time where
            // rows are whole words; bit c of the tile is new token k0 + c - L.
            const int o0 = max(k0 - r.L, 0), o1 = min(min(r.kv_end, k0 + kTile) - r.L, r.n);
            uint64_t lo = 0, hi = 0;
            const auto put = [&](uint64_t bits, int c) {
              if (c < 0) {
                lo |= bits >> -c;
              } else if (c < 64) {
                lo |= bits << c;
                if (c > 60) hi |= bits >> (64 - c);
              } else {
                hi |= bits << (c - 64);
              }
            };
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
#pragma unroll 4
              for (int o = o0; o < o1; ++o) put(ld8(mrow + o) != 0, o + r.L - k0);
            }
            vis[0] |= static_cast<uint32_t>(lo);
            vis[1] |= static_cast<uint32_t>(lo >> 32);
            vis[2] |= static_cast<uint32_t>(hi);
            vis[3] |= static_cast<uint32_t>(hi >> 32);
          }
        }
        if (!(ok = wait_warp(&bars.s_full[s], ph_s++, err))) break;
        __syncwarp();
        if (active) {
          tc_fence_after();
          if (masked) {  // scores that the row does not see become -inf, in place
#pragma unroll 1
            for (int w = 0; w < 4; ++w) {
              const uint32_t bits = w == 0 ? vis[0] : w == 1 ? vis[1] : w == 2 ? vis[2] : vis[3];
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
          float mt = -INFINITY;
#pragma unroll
          for (int ch = 0; ch < kTile / W; ++ch) {
            load_s(ch);
            float q0 = -INFINITY, q1 = -INFINITY, q2 = -INFINITY, q3 = -INFINITY;
#pragma unroll
            for (int k = 0; k < W; k += 4) {
              q0 = fmaxf(q0, __uint_as_float(x[k]));
              q1 = fmaxf(q1, __uint_as_float(x[k + 1]));
              q2 = fmaxf(q2, __uint_as_float(x[k + 2]));
              q3 = fmaxf(q3, __uint_as_float(x[k + 3]));
            }
            mt = fmaxf(mt, fmaxf(fmaxf(q0, q1), fmaxf(q2, q3)));
          }
          // Raise the reference where the tile's maximum is more than 2^8
          // above it (or nothing was seen before).
          const bool up = mt > m_ref && !((mt - m_ref) * p.c <= 8.f);
          if (__any_sync(kFull, up)) {
            float f = 1.f;
            if (up) {
              const float nmc = mt * p.c;
              f = sv::ex2(m_ref == -INFINITY ? -INFINITY : mc - nmc);
              m_ref = mt;
              mc = nmc;
              l *= f;
            }
            __syncwarp();
            if (j > 0) {
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
          const uint64_t c2 = f2_pack(p.c, p.c), nm2 = f2_pack(-mc, -mc);
          uint64_t l2a = 0, l2b = 0;
          // The last chunk first: it is in registers, and P's columns are the
          // upper half of S, where a chunk's P covers only S already taken.
#pragma unroll
          for (int ch = kTile / W - 1; ch >= 0; --ch) {
            if (ch < kTile / W - 1) load_s(ch);
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
              pk[k >> 1] = pack2<Q>(y0, y1);
            }
            if constexpr (W == 64) tc_st32(col_s + kPOff + ch * (W / 2), pk);
            else tc_st16(col_s + kPOff + ch * (W / 2), pk);
            if (ch * W == kTile / 2) {  // the upper half of P is complete: its products may start
              tc_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.p_half[s]));
              __syncwarp();
            }
          }
          float e0, e1, e2, e3;
          f2_unpack(l2a, e0, e1);
          f2_unpack(l2b, e2, e3);
          l += (e0 + e1) + (e2 + e3);
          tc_wait_st();
          tc_fence_before();
        } else if (lane == 0) {
          sv::mbar_arrive(sv::smem_addr(&bars.p_half[s]));
        }
        __syncwarp();
        if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.p_ready[s]));
      }
      if (!ok || !(ok = wait_warp(&bars.o_done[s], ph_o++, err))) break;
      tc_fence_after();
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
        inv = l == 0.f ? 0.f : 1.f / l;
        if (mine && a.lse && !bad) a.lse[row] = l == 0.f ? -INFINITY : mx * kLn2 + logf(l);
        if (boss)
          p.dirty[(static_cast<int64_t>(sg.b) * a.c.heads + sg.h) * p.MP + sg.mp] = bad ? 1 : 0;
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
      __syncwarp();
      if (active && !bad) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tc_ld32(col_o + c, o);
          tc_wait_ld(o);
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(o[k]);
          if (mine) {
            if (whole) {
#pragma unroll
              for (int k = 0; k < 32; k += 8) {
                uint32_t u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] = pack2<Q>(v[k + 2 * e] * inv, v[k + 2 * e + 1] * inv);
                *reinterpret_cast<uint4 *>(orow + (c + k) * 2) = make_uint4(u[0], u[1], u[2], u[3]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 32; k += 4)
                *reinterpret_cast<float4 *>(slot + (static_cast<size_t>((c + k) >> 2) * p.slot_rows + base_row +
                                                    my) * 4) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            }
          }
          __syncwarp();  // the warp's loads from TMEM are executed together
        }
      }
      tc_fence_before();   // O is read before the next P is announced
    }
  } else if (warp == 8) {
    // --------------------------------------------------------- producer ----
    // Lane i looks up box i of a tile, an elected lane issues all copies.
    const int nb = kTile / p.box;                       // boxes per tile, at most 16
    constexpr int kRing = S::kRaw ? S::kRawStages : S::kStages;
    uint64_t *const fullb = S::kRaw ? bars.rfull : bars.full;
    uint64_t *const emptyb = S::kRaw ? bars.rempty : bars.empty;
    int it = 0, q_issued[2] = {0, 0};
    // A step whose block numbers are on their way: fetched a turn before they
    // are used, for the tables' latency would otherwise bound the loads.
    struct Step {
      Cursor c;
      int id, row;                           // this lane's box; id -2: none
    };
    const auto fetch = [&](const Cursor &c) {
      Step k;
      k.c = c;
      k.id = -2;
      k.row = 0;
      const int pos = c.t * kTile + lane * p.box;
      if (c.on && lane < nb && pos < c.kv_end) {
        const int j = pos / a.c.bs;
        k.row = pos - j * a.c.bs;
        k.id = ld32(a.c.tables + static_cast<size_t>(c.b) * a.c.max_blocks + j);
      }
      return k;
    };
    // A block that is not there marks the segment, whose unit is recomputed;
    // any block is loaded in its place.
    const auto settle = [&](Step &k, int rs) {
      const bool box = lane < nb && k.c.t * kTile + lane * p.box < k.c.kv_end;
      if (box && (k.id < 0 || k.id >= a.c.num_blocks)) {
        report(a.bt.status, k.id == -1 ? SV_KV_MISSING_BLOCK : SV_KV_BAD_BLOCK);
        seg_bad[rs][k.c.seg % kSegRing] = k.c.seg + 1;
        k.id = 0;
      }
      if (!box) k.id = -2;
    };
    // A segment's queries: whole tokens, G heads each, in the swizzled layout.
    const auto load_q = [&](const Cursor &c, int rs) {
      if (lane == 0 && c.cut) report(a.bt.status, SV_KV_TABLE_SHORT);
      if (c.seg > 0 && !wait_warp(&bars.q_empty[rs], (c.seg - 1) & 1, err)) return false;
      const uint32_t bar = sv::smem_addr(&bars.q_full[rs]);
      const uint32_t bytes = S::kTilesPerUnit * S::kHalves * p.qbox * a.G * 128;
      if (elect_one()) {
        sv::mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int i = 0; i < S::kTilesPerUnit; ++i)
#pragma unroll
          for (int hf = 0; hf < S::kHalves; ++hf)
            tma_4d(sv::smem_addr(sq) + (kPair ? i : rs) * S::kStageBytes + hf * (kTile * 128), &p.qmap,
                   hf * 64, c.h * a.G, c.mp * upt + i * p.TT, c.b, bar);
      }
      __syncwarp();
      ++q_issued[rs];
      return true;
    };
    const auto load = [&](const Step &k, bool is_v) {
      const int st = it % kRing;
      if (it >= kRing && !wait_warp(&emptyb[st], (it / kRing) & 1 ? 0u : 1u, err)) return false;
      const uint32_t bar = sv::smem_addr(&fullb[st]);
      const int boxes = __popc(__ballot_sync(kFull, k.id >= 0));   // the first ones
      constexpr int srow = D / SV_KV_GROUP;
      const uint32_t box_bytes = S::kRaw ? p.box * (D + srow) : S::kHalves * p.box * 128;
      const CUtensorMap *map = is_v ? &p.vmap : &p.kmap;
      const uint32_t dst =
          S::kRaw ? sv::smem_addr(raw + st * S::kRawBytes) : sv::smem_addr(ring + st * S::kStageBytes);
      if (elect_one()) sv::mbar_arrive_expect_tx(bar, boxes * box_bytes);
      __syncwarp();
      for (int i = 0; i < boxes; ++i) {
        const int id = __shfl_sync(kFull, k.id, i), row = __shfl_sync(kFull, k.row, i);
        if (elect_one()) {
          if constexpr (S::kRaw) {
            tma_4d(dst + i * p.box * D, map, 0, row, k.c.h, id, bar);
            bulk_1d(dst + S::kRawData + i * p.box * srow,
                    (is_v ? a.c.vs : a.c.ks) + id * a.c.sblock_bytes +
                        (static_cast<int64_t>(k.c.h) * a.c.bs + row) * srow,
                    p.box * srow, bar);
          } else {
#pragma unroll
            for (int hf = 0; hf < S::kHalves; ++hf)
              tma_4d(dst + hf * (kTile * 128) + i * p.box * 128, map, hf * 64, row, k.c.h, id, bar);
          }
        }
        __syncwarp();
      }
      ++it;
      return true;
    };
    if constexpr (kPair) {
      // K0 V0 K1 V1 ...; a segment's queries behind its first tiles.
      Cursor c;
      advance(c, 0, true);
      Step next = fetch(c);
#pragma unroll 1
      while (ok && next.c.on) {
        Step k = next;
        advance(c, 0);
        next = fetch(c);
        settle(k, 0);
#pragma unroll 1
        for (int v = 0; ok && v < 2; ++v) ok = load(k, v);
        if (ok && k.c.first()) ok = load_q(k.c, 0);
      }
    } else {
      // K of both streams, then by turns V and the next K of each.  A new
      // segment's queries follow the other stream's turn: by then the products
      // that read the buffer have most likely ended.  One turn's code serves
      // both streams, whose states change places after it.
      struct State {
        Cursor c;
        Step now, next;
        bool q_due;
      } me, other;
      int s = 0;
      me.q_due = other.q_due = false;
      me.now.c.on = other.now.c.on = false;
#pragma unroll 1
      for (int turn = 0; ok && (turn < 2 || me.now.c.on || other.now.c.on); ++turn) {
        if (turn < 2) {
          advance(me.c, s, true);
          me.next = fetch(me.c);
          me.now.c.on = me.next.c.on;
        } else if (me.now.c.on) {
          ok = load(me.now, true);
        }
        if (ok && me.now.c.on) {
          me.now = me.next;
          if (me.now.c.on) {
            advance(me.c, s);
            me.next = fetch(me.c);
            settle(me.now, s);
            me.q_due = me.now.c.first();
            ok = load(me.now, false);
          }
        }
        if (ok && other.q_due) {
          ok = load_q(other.now.c, 1 - s);
          other.q_due = false;
        }
        if (ok && me.q_due && (turn < 2 || !other.now.c.on)) {
          ok = load_q(me.now.c, s);
          me.q_due = false;
        }
        swap2(me, other);
        s = 1 - s;
      }
    }
    if (!ok) {  // every copy in flight lands before the block ends
      for (int k = max(0, it - kRing); k < it; ++k) wait_warp(&fullb[k % kRing], (k / kRing) & 1, err);
#pragma unroll
      for (int s = 0; s < S::kStreams; ++s)
        if (q_issued[s] > 0) wait_warp(&bars.q_full[s], (q_issued[s] - 1) & 1, err);
    }
  } else if (warp == 9) {
    // --------------------------------------------------------------- MMA ----
    const uint32_t kQK = mma_desc<Q>(kTile, false) | (p.negate ? kNegateA : 0u);
    constexpr uint32_t kPV = mma_desc<Q>(D, true);
    const uint64_t q_desc = smem_desc(sv::smem_addr(sq), 16), k_desc = smem_desc(sv::smem_addr(ring), 16);
    const uint64_t v_desc = smem_desc(sv::smem_addr(ring), kTile * 128);
    int it = 0;                    // stages taken, in load order
    uint32_t ph_p = 0, fix = 0;    // parities: of P per stream, of its repairs per stage
    const auto take = [&](const Cursor &c, bool is_v) {
      const int st = it % S::kStages;
      bool good = wait_warp(&bars.full[st], (it / S::kStages) & 1, err);
      if (!S::kRaw && good && is_v && (c.t + 1) * kTile > c.new0) {
        good = wait_warp(&bars.fixed[st], (fix >> st) & 1u, err);
        fix ^= 1u << st;
      }
      tc_fence_after();
      return good;
    };
    auto release = [&]() {
      if (elect_one()) tc_commit(sv::smem_addr(&bars.empty[it % S::kStages]));
      ++it;
    };
    auto qk = [&](int s) {
      const uint64_t qd = q_desc + s * (S::kStageBytes >> 4);
      const uint64_t kd = k_desc + (it % S::kStages) * (S::kStageBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4;
          tc_mma_ss(tmem + kColS + 128u * s, qd + off, kd + off, kQK, k > 0);
        }
      }
      __syncwarp();
    };
    // Keys 64 .. 127 of the tile first: their P is ready first.
    auto pv = [&](int s, bool first) {
      const uint64_t vd = v_desc + (it % S::kStages) * (S::kStageBytes >> 4);
#pragma unroll
      for (int half = 1; half >= 0; --half) {
        if (half == 0) {
          if (!wait_warp(&bars.p_ready[s], ph_p >> s, err)) return false;
          ph_p ^= 1u << s;
        }
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 4 * half; k < 4 * half + 4; ++k)
            tc_mma_ts(tmem + kColO + 128u * s, tmem + kColS + 128u * s + kPOff + 8u * k,
                      vd + k * (2048 >> 4), kPV, !(first && k == 4));
        }
        __syncwarp();
      }
      return true;
    };
    auto commit = [&](uint64_t *bar) {
      if (elect_one()) tc_commit(sv::smem_addr(bar));
    };
    if constexpr (kPair) {
      // S of both streams for step c, whose K is stage `it`.
      const auto products = [&](const Cursor &c, int s) {
        if (s == 0) {
          if (c.first() && !wait_warp(&bars.q_full[0], c.seg, err)) return false;
          if (!take(c, false)) return false;
        }
        qk(s);
        commit(&bars.s_full[s]);
        if (s == 1) {
          release();
          if (c.last()) commit(&bars.q_empty[0]);
        }
        return true;
      };
      // One turn is one stream's P V and its next Q K^T; the first two turns
      // have only the latter.  V's stage is `it`, the next K's the one after.
      Cursor c, n;
      advance(n, 0, true);
      c.on = false;
#pragma unroll 1
      for (int turn = 0; ok && (n.on || c.on); ++turn) {
        const int s = turn & 1;
        if (turn >= 2) {
          ok = wait_warp(&bars.p_half[s], ph_p >> s, err) && (s == 1 || take(c, true)) && pv(s, c.first());
          if (!ok) break;
          if (s == 1) release();                     // V
          if (c.last()) commit(&bars.o_done[s]);
          if (n.on) {
            if (s == 0) ++it;
            ok = products(n, s);
            if (s == 0) --it;
          }
        } else {
          ok = products(n, s);
        }
        if (s == 1) {                                // both streams have taken the step
          c = n;
          if (n.on) advance(n, 0);
        }
      }
    } else {
      Cursor me, other;
      int s = 0;
      me.on = other.on = false;
#pragma unroll 1
      for (int turn = 0; ok && (turn < 2 || me.on || other.on); ++turn) {
        if (turn < 2) {
          advance(me, s, true);
        } else if (me.on) {
          ok = wait_warp(&bars.p_half[s], ph_p >> s, err) && take(me, true) && pv(s, me.first());
          release();
          if (me.last()) commit(&bars.o_done[s]);
          advance(me, s);
        }
        if (ok && me.on) {
          ok = (!me.first() || wait_warp(&bars.q_full[s], me.seg, err)) && take(me, false);
          if (ok) {
            qk(s);
            commit(&bars.s_full[s]);
            release();
            if (me.last()) commit(&bars.q_empty[s]);
          }
        }
        swap2(me, other);
        s = 1 - s;
      }
    }
    if (!ok) {  // issued products end before TMEM is freed
      if (elect_one()) tc_commit(sv::smem_addr(&bars.drain));
      __syncwarp();
      wait_warp(&bars.drain, 0, err);
    }
  } else {
    // ------------------------------------------------------------ helpers ----
    const int ht = tid - 320;                           // helper thread
    constexpr int kHT = S::kHelpers * 32;
    int it = 0, rit = 0;
    uint32_t found = 0;
    // Not kRaw: V tiles that reach past the committed tokens, in place.
    const auto repair = [&](const Cursor &c) {
      const int st = it % S::kStages;
      uint8_t *base = ring + st * S::kStageBytes;
      const int k0 = c.t * kTile, r0 = max(c.new0 - k0, 0), r1 = c.kv_end - k0;  // new rows [r0, r1)
      constexpr int kCh = S::kHalves * 8;
      for (int i = ht + r0 * kCh; i < kTile * kCh; i += kHT) {
        const int row = i / kCh, ch = i % kCh;
        uint4 *w = reinterpret_cast<uint4 *>(base + (ch >> 3) * (kTile * 128) + row * 128 + (ch & 7) * 16);
        if (row >= r1) {
          *w = make_uint4(0, 0, 0, 0);
        } else {
          const uint4 v = *w;
          if (odd16<Q>(v.x) || odd16<Q>(v.y) || odd16<Q>(v.z) || odd16<Q>(v.w)) found = 1;
        }
      }
    };
    // kRaw: 16 codes at a time, widened into the swizzled layout.
    const auto widen = [&](const Cursor &c, bool is_v) {
      const int st = it % S::kStages, rs = rit % (S::kRaw ? S::kRawStages : 1);
      if (!wait_warp(&bars.rfull[rs], (rit / (S::kRaw ? S::kRawStages : 1)) & 1, err)) return false;
      if (it >= S::kStages && !wait_warp(&bars.empty[st], (it / S::kStages) & 1 ? 0u : 1u, err)) return false;
      const uint8_t *src = raw + rs * S::kRawBytes;
      const uint8_t *sc = src + S::kRawData;
      uint8_t *dst = ring + st * S::kStageBytes;
      constexpr int kCh = D / 16;                       // 16-code chunks per row
      const int k0 = c.t * kTile, r0 = max(c.new0 - k0, 0), r1 = is_v ? c.kv_end - k0 : kTile;
      const bool look = is_v && k0 + kTile > c.new0;
#pragma unroll 4
      for (int i = ht; i < kTile * kCh; i += kHT) {
        const int row = i / kCh, ch = i % kCh;
        const uint4 w = *reinterpret_cast<const uint4 *>(src + i * 16);
        const float m = scale_value(sc[row * (D / SV_KV_GROUP) + (ch >> 1)]);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
              static_cast<__nv_fp8x2_storage_t>(u[k >> 1] >> (16 * (k & 1))), __NV_E4M3);
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
          o[k] = pack2<Q>(f.x * m, f.y * m);
        }
        if (look && row >= r0) {
          if (row >= r1) {
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = 0;
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (odd16<Q>(o[k])) found = 1;
          }
        }
        // Odd chunk pairs are written in the other order: the two 64-column
        // halves of a row lie in the same banks.
        uint8_t *d = dst + (ch >> 2) * (kTile * 128) + row * 128;
        const int c0 = (ch & 3) * 2, sw = row & 7;
        const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
        const bool swap = ch >> 2;
        *reinterpret_cast<uint4 *>(d + (((c0 + (swap ? 1 : 0)) ^ sw) << 4)) = swap ? hi : lo;
        *reinterpret_cast<uint4 *>(d + (((c0 + (swap ? 0 : 1)) ^ sw) << 4)) = swap ? lo : hi;
      }
      return true;
    };
    // One stage of the load order.
    const auto stage = [&](const Cursor &c, bool is_v, int rs) {
      if constexpr (S::kRaw) {
        if (!widen(c, is_v)) return false;
        if (found) seg_bad[rs][c.seg % kSegRing] = c.seg + 1;
        found = 0;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          sv::mbar_arrive(sv::smem_addr(&bars.full[it % S::kStages]));
          sv::mbar_arrive(sv::smem_addr(&bars.rempty[rit % (S::kRaw ? S::kRawStages : 1)]));
        }
        ++rit;
      } else {
        // Every stage is looked at, also those that need nothing: a warp that
        // ran ahead would take an older phase of the barrier for its own, and
        // one that fell behind would miss a phase.
        const int st = it % S::kStages;
        if (!wait_warp(&bars.full[st], (it / S::kStages) & 1, err)) return false;
        const bool fix = is_v && (c.t + 1) * kTile > c.new0;
        if (fix) {
          repair(c);
          if (found) seg_bad[rs][c.seg % kSegRing] = c.seg + 1;
          found = 0;
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          if (fix) sv::mbar_arrive(sv::smem_addr(&bars.fixed[st]));
          sv::mbar_arrive(sv::smem_addr(&bars.empty[st]));
        }
      }
      ++it;
      return true;
    };
    if constexpr (kPair) {
      Cursor c;
      advance(c, 0, true);
#pragma unroll 1
      for (int v = 0; ok && c.on; v ^= 1) {
        ok = stage(c, v, 0);
        if (v) advance(c, 0);
      }
    } else {
      // K of both streams, then by turns V and the next K of each.
      Cursor me, other;
      int s = 0;
      me.on = other.on = false;
#pragma unroll 1
      for (int turn = 0; ok && (turn < 4 || me.on || other.on); ++turn) {
        const bool v = !(turn & 1);                  // turns 0 and 2 begin a stream instead
        if (turn < 4 && v) {
          advance(me, s, true);
        } else if (me.on) {
          ok = stage(me, v, s);
          if (v) advance(me, s);
        }
        if (!v) {
          swap2(me, other);
          s = 1 - s;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tc_dealloc(tmem, 512);
}

// ---------------------------------------------------------- second kernel ----

constexpr int kJoinThreads = 256;

// Joins the partial results of units that ranges cut, and recomputes marked
// ones.  Grid: (units, parts of a unit's rows x D / 4 columns).
template <typename Q, typename C, int D, bool kPair>
__global__ void __launch_bounds__(kJoinThreads) sv_attn_join_kernel(const __grid_constant__ TcParams p) {
  __shared__ float qs[kJoinThreads / 32][D];
  const AttnParams &a = p.a;
  const int per_b = a.c.heads * p.MP;
  const int b = blockIdx.x / per_b, rem = blockIdx.x - b * per_b, h = rem / p.MP, mp = rem - h * p.MP;
  sv::pdl_wait();
  sv::pdl_launch_dependents();
  uint32_t st = 0;
  const int upt = p.TT * (kPair ? 2 : 1);
  const Req r = request(a, upt, b, st);
  if (mp >= r.mp) return;
  const int tok0 = mp * upt, rows = min(upt, r.n - tok0) * a.G;
  const int total = ld32(p.head), start = ld32(p.pre + b) + (h * r.mp + mp) * r.kt;
  const int N = min(p.ranges, total);
  const int c0 = range_of(start, N, total), c1 = range_of(start + r.kt - 1, N, total);
  const int late = range_start(c0, N, total) == start ? 0 : 1;  // not the first segment of range c0
  auto slot_of = [&](int c) {
    return p.slots + (static_cast<size_t>(c) * 2 + (c == c0 ? late : 0)) * p.slot_floats;
  };
  int bad = 0;
  if (c0 == c1) {
    if (!ld8(p.dirty + (static_cast<int64_t>(b) * a.c.heads + h) * p.MP + mp)) return;
    bad = 1;
  } else {
    for (int c = c0; c <= c1; ++c)
      bad |= ld32(reinterpret_cast<const int32_t *>(slot_of(c)) + (D + 2) * p.slot_rows);
  }
  const auto out_row = [&](int row) {
    const int t = tok0 + row / a.G, g = row % a.G;
    return (static_cast<int64_t>(b) * a.bt.T + t) * a.Hq + h * a.G + g;
  };
  if (bad) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int row = blockIdx.y * (kJoinThreads / 32) + warp; row < rows;
         row += gridDim.y * (kJoinThreads / 32)) {
      const int t = tok0 + row / a.G, g = row % a.G;
      const uint8_t *q = a.q + b * a.qsb + t * a.qst + static_cast<int64_t>(h * a.G + g) * a.qsh;
      __syncwarp();
      for (int d = lane; d < D; d += 32) {
        const uint16_t w = static_cast<uint16_t>(ld16(q + 2 * d));
        qs[warp][d] = load1<Q>(&w) * a.scale_log2;
      }
      __syncwarp();
      RowState<D> rs;
      rs.m = -INFINITY;
      rs.l = 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) rs.o[e] = 0.f;
      uint32_t none = 0;
      attend<C, D>(a, b, t, h, r.L, r.n, r.L + r.n, qs[warp], 0, 32, lane, rs, none);
      store_row<Q, D>(a, out_row(row), lane, rs);
    }
    return;
  }
  const int i = blockIdx.y * kJoinThreads + threadIdx.x;
  if (i >= rows * (D / 4)) return;
  const int row = i % rows, d4 = i / rows;
  // Rows of the second tile start at row 128 of a slot.
  const int tile_rows = p.TT * a.G, srow = row < tile_rows ? row : kTile + row - tile_rows;
  float m = -INFINITY;
  for (int c = c0; c <= c1; ++c) m = fmaxf(m, __ldcg(slot_of(c) + D * p.slot_rows + srow));
  const float mb = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const float *s = slot_of(c);
    const float f = sv::ex2(__ldcg(s + D * p.slot_rows + srow) - mb);
    l += __ldcg(s + (D + 1) * p.slot_rows + srow) * f;
    const float4 v = __ldcg(reinterpret_cast<const float4 *>(s) + static_cast<size_t>(d4) * p.slot_rows + srow);
    o.x += v.x * f;
    o.y += v.y * f;
    o.z += v.z * f;
    o.w += v.w * f;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t orow = out_row(row);
  *reinterpret_cast<uint2 *>(a.out + orow * (D * 2) + d4 * 8) =
      make_uint2(pack2<Q>(o.x * inv, o.y * inv), pack2<Q>(o.z * inv, o.w * inv));
  if (a.lse && d4 == 0) a.lse[orow] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

}  // namespace svp
