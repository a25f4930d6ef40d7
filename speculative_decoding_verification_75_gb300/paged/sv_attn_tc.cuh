// sv_attn_tc.cuh -- tree attention over the paged cache on the tensor cores
// (tcgen05), for head dimensions 64 and 128.
//
// Rows.  All n new tokens and the G query heads that share a KV head form one
// matrix of n * G rows, row r = token r / G, head r % G, so that a key is read
// once for all of them; a tile takes as many whole tokens as fit 128 rows.  S = Q K^T and O = P V run as M = 128 row tiles with
// 128 keys a step; S and O live in tensor memory (TMEM: lane = row, one
// thread per row), P overwrites half of its S as the 16-bit A operand.
//
// Two streams of such steps alternate, each with a softmax warpgroup of its
// own, so that the tensor cores work on one while the other takes
// exponentials: with at most 128 rows both streams work on the same rows,
// one on the even and one on the odd key tiles of the range, and are joined
// in the end (kPair = false); with more, each has 128 rows of its own and
// both use every key tile (kPair = true).
//
// Work.  The key tiles of all units (request, KV head, row tiles) form one
// sequence that is cut into equal ranges, one per thread block (one block per
// SM): ragged lengths are balanced to within a tile.  A unit cut by a range's
// end leaves partial results (unnormalised O, row maximum and sum) in the
// workspace, joined by the second kernel in range order, so results do not
// depend on timing.  The lengths are read on the device; the host never waits.
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
  int32_t *head;       // [0] tiles per range
  int32_t *pre;        // [B + 1] tiles before each request
  uint8_t *dirty;      // [B * heads * MP] units to recompute (whole ranges)
  float *slots;        // [grid * 2] partial results
  int slot_rows;       // rows of a slot
  int slot_floats;
  int MP;              // row-tile groups per (request, head), at most
  int box;             // rows of a TMA box of the cache
  int TT;              // tokens of a row tile: its rows are TT * G <= 128
  int qbox;            // tokens of a TMA box of the queries
  float c;             // |scale| * log2(e), at least 1e-30
  int negate;          // scale < 0: the signs of S are flipped
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

__device__ __forceinline__ void named_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Shared-memory operand descriptor: 128-byte swizzle, 8-row groups 1024 bytes
// apart; `lead`: distance of the next 64 elements along the contiguous
// dimension where the operand is not K-major.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

// Instruction descriptor: fp32 accumulators, M = 128; b_mn: B's N runs
// contiguously.
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
  // Q: one tile per stream, or one for both and room for the next segment's.
  static constexpr int kQBufs = kPair ? 1 : 2;
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
  uint64_t s_full[2], p_ready[2], o_done[2], q_full[2], q_empty[2], drain;
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

  __device__ __forceinline__ Req fetch(const AttnParams &p, int upt, const ReqCache &rc) const {
    if (b - rc.b0 < kReqCache) {
      const int2 v = rc.len[b - rc.b0];
      return make_request(p, upt, v.x, v.y);
    }
    uint32_t st = 0;
    return request(p, upt, b, st);
  }
  __device__ __forceinline__ void start(const AttnParams &p, int upt, const ReqCache &rc, int rem,
                                        int count) {
    left = count;
    if (left <= 0) return;
    b = rc.b0;
    r = fetch(p, upt, rc);
    unit = rem / r.kt;
    tile = rem - unit * r.kt;
  }
  __device__ __forceinline__ bool next(const AttnParams &p, int upt, const ReqCache &rc, Seg &s) {
    if (left <= 0) return false;
    s.b = b;
    s.r = r;
    s.unit = unit;
    s.h = unit / r.mp;
    s.mp = unit - s.h * r.mp;
    s.t0 = tile;
    s.t1 = min(r.kt, tile + left);
    left -= s.t1 - s.t0;
    tile = s.t1;
    if (tile == r.kt) {
      tile = 0;
      if (++unit == p.c.heads * r.mp) {
        unit = 0;
        if (left > 0) {
          do {
            ++b;
            r = fetch(p, upt, rc);
          } while (r.weight == 0);
        }
      }
    }
    return true;
  }
};

// Steps of a segment and stream: pair: every tile for both streams;
// otherwise tile i for stream i & 1.
template <bool kPair>
__device__ __forceinline__ int steps_of(int nt, int s) {
  return kPair ? nt : (nt + 1 - s) >> 1;
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
  __shared__ ReqCache rc;                     // rc.b0: the range's first request
  __shared__ int sh_rem;                      // tiles of it before the range
  __shared__ int sh_scan[S::kWarps + 1];
  __shared__ int seg_bad[kSegRing];
  __shared__ int failed;                      // a softmax warp's wait gave up
  __shared__ float sh_m[2][kTile], sh_l[2][kTile];

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
      sv::mbar_init(sv::smem_addr(&bars.o_done[s]), 1);
      sv::mbar_init(sv::smem_addr(&bars.q_full[s]), 1);
      sv::mbar_init(sv::smem_addr(&bars.q_empty[s]), 1);
    }
    sv::mbar_init(sv::smem_addr(&bars.drain), 1);
    for (int i = 0; i < kSegRing; ++i) seg_bad[i] = 0;
    failed = 0;
    sv::fence_mbar_init();
  }
  if (tid == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.vmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&p.qmap) : "memory");
  }
  const AttnParams &a = p.a;
  const int B = a.bt.B;
  sv::pdl_wait();
  sv::pdl_launch_dependents();

  // This block's range of the tile sequence: all requests' tiles are summed
  // and scanned by the block, in one go for up to kThreads requests.
  const int upt = p.TT * S::kTilesPerUnit;
  int total = 0, quota = 0, begin = 0, count = 0;
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
        quota = (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
        begin = static_cast<int>(min(static_cast<int64_t>(blockIdx.x) * quota, static_cast<int64_t>(total)));
        const int excl = before + incl - w;
        if (w > 0 && begin >= excl && begin < excl + w) {
          rc.b0 = b;
          sh_rem = begin - excl;
        }
        if (blockIdx.x == 0 && b < B) p.pre[b] = excl;
      }
    }
    if (pass == 0) total = base;
  }
  count = min(quota, total - begin);
  if (blockIdx.x == 0 && tid == 0) p.head[0] = quota;
  __syncthreads();
  if (count > 0 && tid < kReqCache && rc.b0 + tid < B) {
    uint32_t st = 0;
    int L, n;
    lengths(a.bt, rc.b0 + tid, L, n, st);
    rc.len[tid] = make_int2(L, n);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  Walk walk;
  walk.start(a, upt, rc, count > 0 ? sh_rem : 0, count);
  uint32_t *const err = p.err;
  Seg sg;
  bool ok = true;

  if (warp < 8) {
    // ------------------------------------------------ softmax warpgroups ----
    const int s = warp >> 2;                 // stream
    const int wq = warp & 3;                 // TMEM lanes 32 wq ..
    const uint32_t lanes = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t col_s = lanes + kColS + 128u * s, col_o = lanes + kColO + 128u * s;
    const int my = wq * 32 + lane;           // row of the 128-row tile
    uint32_t ph_s = 0, ph_o = 0;
    int seg = 0;
    for (; ok && walk.next(a, upt, rc, sg); ++seg) {
      const Req &r = sg.r;
      const int nt = sg.t1 - sg.t0, nsteps = steps_of<kPair>(nt, s);
      // Tokens and rows of this stream's tile.
      const int tok0 = sg.mp * upt + (kPair ? s * p.TT : 0);
      const int tile_rows = min(max(r.n - tok0, 0), p.TT) * a.G;
      const bool active = wq * 32 < tile_rows;               // warp-uniform
      const int t_row = tok0 + min(my, max(tile_rows - 1, 0)) / a.G;
      const int full_end = min(r.L, r.kv_end);               // every row sees these
      const uint8_t *mrow = a.mask ? a.mask + sg.b * a.msb + static_cast<int64_t>(t_row) * a.bt.T : nullptr;
      float m_ref = -INFINITY, mc = 0.f, l = 0.f;            // mc = m_ref * c, 0 before a key is seen
      for (int j = 0; j < nsteps; ++j) {
        // Which of the tile's keys the row sees, while S is being computed.
        const int k0 = (sg.t0 + (kPair ? j : 2 * j + s)) * kTile;
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
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int c0 = max(max(r.L - k0, 0), 32 * w), c1 = min(min(r.kv_end - k0, kTile), 32 * w + 32);
#pragma unroll 8
              for (int c = c0; c < c1; ++c)
                vis[w] |= (ld8(mrow + (k0 + c - r.L)) ? 1u : 0u) << (c & 31);
            }
          }
        }
        if (!(ok = wait_warp(&bars.s_full[s], ph_s++, err))) break;
        if (active) {
          tc_fence_after();
          // A chunk of S; the last one of the first pass stays in registers.
          constexpr int W = S::kChunk;
          uint32_t x[W];
          const auto load_s = [&](int ch) {
#pragma unroll
            for (int k = 0; k < W; k += 32) tc_ld32(col_s + ch * W + k, x + k);
            tc_wait_ld(x);
            if (p.negate) {
#pragma unroll
              for (int k = 0; k < W; ++k) x[k] ^= 0x80000000u;
            }
            if (masked) {
#pragma unroll
              for (int k = 0; k < W; ++k)
                if (!((vis[(ch * W + k) >> 5] >> (k & 31)) & 1u)) x[k] = 0xff800000u;
            }
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
            if (j > 0) {
#pragma unroll
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
          }
          float e0, e1, e2, e3;
          f2_unpack(l2a, e0, e1);
          f2_unpack(l2b, e2, e3);
          l += (e0 + e1) + (e2 + e3);
          tc_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) sv::mbar_arrive(sv::smem_addr(&bars.p_ready[s]));
      }
      if (ok && nsteps > 0) ok = wait_warp(&bars.o_done[s], ph_o++, err);
      // Both streams' sums are final: join and store.
      if (!ok) failed = 1;
      sh_m[s][my] = l == 0.f ? -INFINITY : mc;
      sh_l[s][my] = l;
      tc_fence_before();
      named_bar(1, 256);
      tc_fence_after();
      const bool bad = seg_bad[seg % kSegRing] != 0;
      ok = failed == 0;   // the same for both warpgroups: they leave together
      const bool whole = sg.t0 == 0 && sg.t1 == r.kt;
      float f0 = 1.f, f1 = 0.f, lsum = l, mx = sh_m[s][my];
      if (!kPair) {
        const float a0 = sh_m[0][my], a1 = sh_m[1][my];
        mx = fmaxf(a0, a1);
        const float mb = mx == -INFINITY ? 0.f : mx;
        f0 = sv::ex2(a0 - mb);
        f1 = sv::ex2(a1 - mb);
        lsum = sh_l[0][my] * f0 + sh_l[1][my] * f1;
      }
      const int base_row = kPair ? s * kTile : 0;            // of the slot
      const bool two = !kPair && nt > 1;
      const bool mine = my < tile_rows;
      float *slot = nullptr;
      uint8_t *orow = nullptr;
      float inv = 1.f;
      if (whole) {
        const int t = tok0 + my / a.G, g = my % a.G;
        const int64_t row = (static_cast<int64_t>(sg.b) * a.bt.T + t) * a.Hq + sg.h * a.G + g;
        orow = a.out + row * (D * 2);
        inv = lsum == 0.f ? 0.f : 1.f / lsum;
        if (mine && a.lse && !bad && (kPair || s == 0))
          a.lse[row] = lsum == 0.f ? -INFINITY : mx * kLn2 + logf(lsum);
        if (tid == 0)
          p.dirty[(static_cast<int64_t>(sg.b) * a.c.heads + sg.h) * p.MP + sg.mp] = bad ? 1 : 0;
      } else {
        // Slot 0 of the range where the segment starts it, else slot 1.
        slot = p.slots + (static_cast<size_t>(blockIdx.x) * 2 + (seg == 0 ? 0 : 1)) * p.slot_floats;
        if (mine && (kPair || s == 0)) {
          slot[D * p.slot_rows + base_row + my] = mx;
          slot[(D + 1) * p.slot_rows + base_row + my] = lsum;
        }
        if (tid == 0) reinterpret_cast<int *>(slot)[(D + 2) * p.slot_rows] = bad ? 1 : 0;
      }
      if (active && ok && !bad) {
        // kPair: a warpgroup stores its own rows; otherwise each takes half
        // of the columns of all rows.
        constexpr int kCols = kPair ? D : D / 2;
        const int d0 = kPair ? 0 : s * kCols;
        const uint32_t o0 = lanes + kColO + (kPair ? 128u * s : 0u) + d0, o1 = lanes + kColO + 128u + d0;
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          uint32_t o[32];
          tc_ld32(o0 + c, o);
          tc_wait_ld(o);
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(o[k]);
          if (two) {
            uint32_t q[32];
            tc_ld32(o1 + c, q);
            tc_wait_ld(q);
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = v[k] * f0 + __uint_as_float(q[k]) * f1;
          }
          if (!mine) continue;
          if (whole) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              uint32_t u[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                u[e] = pack2<Q>(v[k + 2 * e] * inv, v[k + 2 * e + 1] * inv);
              *reinterpret_cast<uint4 *>(orow + (d0 + c + k) * 2) = make_uint4(u[0], u[1], u[2], u[3]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4 *>(slot + (static_cast<size_t>((d0 + c + k) >> 2) * p.slot_rows +
                                                  base_row + my) * 4) =
                  make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
          }
        }
      }
      tc_fence_before();
      named_bar(1, 256);
      tc_fence_after();
      if (tid == 0) seg_bad[seg % kSegRing] = 0;
    }
  } else if (warp == 8) {
    // --------------------------------------------------------- producer ----
    const int nb = kTile / p.box;                       // boxes per tile (and half)
    const int half = S::kRaw ? 0 : lane / nb, bi = S::kRaw ? lane : lane - half * nb;
    const bool lane_on = S::kRaw ? lane < nb : half < S::kHalves;
    constexpr int kRing = S::kRaw ? S::kRawStages : S::kStages;
    uint64_t *const fullb = S::kRaw ? bars.rfull : bars.full;
    uint64_t *const emptyb = S::kRaw ? bars.rempty : bars.empty;
    int it = 0, seg = 0, q_issued = 0;
    // Block of this lane's box in a tile; -2 behind the last token.  A block
    // that is not there marks the segment, whose unit is recomputed; any block
    // is loaded in its place.
    auto lookup = [&](const Seg &g, int tile) {
      const int pos = tile * kTile + bi * p.box;
      if (!lane_on || tile >= g.t1 || pos >= g.r.kv_end) return -2;
      int id = ld32(a.c.tables + static_cast<size_t>(g.b) * a.c.max_blocks + pos / a.c.bs);
      if (id < 0 || id >= a.c.num_blocks) {
        report(a.bt.status, id == -1 ? SV_KV_MISSING_BLOCK : SV_KV_BAD_BLOCK);
        seg_bad[seg % kSegRing] = 1;
        id = 0;
      }
      return id;
    };
    // A segment's queries: whole tokens, G heads each, in the swizzled layout.
    auto load_q = [&](const Seg &g) {
      const int qb = seg % S::kQBufs, use = seg / S::kQBufs;
      if (use > 0 && !wait_warp(&bars.q_empty[qb], (use - 1) & 1, err)) return false;
      const uint32_t bar = sv::smem_addr(&bars.q_full[qb]);
      const uint32_t bytes = S::kTilesPerUnit * S::kHalves * p.qbox * a.G * 128;
      if (elect_one()) {
        sv::mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int i = 0; i < S::kTilesPerUnit; ++i)
#pragma unroll
          for (int hf = 0; hf < S::kHalves; ++hf)
            tma_4d(sv::smem_addr(sq) + (kPair ? i : qb) * S::kStageBytes + hf * (kTile * 128), &p.qmap,
                   hf * 64, g.h * a.G, g.mp * upt + i * p.TT, g.b, bar);
      }
      __syncwarp();
      ++q_issued;
      return true;
    };
    auto load = [&](const Seg &g, int tile, int id, bool is_v) {
      const int st = it % kRing;
      if (it >= kRing && !wait_warp(&emptyb[st], (it / kRing) & 1 ? 0u : 1u, err)) return false;
      const uint32_t bar = sv::smem_addr(&fullb[st]);
      const unsigned on = __ballot_sync(kFull, id >= 0);
      const uint32_t box_bytes = S::kRaw ? p.box * (D + D / SV_KV_GROUP) : p.box * 128;
      if (lane == 0) sv::mbar_arrive_expect_tx(bar, __popc(on) * box_bytes);
      __syncwarp();
      if (id >= 0) {
        const int row = (tile * kTile + bi * p.box) % a.c.bs;
        const CUtensorMap *map = is_v ? &p.vmap : &p.kmap;
        if constexpr (S::kRaw) {
          const uint32_t dst = sv::smem_addr(raw + st * S::kRawBytes);
          tma_4d(dst + bi * p.box * D, map, 0, row, g.h, id, bar);
          constexpr int srow = D / SV_KV_GROUP;
          bulk_1d(dst + S::kRawData + bi * p.box * srow,
                  (is_v ? a.c.vs : a.c.ks) + id * a.c.sblock_bytes +
                      (static_cast<int64_t>(g.h) * a.c.bs + row) * srow,
                  p.box * srow, bar);
        } else {
          tma_4d(sv::smem_addr(ring + st * S::kStageBytes) + half * (kTile * 128) + bi * p.box * 128,
                 map, half * 64, row, g.h, id, bar);
        }
      }
      ++it;
      return true;
    };
    for (; ok && walk.next(a, upt, rc, sg); ++seg) {
      if (lane == 0 && sg.r.kv_end < sg.r.L + sg.r.n) report(a.bt.status, SV_KV_TABLE_SHORT);
      int id = lookup(sg, sg.t0), before = -2;
      if (!kPair) ok = load_q(sg);
      for (int t = sg.t0; ok && t < sg.t1; ++t) {
        const int next = lookup(sg, t + 1);
        ok = load(sg, t, id, false);
        if (kPair) {
          ok = ok && load(sg, t, id, true);
          // One buffer: the first tiles are on their way before it is free.
          if (t == sg.t0) ok = ok && load_q(sg);
        } else {
          if (t > sg.t0) ok = ok && load(sg, t - 1, before, true);
          before = id;
        }
        id = next;
      }
      if (!kPair) ok = ok && load(sg, sg.t1 - 1, before, true);
    }
    if (!ok) {  // every copy in flight lands before the block ends
      for (int k = max(0, it - kRing); k < it; ++k) wait_warp(&fullb[k % kRing], (k / kRing) & 1, err);
      for (int k = max(0, seg - S::kQBufs); k <= seg; ++k)
        if (q_issued > k) wait_warp(&bars.q_full[k % S::kQBufs], (k / S::kQBufs) & 1, err);
    }
  } else if (warp == 9) {
    // --------------------------------------------------------------- MMA ----
    constexpr uint32_t kQK = mma_desc<Q>(kTile, false), kPV = mma_desc<Q>(D, true);
    const uint64_t q_desc = smem_desc(sv::smem_addr(sq), 16), k_desc = smem_desc(sv::smem_addr(ring), 16);
    const uint64_t v_desc = smem_desc(sv::smem_addr(ring), kTile * 128);
    int it = 0, seg = 0;           // stages taken, in load order
    uint32_t ph_p[2] = {0, 0}, fix = 0;  // fix: per stage, parity of its repairs
    auto take = [&](int k0, int full_end, bool is_v) {
      const int st = it % S::kStages;
      bool good = wait_warp(&bars.full[st], (it / S::kStages) & 1, err);
      if (!S::kRaw && good && is_v && k0 + kTile > full_end) {
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
      const uint64_t qd = q_desc + (kPair ? s : seg % S::kQBufs) * (S::kStageBytes >> 4);
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
    auto pv = [&](int s, bool first) {
      const uint64_t vd = v_desc + (it % S::kStages) * (S::kStageBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          tc_mma_ts(tmem + kColO + 128u * s, tmem + kColS + 128u * s + kPOff + 8u * k,
                    vd + k * (2048 >> 4), kPV, !first || k > 0);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t *bar) {
      if (elect_one()) tc_commit(sv::smem_addr(bar));
    };
    for (; ok && walk.next(a, upt, rc, sg); ++seg) {
      const int nt = sg.t1 - sg.t0, full_end = min(sg.r.L, sg.r.kv_end);
      const auto key0 = [&](int t) { return (sg.t0 + t) * kTile; };
      uint64_t *const q_free = &bars.q_empty[seg % S::kQBufs];
      if (!(ok = wait_warp(&bars.q_full[seg % S::kQBufs], seg / S::kQBufs, err))) break;
      tc_fence_after();
      if (kPair) {
        // Stages in order K0 V0 K1 V1 ...
        if (!(ok = take(key0(0), full_end, false))) break;
        qk(0);
        commit(&bars.s_full[0]);
        qk(1);
        commit(&bars.s_full[1]);
        release();
        if (nt == 1) commit(q_free);
        for (int t = 0; ok && t < nt; ++t) {
          ok = wait_warp(&bars.p_ready[0], ph_p[0]++, err) && take(key0(t), full_end, true);
          if (!ok) break;
          tc_fence_after();
          pv(0, t == 0);
          const int v_it = it;
          if (t + 1 == nt) {
            commit(&bars.o_done[0]);
          } else {
            ++it;                                    // K of the next tile
            ok = take(key0(t + 1), full_end, false);
            if (!ok) break;
            qk(0);
            commit(&bars.s_full[0]);
            it = v_it;
          }
          ok = wait_warp(&bars.p_ready[1], ph_p[1]++, err);
          if (!ok) break;
          tc_fence_after();
          pv(1, t == 0);
          release();                                 // V
          if (t + 1 == nt) {
            commit(&bars.o_done[1]);
          } else {
            qk(1);
            commit(&bars.s_full[1]);
            release();                               // K
            if (t + 2 == nt) commit(q_free);
          }
        }
      } else {
        // Stages in order K0 K1 V0 K2 V1 ...; tile t belongs to stream t & 1.
        for (int t = 0; ok && t < min(nt, 2); ++t) {
          if (!(ok = take(key0(t), full_end, false))) break;
          qk(t);
          commit(&bars.s_full[t]);
          release();
        }
        if (ok && nt <= 2) commit(q_free);
        for (int t = 0; ok && t < nt; ++t) {
          const int s = t & 1;
          ok = wait_warp(&bars.p_ready[s], ph_p[s]++, err) && take(key0(t), full_end, true);
          if (!ok) break;
          tc_fence_after();
          pv(s, t < 2);
          release();
          if (t + 2 < nt) {
            if (!(ok = take(key0(t + 2), full_end, false))) break;
            qk(s);
            commit(&bars.s_full[s]);
            release();
            if (t + 3 == nt) commit(q_free);
          } else {
            commit(&bars.o_done[s]);
          }
        }
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
    int it = 0, rit = 0, seg = 0;
    uint32_t found = 0;
    // Not kRaw: V tiles that reach past the committed tokens, in place.
    auto repair = [&](const Seg &g, int tile) {
      const int st = it % S::kStages;
      uint8_t *base = ring + st * S::kStageBytes;
      const int k0 = tile * kTile;
      const int r0 = max(min(g.r.L, g.r.kv_end) - k0, 0), r1 = g.r.kv_end - k0;  // new rows [r0, r1)
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
    auto widen = [&](const Seg &g, int tile, bool is_v) {
      const int st = it % S::kStages, rs = rit % (S::kRaw ? S::kRawStages : 1);
      if (!wait_warp(&bars.rfull[rs], (rit / (S::kRaw ? S::kRawStages : 1)) & 1, err)) return false;
      if (it >= S::kStages && !wait_warp(&bars.empty[st], (it / S::kStages) & 1 ? 0u : 1u, err)) return false;
      const uint8_t *src = raw + rs * S::kRawBytes;
      const uint8_t *sc = src + S::kRawData;
      uint8_t *dst = ring + st * S::kStageBytes;
      constexpr int kCh = D / 16;                       // 16-code chunks per row
      const int k0 = tile * kTile, r1 = is_v ? g.r.kv_end - k0 : kTile;
      const bool look = is_v && k0 + kTile > min(g.r.L, g.r.kv_end);
      const int r0 = max(min(g.r.L, g.r.kv_end) - k0, 0);
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
    auto stage = [&](const Seg &g, int tile, bool is_v) {
      if constexpr (S::kRaw) {
        if (!widen(g, tile, is_v)) return false;
        if (found) seg_bad[seg % kSegRing] = 1;
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
        const bool fix = is_v && (tile + 1) * kTile > min(g.r.L, g.r.kv_end);
        if (fix) {
          repair(g, tile);
          if (found) seg_bad[seg % kSegRing] = 1;
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
    for (; ok && walk.next(a, upt, rc, sg); ++seg) {
      for (int t = sg.t0; ok && t < sg.t1; ++t) {
        ok = stage(sg, t, false);
        if (kPair) ok = ok && stage(sg, t, true);
        else if (t > sg.t0) ok = ok && stage(sg, t - 1, true);
      }
      if (!kPair) ok = ok && stage(sg, sg.t1 - 1, true);
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
  const int quota = ld32(p.head), start = ld32(p.pre + b) + (h * r.mp + mp) * r.kt;
  const int c0 = start / quota, c1 = (start + r.kt - 1) / quota;
  auto slot_of = [&](int c) {
    return p.slots + (static_cast<size_t>(c) * 2 + (c == c0 && start % quota ? 1 : 0)) * p.slot_floats;
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
