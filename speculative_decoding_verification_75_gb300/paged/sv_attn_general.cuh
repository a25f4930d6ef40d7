// sv_attn_general.cuh -- attention of one query row over the paged cache,
// right for every block size, head dimension and type: the kernel for what
// the tensor-core kernel does not take, and the one that recomputes rows
// whose masked places hold values that a product with 0 would not hide.
#pragma once

#include "sv_paged_common.cuh"

namespace svp {

struct AttnParams {
  Cache c;
  Batch bt;
  const uint8_t *q;
  int64_t qsb, qst, qsh;       // bytes
  const uint8_t *mask;         // NULL: chain
  int64_t msb;                 // bytes between requests
  uint8_t *out;
  float *lse;
  float scale_log2;            // scale * log2(e)
  int Hq, G;                   // query heads, query heads per KV head
  int qvec;                    // query rows on 16-byte boundaries
};

constexpr float kLn2 = 0.693147180559945309f;

// Online softmax state of one row, spread over a warp: m and l are the same
// in every lane, lane i holds output elements i, i + 32, ...
template <int kMaxD>
struct RowState {
  float m, l;                  // max and sum of 2^(x - m), x in log2 units
  float o[kMaxD / 32];
};

// Positions of request b that the table holds.  A length far behind it costs no
// look-ups: 2^31 positions of a row would take seconds.
__device__ __forceinline__ int held(const Cache &c, int L, int n, uint32_t &st) {
  const int total = min(L + n, c.max_blocks * c.bs);  // both below 2^31
  if (total < L + n) st |= SV_KV_TABLE_SHORT;
  return total;
}

// Positions j0 + lane, j0 + step + lane, ... below `total` of row (b, i) and
// KV head h, by one warp.  load_q(d, f): elements d .. d + 7 of the row.
template <typename C, int kMaxD, typename LoadQ>
__device__ __forceinline__ void attend(const AttnParams &p, int b, int i, int h, int L, int n,
                                       int total, const LoadQ &load_q, int j0, int step, int lane,
                                       RowState<kMaxD> &r, uint32_t &st) {
  const int D = p.c.D, row_bytes = D / 8 * C::kBits, srow = D / SV_KV_GROUP;
  const int64_t head_bytes = static_cast<int64_t>(h) * p.c.bs * row_bytes;
  const int64_t shead = static_cast<int64_t>(h) * p.c.bs * srow;
  const uint8_t *mrow =
      p.mask ? p.mask + b * p.msb + static_cast<int64_t>(i) * p.bt.T : nullptr;
  for (int64_t jj = j0; jj < total; jj += step) {
    const int j = static_cast<int>(jj) + lane;
    const bool in = jj + lane < total;
    const int id = in ? block_of(p.c, b, j, st) : -1;  // hidden positions too: their problems are reported
    bool see = id >= 0;
    if (see && j >= L) see = mrow ? ld8(mrow + (j - L)) != 0 : j - L <= i;
    int64_t at = 0, sat = 0;
    if (see) {
      const int row = j % p.c.bs;
      at = id * p.c.block_bytes + head_bytes + static_cast<int64_t>(row) * row_bytes;
      sat = id * p.c.sblock_bytes + shead + static_cast<int64_t>(row) * srow;
    }
    float x = -INFINITY;
    if (see) {
      x = 0.f;
      for (int d = 0; d < D; d += 8) {
        const uint4 raw = load8<C>(p.c.k + at + d / 8 * C::kBits);
        float f[8], q[8];
        unpack8<C>(&raw, f);
        load_q(d, q);
        float s8 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s8 = fmaf(q[e], f[e], s8);
        if constexpr (C::kScaled) s8 *= scale_value<C>(ld8(p.c.ks + sat + d / SV_KV_GROUP));
        x += s8;
      }
    }
    x *= p.scale_log2;
    if (!see) x = -INFINITY;
    // fmaxf drops a NaN: it comes back through 2^(x - m) below.
    const float mt = fmaxf(r.m, sv::warp_max(x));
    const float base = mt == -INFINITY ? 0.f : mt;
    const float f = sv::ex2(r.m - base);
    const float w = see ? sv::ex2(x - base) : 0.f;
    r.m = mt;
    r.l = r.l * f + sv::warp_sum(w);
#pragma unroll
    for (int e = 0; e < kMaxD / 32; ++e) r.o[e] *= f;
    unsigned todo = __ballot_sync(kFull, see);
    while (todo) {
      const int s = __ffs(todo) - 1;
      todo &= todo - 1;
      const float ws = __shfl_sync(kFull, w, s);
      const int64_t vs = __shfl_sync(kFull, at, s), ss = __shfl_sync(kFull, sat, s);
#pragma unroll
      for (int e = 0; e < kMaxD / 32; ++e) {
        const int d = lane + 32 * e;
        if (d < D) {
          float v;
          if constexpr (C::kBits == 8) {
            const __half_raw hr = __nv_cvt_fp8_to_halfraw(
                static_cast<__nv_fp8_storage_t>(ld8(p.c.v + vs + d)), __NV_E4M3);
            v = __half2float(__half(hr)) * scale_value<C>(ld8(p.c.vs + ss + d / SV_KV_GROUP));
          } else if constexpr (C::kBits == 4) {
            const uint32_t code = ld8(p.c.v + vs + d / 2) >> (4 * (d & 1)) & 15u;
            v = static_cast<float>(static_cast<int>(code) - 8) * scale_value<C>(ld8(p.c.vs + ss + d / SV_KV_GROUP));
          } else if constexpr (sizeof(typename C::raw) == 2) {
            const uint16_t w16 = static_cast<uint16_t>(ld16(p.c.v + vs + d * 2));
            v = load1<C>(&w16);
          }
          r.o[e] = fmaf(ws, v, r.o[e]);
        }
      }
    }
  }
}

// Stores a row: o / l in the output's type, 0 where nothing was seen.
template <typename Q, int kMaxD>
__device__ __forceinline__ void store_row(const AttnParams &p, int64_t row, int lane,
                                          const RowState<kMaxD> &r) {
  const float inv = r.l == 0.f ? 0.f : 1.f / r.l;
#pragma unroll
  for (int e = 0; e < kMaxD / 32; ++e) {
    const int d = lane + 32 * e;
    if (d < p.c.D) store1<Q>(p.out + (row * p.c.D + d) * 2, r.l == 0.f ? 0.f : r.o[e] * inv);
  }
  if (p.lse && lane == 0)
    p.lse[row] = r.l == 0.f ? -INFINITY : r.m * kLn2 + logf(r.l);
}

// A whole row by one warp, for query rows on 16-byte boundaries.  Not inlined:
// the rare way out of the tensor-core kernels.
template <typename Q, typename C, int D>
__device__ __noinline__ void recompute_row(const AttnParams &p, int b, int i, int hq) {
  const int lane = threadIdx.x & 31;
  uint32_t st = 0;
  int L, n;
  lengths(p.bt, b, L, n, st);
  const uint8_t *q = p.q + b * p.qsb + i * p.qst + hq * p.qsh;
  const auto load_q = [&](int d, float (&f)[8]) {
    const uint4 w = ld128(q + d * 2);
    unpack8<Q>(&w, f);
  };
  RowState<D> r;
  r.m = -INFINITY;
  r.l = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) r.o[e] = 0.f;
  attend<C, D>(p, b, i, hq / p.G, L, n, held(p.c, L, n, st), load_q, 0, 32, lane, r, st);
  store_row<Q, D>(p, (static_cast<int64_t>(b) * p.bt.T + i) * p.Hq + hq, lane, r);
}

constexpr int kGenWarps = 4;

// One thread block per (request, new token, head); its warps take every
// fourth run of 32 positions and are merged in order.
template <typename Q, typename C>
__global__ void __launch_bounds__(32 * kGenWarps) sv_attn_general_kernel(const AttnParams p) {
  constexpr int kMaxD = SV_KV_MAX_HEAD_DIM;
  __shared__ float qs[kMaxD];
  __shared__ float part[kGenWarps][kMaxD + 2];
  sv::pdl_wait();
  sv::pdl_launch_dependents();
  const int64_t row = blockIdx.x;
  const int h = static_cast<int>(row % p.Hq);
  const int64_t bi = row / p.Hq;
  const int i = static_cast<int>(bi % p.bt.T), b = static_cast<int>(bi / p.bt.T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t st = 0;
  int L, n;
  lengths(p.bt, b, L, n, st);
  if (i >= n) {
    if (threadIdx.x == 0) report(p.bt.status, st);
    return;
  }
  const uint8_t *q = p.q + b * p.qsb + i * p.qst + h * p.qsh;
  for (int d = threadIdx.x; d < p.c.D; d += 32 * kGenWarps) {
    const uint16_t w = static_cast<uint16_t>(ld16(q + 2 * d));
    qs[d] = load1<Q>(&w);
  }
  __syncthreads();
  RowState<kMaxD> r;
  r.m = -INFINITY;
  r.l = 0.f;
#pragma unroll
  for (int e = 0; e < kMaxD / 32; ++e) r.o[e] = 0.f;
  const auto load_q = [&](int d, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = qs[d + e];
  };
  attend<C, kMaxD>(p, b, i, h / p.G, L, n, held(p.c, L, n, st), load_q, warp * 32, 32 * kGenWarps, lane, r, st);
#pragma unroll
  for (int e = 0; e < kMaxD / 32; ++e) part[warp][lane + 32 * e] = r.o[e];
  if (lane == 0) {
    part[warp][kMaxD] = r.m;
    part[warp][kMaxD + 1] = r.l;
  }
  report(p.bt.status, st);
  __syncthreads();
  if (warp != 0) return;
  float m = -INFINITY;
  for (int w = 0; w < kGenWarps; ++w) m = fmaxf(m, part[w][kMaxD]);
  const float base = m == -INFINITY ? 0.f : m;
  RowState<kMaxD> t;
  t.m = m;
  t.l = 0.f;
#pragma unroll
  for (int e = 0; e < kMaxD / 32; ++e) t.o[e] = 0.f;
  for (int w = 0; w < kGenWarps; ++w) {
    const float f = sv::ex2(part[w][kMaxD] - base);
    t.l += part[w][kMaxD + 1] * f;
#pragma unroll
    for (int e = 0; e < kMaxD / 32; ++e) t.o[e] += part[w][lane + 32 * e] * f;
  }
  store_row<Q, kMaxD>(p, row, lane, t);
}

}  // namespace svp
