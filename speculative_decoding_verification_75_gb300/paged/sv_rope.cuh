// sv_rope.cuh -- norms of queries and keys for each head, the rotation by their
// positions, and the keys and values into the paged cache, in one pass.
//
// A head's row x of D elements becomes y = x / sqrt(mean(x^2) + eps) * w, whose
// first R elements turn in pairs (a, b) by the angle of the token's position:
// (a cos - b sin, b cos + a sin); pairs are (i, i + R / 2) or (2 i, 2 i + 1).
//
// Bound by HBM where there are many tokens: every element is read and written
// once.  A lane holds 8 adjacent elements (16 bytes) of a row, D / 8 lanes a row;
// the sum of squares and a pair's other half come by shuffles.  A warp takes
// several rows of one token, so that the angles and weights of its 8 columns stay
// in registers, and has the loads of kRopeRows rows in flight.
#pragma once

#include "sv_paged_quant.cuh"

namespace svp {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4;
constexpr int kRopeWarps = 152 * 32;   // warps that a batch is spread over at least

struct RopeParams {
  Cache c;                       // c.k NULL: none
  const uint8_t *q, *k, *v;
  uint8_t *qo, *ko;              // ko may be NULL
  int64_t qsb, qst, qsh, ksb, kst, ksh, vsb, vst, vsh;        // strides in bytes
  int64_t qosb, qost, qosh, kosb, kost, kosh;
  const uint8_t *qw, *kw;        // NULL: no norm
  const float *cos_sin;          // [P, R]: R / 2 cosines, R / 2 sines
  const int32_t *positions;      // [B, T]
  const int64_t *slots;          // [B, T] or NULL
  float eps;
  int B, T, Hq, Hkv, D, R, P;
  int lanes;                     // of a row: a power of two, at least D / 8
  int rows, steps, runs;         // rows of a token; of a warp, in groups of 32 / lanes; warps of a token
  int vec;                       // rows on 16-byte boundaries
  uint32_t *status;
};

__device__ __forceinline__ void store16(uint8_t *d, const uint4 &v, bool vec) {
  if (vec) {
    *reinterpret_cast<uint4 *>(d) = v;
    return;
  }
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint16_t *>(d + 2 * i) = static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
}

// Q: type of queries, keys and values; C: the cache's (Q: its own type, or no
// cache); kPairs: neighbours turn together.
template <typename Q, typename C, bool kPairs>
__global__ void __launch_bounds__(kRopeThreads) sv_rope_kernel(const RopeParams p) {
  sv::pdl_wait();
  sv::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int64_t token = task / p.runs;
  if (token >= static_cast<int64_t>(p.B) * p.T) return;        // whole warps
  const int run = static_cast<int>(task - token * p.runs);
  const int b = static_cast<int>(token / p.T), t = static_cast<int>(token - static_cast<int64_t>(b) * p.T);

  // The token's angle and its place in the cache.
  const int pos = ld32(p.positions + token);
  int64_t at = 0, sat = 0;
  if (p.slots) {
    const uint2 w = ld64(p.slots + token);
    const int64_t slot = static_cast<int64_t>(static_cast<uint64_t>(w.y) << 32 | w.x);
    if (slot < 0) return;                                      // no token here
    const int64_t id = slot / p.c.bs;
    if (id >= p.c.num_blocks) {
      if (run == 0 && lane == 0) report(p.status, SV_KV_BAD_BLOCK);
      return;
    }
    const int row = static_cast<int>(slot - id * p.c.bs);
    at = id * p.c.block_bytes + static_cast<int64_t>(row) * (p.D / 8 * C::kBits);
    sat = id * p.c.sblock_bytes + static_cast<int64_t>(row) * (p.D / SV_KV_GROUP);
  }
  if (p.R > 0 && (pos < 0 || pos >= p.P)) {
    if (run == 0 && lane == 0) report(p.status, SV_KV_BAD_LENGTH);
    return;
  }
  const int ch = lane & (p.lanes - 1), group = 32 / p.lanes, sub = lane / p.lanes;
  const bool in = ch < p.D / 8;
  // The lane's angles: cs[e], sn[e] of element e; the partner of element e is
  // element e of lane `mate`, or (kPairs) its neighbour.  sn has the sign of the
  // partner's term.
  float cs[8] = {}, sn[8] = {};
  const int turned = min(max(p.R - 8 * ch, 0), 8);             // of the lane's elements, the first ones
  const float *angles = p.cos_sin + static_cast<int64_t>(pos) * p.R;
  int mate = lane;
  if (kPairs) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = ch * 4 + e;
      if (2 * e < turned) {
        const float c = __uint_as_float(static_cast<uint32_t>(ld32(reinterpret_cast<const int32_t *>(angles + j))));
        const float s = __uint_as_float(static_cast<uint32_t>(ld32(reinterpret_cast<const int32_t *>(angles + p.R / 2 + j))));
        cs[2 * e] = cs[2 * e + 1] = c;
        sn[2 * e] = -s;
        sn[2 * e + 1] = s;
      }
    }
  } else {
    const int half = p.R / 16;                                 // lanes of a half
    if (turned) {
      const bool low = ch < half;
      mate = low ? lane + half : lane - half;
      const float *a = angles + (low ? ch : ch - half) * 8;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const uint4 c = ld128(a + e), s = ld128(a + p.R / 2 + e);
        const uint32_t cu[4] = {c.x, c.y, c.z, c.w}, su[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          cs[e + k] = __uint_as_float(cu[k]);
          sn[e + k] = low ? -__uint_as_float(su[k]) : __uint_as_float(su[k]);
        }
      }
    }
  }
  const uint4 none = make_uint4(0, 0, 0, 0);
  const uint4 wq = p.qw && in ? ld128(p.qw + ch * 16) : none, wk = p.kw && in ? ld128(p.kw + ch * 16) : none;
  const int r0 = run * p.steps * group;
#pragma unroll 1
  for (int s0 = 0; s0 < p.steps; s0 += kRopeRows) {
    uint4 raw[kRopeRows];
#pragma unroll
    for (int i = 0; i < kRopeRows; ++i) {
      const int r = r0 + (s0 + i) * group + sub;
      raw[i] = none;
      if (in && s0 + i < p.steps && r < p.rows) {
        const uint8_t *src = r < p.Hq ? p.q + b * p.qsb + t * p.qst + r * p.qsh
                             : r < p.Hq + p.Hkv ? p.k + b * p.ksb + t * p.kst + (r - p.Hq) * p.ksh
                                                : p.v + b * p.vsb + t * p.vst + (r - p.Hq - p.Hkv) * p.vsh;
        raw[i] = load16(src + ch * 16, p.vec);
      }
    }
#pragma unroll
    for (int i = 0; i < kRopeRows; ++i) {
      const int r = r0 + (s0 + i) * group + sub;
      if (s0 + i >= p.steps || r0 + (s0 + i) * group >= p.rows) break;   // the same for the warp
      const bool is_q = r < p.Hq, is_k = !is_q && r < p.Hq + p.Hkv, on = in && r < p.rows;
      if (__any_sync(kFull, on && (is_q || is_k))) {           // not a warp of values alone
        float x[8];
        unpack8<Q>(&raw[i], x);
        const bool norm = is_q ? p.qw != nullptr : p.kw != nullptr;
        if (p.qw || p.kw) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
          for (int o = 1; o < p.lanes; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
          if (norm) {
            const float f = 1.f / sqrtf(ss / static_cast<float>(p.D) + p.eps);
            float w[8];
            const uint4 ww = is_q ? wq : wk;
            unpack8<Q>(&ww, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * f * w[e];
          }
        }
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float other = kPairs ? x[e ^ 1] : __shfl_sync(kFull, x[e], mate);
          y[e] = e < turned ? fmaf(other, sn[e], x[e] * cs[e]) : x[e];   // not x + 0 * other: it may be infinite
        }
        if (is_q || is_k) pack8<Q>(&raw[i], y);
      }
      if (on && is_q) store16(p.qo + b * p.qosb + t * p.qost + r * p.qosh + ch * 16, raw[i], p.vec);
      if (on && is_k && p.ko) store16(p.ko + b * p.kosb + t * p.kost + (r - p.Hq) * p.kosh + ch * 16, raw[i], p.vec);
      if (p.slots && __any_sync(kFull, on && !is_q)) {
        const int h = is_k ? r - p.Hq : r - p.Hq - p.Hkv;
        const bool put = on && !is_q;
        uint8_t *dst = (is_k ? p.c.k : p.c.v) + at + static_cast<int64_t>(h) * p.c.bs * (p.D / 8 * C::kBits) + ch * C::kBits;
        if constexpr (C::kScaled) {
          typename Codes<C>::type codes;
          const uint32_t sc = quantise8<Q>(raw[i], codes);
          if (put) {
            *reinterpret_cast<typename Codes<C>::type *>(dst) = codes;
            if ((ch & 3) == 0)
              (is_k ? p.c.ks : p.c.vs)[sat + static_cast<int64_t>(h) * p.c.bs * (p.D / SV_KV_GROUP) + ch / 4] =
                  static_cast<uint8_t>(sc);
          }
        } else {
          if (put) *reinterpret_cast<uint4 *>(dst) = raw[i];
        }
      }
    }
  }
}

}  // namespace svp
