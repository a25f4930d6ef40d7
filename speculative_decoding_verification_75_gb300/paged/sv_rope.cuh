// sv_rope.cuh -- norms of queries and keys for each head, the rotation by their
// positions, and the keys and values into the paged cache, in one pass.
//
// A head's row x of D elements becomes y = x / sqrt(mean(x^2) + eps) * w, whose
// first R elements turn in pairs (a, b) by the angle of the token's position:
// (a cos - b sin, b cos + a sin); pairs are (i, i + R / 2) or (2 i, 2 i + 1).
//
// Every element is read and written once.  A lane holds 8 adjacent elements (16 bytes)
// of a row, D / 8 lanes a row; the sum of squares and a pair's other half come by
// shuffles.  A warp takes several steps of one token, each of a few rows of one kind
// (queries, keys or values), so that the angles of its 8 columns stay in registers,
// arithmetic is on pairs, and the loads of the next kRopeRows steps are in flight.
// The columns' cosines and sines carry the weights, so that an element takes two
// products, and the norm's factor comes last.
//
// Measured: 8 prompts of up to 4096 tokens, 32 heads on 8, into a bf16 cache: 115 us, 5.3
// TB/s, by its instructions (issue slots 81 % busy, 28 warps of 72 registers on an SM; with
// 4 steps a turn and 16 warps of 128 registers 145, one step a turn and 32 warps 130);
// 128 x 6 tokens, 64 heads on 8: 9.7 us (10.8 with twice as many warps, each with half of
// the steps).
#pragma once

#include "sv_paged_quant.cuh"

namespace svp {

constexpr int kRopeThreads = 128;
constexpr int kRopeRows = 2;
constexpr int kRopeWarps = 152 * 24;   // warps that a batch is spread over: 24 (of the fewest registers 28) fit an SM

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
  float eps, root_eps, inv_d;    // root_eps: eps^(1/2), inv_d: 1 / D
  float least;                   // kLeastSquares, or 0 where eps is kLeastEps or more
  int B, T, Hq, Hkv, D, R, P;
  int lanes;                     // of a row: a power of two, at least D / 8
  int steps_q, steps_k, steps;   // of 32 / lanes rows of one kind: queries, keys, all of a token
  int per, runs;                 // steps of a warp, warps of a token
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

// bf16 reaches as far as fp32: a row's squares may leave it, and so may its products with
// the weights, before the norm's factor.  Where a lane's squares sum up to kMostSquares
// at most neither does, for weights below 2^64 (with others a head's weights are taken at
// 2^-64, and the factor at 2^64; what is below 2^-62 beside these may become 0): |x| <=
// 2^40, |x w| <= 2^104.  Nor is anything lost below 2^-149 while the
// factor is at most 2^15, which eps holds; where eps is below 2^-30, kLeastSquares.  Rows
// outside are moved by a power of two first.  (The check costs prompts 111 -> 115 us,
// drafts 9.5 -> 9.7; in line, where registers for it left 6 blocks on an SM instead of 7,
// 119 and 125.)
constexpr uint32_t kHeavy = (127u + 64u) << 7;   // 2^64 in bf16
constexpr float kMostSquares = 0x1p80f, kLeastSquares = 0x1p-20f, kLeastEps = 0x1p-30f;

__device__ __forceinline__ float squares8(const float (&f)[8]) {
  uint64_t s2 = f2_mul(f2_pack(f[0], f[1]), f2_pack(f[0], f[1]));
#pragma unroll
  for (int e = 2; e < 8; e += 2) s2 = f2_fma(f2_pack(f[e], f[e + 1]), f2_pack(f[e], f[e + 1]), s2);
  float a, b;
  f2_unpack(s2, a, b);
  return a + b;
}

// A row moved by the power of two that takes the larger of its largest magnitude and
// eps^(1/2) to 2^57, exactly but for what lies 2^180 below that, and its lane's sum of
// squares, to which the row's first lane adds what eps becomes beside itself (eps is added
// to the mean later: at most 2^100, where that is 2^106 at least).  By the whole warp.
struct Moved {
  uint4 row;
  float squares;
};
__device__ __noinline__ Moved tame(uint4 row, float root_eps, float eps, int D, int lanes, bool first) {
  uint32_t big = largest8(row);
#pragma unroll 1
  for (int o = 1; o < lanes; o <<= 1) big = max(big, __shfl_xor_sync(kFull, big, o));
  big = max(big, __float_as_uint(root_eps) >> 16);
  const int e = 184 - static_cast<int>(big >> 7);
  const float r1 = __uint_as_float(static_cast<uint32_t>(127 + (e >> 1)) << 23);
  const float r2 = __uint_as_float(static_cast<uint32_t>(127 + e - (e >> 1)) << 23);
  float f[8];
  unpack8<BF16>(&row, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = f[i] * r1 * r2;
  pack8<BF16>(&row, f);
  const float root = root_eps * r1 * r2;
  return Moved{row, squares8(f) + (first ? fmaf(root, root, -eps) * static_cast<float>(D) : 0.f)};
}

// Q: type of queries, keys and values; C: the cache's (Q: its own type, or no
// cache); kPairs: neighbours turn together.
template <typename Q, typename C, bool kPairs>
__global__ void __launch_bounds__(kRopeThreads, 6) sv_rope_kernel(const RopeParams p) {
  sv::pdl_wait();
  sv::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);    // the same for the warp, and known to be
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + warp;
  const int64_t token = task / p.runs;
  if (token >= static_cast<int64_t>(p.B) * p.T) return;        // whole warps
  const int run = static_cast<int>(task - token * p.runs);
  const int b = static_cast<int>(token / p.T), t = static_cast<int>(token - static_cast<int64_t>(b) * p.T);
  const int ch = lane & (p.lanes - 1), group = 32 / p.lanes, sub = lane / p.lanes;
  const bool in = ch < p.D / 8;
  const uint4 none = make_uint4(0, 0, 0, 0);
  const int s_begin = run * p.per, s_end = min(s_begin + p.per, p.steps);
  const int s_k = p.steps_q, s_v = p.steps_q + p.steps_k;      // first steps of keys and values
  // Where the steps' rows come from: a pointer that moves on by a step's rows.
  const uint8_t *src = nullptr;
  int64_t src_step = 0;
  int src_left = 0;              // rows of the kind from the lane's on
  const auto aim = [&](int s) {
    const bool is_q = s < s_k, is_k = s < s_v;
    const int row = (s - (is_q ? 0 : is_k ? s_k : s_v)) * group + sub;
    const int64_t head = is_q ? p.qsh : is_k ? p.ksh : p.vsh;
    src = (is_q ? p.q + b * p.qsb + t * p.qst : is_k ? p.k + b * p.ksb + t * p.kst : p.v + b * p.vsb + t * p.vst) +
          row * head + ch * 16;
    src_step = group * head;
    src_left = in ? (is_q ? p.Hq : p.Hkv) - row : 0;
  };
  uint4 raw[kRopeRows];
  const auto fetch = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kRopeRows; ++i) {
      const int s = s0 + i;
      raw[i] = none;
      if (s >= s_end) continue;                                // the same for the warp
      if (s == s_begin || s == s_k || s == s_v) aim(s);
      if (src_left > 0) raw[i] = load16(src, p.vec);
      src += src_step;
      src_left -= group;
    }
  };
  fetch(s_begin);                // on its way while the token's place and angles are looked up

  // The token's angle and its place in the cache.
  const int pos = ld32(p.positions + token);
  int64_t at = 0, sat = 0;
  if (p.slots) {
    const uint2 w = ld64(p.slots + token);
    const int64_t slot = static_cast<int64_t>(static_cast<uint64_t>(w.y) << 32 | w.x);
    if (slot < 0) return;                                      // no token here
    const int64_t id = slot < 0x80000000ll ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.c.bs) : slot / p.c.bs;
    if (id >= p.c.num_blocks) {
      if (run == 0 && lane == 0) report(p.status, SV_KV_BAD_BLOCK);
      return;
    }
    const int row = static_cast<int>(slot - id * p.c.bs);
    at = id * p.c.block_bytes + static_cast<int64_t>(row) * (p.D / 8 * C::kBits) + ch * C::kBits;
    sat = id * p.c.sblock_bytes + static_cast<int64_t>(row) * (p.D / SV_KV_GROUP) + ch / 4;
  }
  if (p.R > 0 && (pos < 0 || pos >= p.P)) {
    if (run == 0 && lane == 0) report(p.status, SV_KV_BAD_LENGTH);
    return;
  }
  // A row's elements 2 e, 2 e + 1 become x * own[e] + (their partners) * mate_by[e]: the
  // angles' cosines times the weights, and the sines, with the sign of the partner's
  // term, times the partner's weight.  A partner is the same element of lane `mate`, or
  // (kPairs) the neighbour.
  uint64_t own[4] = {}, mate_by[4] = {};
  const int turned = min(max(p.R - 8 * ch, 0), 8);             // of the lane's elements, the first ones
  const int half = p.R / 16;                                   // lanes of a half
  const bool low = ch < half;
  const int mate = kPairs || !turned ? lane : low ? lane + half : lane - half;
  const float *angles = p.cos_sin + static_cast<int64_t>(pos) * p.R;
  float lift = 1.f;                                            // the weights are at 1 / lift
  const auto weigh = [&](const uint8_t *weight) {
    float c[8], s[8], w[8], wm[8];
    bool heavy = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = w[e] = 1.f;
      s[e] = 0.f;
    }
    if (kPairs) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        if (e < turned) {
          const float *a = angles + ch * 4 + e / 2;
          c[e] = c[e + 1] = __uint_as_float(static_cast<uint32_t>(ld32(reinterpret_cast<const int32_t *>(a))));
          s[e + 1] = __uint_as_float(static_cast<uint32_t>(ld32(reinterpret_cast<const int32_t *>(a + p.R / 2))));
          s[e] = -s[e + 1];
        }
      }
    } else if (turned) {
      const float *a = angles + (low ? ch : ch - half) * 8;
      const float sign = low ? -1.f : 1.f;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const uint4 x = ld128(a + e), y = ld128(a + p.R / 2 + e);
        const uint32_t u[4] = {x.x, x.y, x.z, x.w}, z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          c[e + k] = __uint_as_float(u[k]);
          s[e + k] = sign * __uint_as_float(z[k]);
        }
      }
    }
    if (weight && in) {
      const uint4 x = ld128(weight + ch * 16);
      unpack8<Q>(&x, w);
      heavy = Q::kIsBf16 && largest8(x) >= kHeavy;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) wm[e] = kPairs ? w[e ^ 1] : w[e];
    if (!kPairs && weight && turned) {
      const uint4 x = ld128(weight + (low ? ch + half : ch - half) * 16);
      unpack8<Q>(&x, wm);
    }
    if (Q::kIsBf16) {
      lift = 1.f;
      if (__any_sync(kFull, heavy)) {
        lift = 0x1p64f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[e] *= 0x1p-64f;
          wm[e] *= 0x1p-64f;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      own[e] = f2_pack(c[2 * e] * w[2 * e], c[2 * e + 1] * w[2 * e + 1]);
      mate_by[e] = f2_pack(s[2 * e] * wm[2 * e], s[2 * e + 1] * wm[2 * e + 1]);
    }
  };
  // Where the rows go, likewise: the output, and the cache's place of the row's head.
  uint8_t *to = nullptr, *cell = nullptr, *cell_s = nullptr;
  int64_t to_step = 0;
  const int64_t cell_step = static_cast<int64_t>(group) * p.c.bs * (p.D / 8 * C::kBits);
  const int64_t cell_s_step = static_cast<int64_t>(group) * p.c.bs * (p.D / SV_KV_GROUP);
  int left = 0;
  const auto aim_out = [&](int s) {
    const bool is_q = s < s_k, is_k = s < s_v;
    const int row = (s - (is_q ? 0 : is_k ? s_k : s_v)) * group + sub;
    left = in ? (is_q ? p.Hq : p.Hkv) - row : 0;
    const int64_t head = is_q ? p.qosh : p.kosh;
    to = is_q ? p.qo + b * p.qosb + t * p.qost : is_k && p.ko ? p.ko + b * p.kosb + t * p.kost : nullptr;
    if (to) to += row * head + ch * 16;
    to_step = to ? group * head : 0;
    if (is_k) weigh(is_q ? p.qw : p.kw);
    if (!is_q && p.slots) {
      cell = (is_k ? p.c.k : p.c.v) + at + static_cast<int64_t>(row) * p.c.bs * (p.D / 8 * C::kBits);
      if (C::kScaled) cell_s = (is_k ? p.c.ks : p.c.vs) + sat + static_cast<int64_t>(row) * p.c.bs * (p.D / SV_KV_GROUP);
    }
  };
  const bool normed = p.qw || p.kw;
#pragma unroll 1
  for (int s0 = s_begin; s0 < s_end; s0 += kRopeRows) {
    uint4 now[kRopeRows];
#pragma unroll
    for (int i = 0; i < kRopeRows; ++i) now[i] = raw[i];
    if (s0 + kRopeRows < s_end) fetch(s0 + kRopeRows);         // the next steps', meanwhile
    // The steps' sums of squares side by side: alone each is a chain of shuffles.
    float ss[kRopeRows];
    if (normed && s0 < s_v) {
#pragma unroll
      for (int i = 0; i < kRopeRows; ++i) {
        float f[8];
        unpack8<Q>(&now[i], f);
        ss[i] = squares8(f);
      }
      if constexpr (Q::kIsBf16) {
        float top = ss[0], low = ss[0];
#pragma unroll
        for (int i = 1; i < kRopeRows; ++i) {
          top = fmaxf(top, ss[i]);
          low = fminf(low, ss[i]);
        }
        if (__any_sync(kFull, top > kMostSquares || low < p.least)) {
#pragma unroll
          for (int i = 0; i < kRopeRows; ++i) {
            if (s0 + i < s_k ? p.qw != nullptr : s0 + i < s_v && p.kw) {   // the same for the warp
              const Moved y = tame(now[i], p.root_eps, p.eps, p.D, p.lanes, ch == 0);
              now[i] = y.row;
              ss[i] = y.squares;
            }
          }
        }
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        if (o >= p.lanes) break;
#pragma unroll
        for (int i = 0; i < kRopeRows; ++i) ss[i] += __shfl_xor_sync(kFull, ss[i], o);
      }
#pragma unroll
      for (int i = 0; i < kRopeRows; ++i) ss[i] = rsqrtf(fmaf(ss[i], p.inv_d, p.eps));   // off by 2^-22
    }
#pragma unroll
    for (int i = 0; i < kRopeRows; ++i) {
      const int s = s0 + i;
      if (s >= s_end) break;                                   // the same for the warp
      if (s == s_begin || s == s_k || s == s_v) aim_out(s);
      const bool is_q = s < s_k, on = left > 0;
      if (s < s_v) {
        float f[8], g[8];
        unpack8<Q>(&now[i], f);
        if (kPairs) {
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = f[e ^ 1];
        } else if (p.R > 0) {
          const uint4 o = make_uint4(__shfl_sync(kFull, now[i].x, mate), __shfl_sync(kFull, now[i].y, mate),
                                     __shfl_sync(kFull, now[i].z, mate), __shfl_sync(kFull, now[i].w, mate));
          unpack8<Q>(&o, g);
        }
        uint64_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = f2_mul(f2_pack(f[2 * e], f[2 * e + 1]), own[e]);
        if (p.R > 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (2 * e < turned) x[e] = f2_fma(f2_pack(g[2 * e], g[2 * e + 1]), mate_by[e], x[e]);   // else it may be infinite
        }
        if (is_q ? p.qw != nullptr : p.kw != nullptr) {
          const float by = Q::kIsBf16 ? ss[i] * lift : ss[i];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = f2_mul(x[e], f2_pack(by, by));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) f2_unpack(x[e], f[2 * e], f[2 * e + 1]);
        pack8<Q>(&now[i], f);
      }
      if (on && to) store16(to, now[i], p.vec);
      to += to_step;
      left -= group;
      if (is_q || !p.slots) continue;
      if constexpr (C::kScaled) {
        typename Codes<C>::type codes;
        const uint32_t sc = quantise8<Q>(now[i], codes);
        if (on) {
          *reinterpret_cast<typename Codes<C>::type *>(cell) = codes;
          if ((ch & 3) == 0) *cell_s = static_cast<uint8_t>(sc);
        }
        cell_s += cell_s_step;
      } else {
        if (on) *reinterpret_cast<uint4 *>(cell) = now[i];
      }
      cell += cell_step;
    }
  }
}

}  // namespace svp
