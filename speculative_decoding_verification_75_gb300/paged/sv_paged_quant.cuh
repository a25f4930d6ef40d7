// sv_paged_quant.cuh -- 16-bit elements on their way into a cache of codes.
#pragma once

#include "sv_paged_common.cuh"

namespace svp {

// Eight codes.
template <typename C>
struct Codes {
  using type = uint2;
};
template <>
struct Codes<I4> {
  using type = uint32_t;
};

// The largest magnitudes of the even and of the odd of eight 16-bit numbers, as integers.
__device__ __forceinline__ uint32_t halves8(const uint4 &raw) {
  uint32_t big = 0;
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) big = __vmaxu2(big, u[i] & 0x7fff7fffu);
  return big;
}
__device__ __forceinline__ uint32_t largest8(const uint4 &raw) {
  const uint32_t big = halves8(raw);
  return max(big & 0xffffu, big >> 16);
}

// Quantises 32 elements that 4 adjacent lanes hold (8 each); returns the
// scale byte.  Every lane of the warp takes part.  Magnitudes are compared as
// 16-bit integers, two at a time, and only a warp that meets an infinity or NaN
// looks at its elements one by one (8 prompts of up to 8192 tokens: 58 us, 5.3 TB/s;
// 68 us with comparisons of single fp32 magnitudes).
template <typename Q>
__device__ __forceinline__ uint32_t quantise8(const uint4 &raw, uint2 &codes) {
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
  constexpr uint32_t kInf = Q::kIsBf16 ? 0x7f80u : 0x7c00u;
  uint32_t big = largest8(raw);
  const bool odd = __any_sync(kFull, big >= kInf);
  if (odd) {                                       // the largest finite magnitude
    big = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = u[i] & 0x7fffu, hi = (u[i] >> 16) & 0x7fffu;
      big = max(big, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
    }
  }
  big = max(big, __shfl_xor_sync(kFull, big, 1));
  big = max(big, __shfl_xor_sync(kFull, big, 2));
  float a[8];
  const uint4 only = make_uint4(big, 0, 0, 0);
  unpack8<Q>(&only, a);
  // a = 1.f * 2^E <= 448 * 2^e = 1.75 * 2^(e + 8): e = E - 8, or E - 7 where
  // 1.f is above 1.75.  (Subnormal a: E is too large, but e is -120 anyway.)
  const uint32_t v = __float_as_uint(a[0]);
  int e = static_cast<int>(v >> 23) - 127 - 8 + ((v & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, -120);
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  float f[8];
  unpack8<Q>(&raw, f);
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 y = make_float2(f[2 * i] * inv, f[2 * i + 1] * inv);  // exact, or below every code
    if (odd) {  // at most 448 where f is finite; an infinity becomes NaN, not 448
      if (!(fabsf(y.x) <= 448.f)) y.x = __uint_as_float(0x7fc00000u);
      if (!(fabsf(y.y) <= 448.f)) y.y = __uint_as_float(0x7fc00000u);
    }
    h[i] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
  }
  codes = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  return static_cast<uint32_t>(e + 127);
}

// A group's scale as codes of 4 bits have it: f, the smallest with amax <= 7 f, its byte,
// and 1 / f.  An infinity or NaN makes the group's scale NaN.
struct Scale4 {
  int s;
  float f, inv;
  bool odd, over;                                // not finite; that, or above every scale
};
template <typename Q>
__device__ __forceinline__ Scale4 scale4(uint32_t big) {
  constexpr uint32_t kInf = Q::kIsBf16 ? 0x7f80u : 0x7c00u;
  Scale4 r;
  r.odd = big >= kInf;
  float amax;
  if constexpr (Q::kIsBf16) amax = __uint_as_float(big << 16);
  else amax = __half2float(*reinterpret_cast<const __half *>(&big));
  // The quotient's upper bits are the byte, moved by 113 * 8, unless 7 f is too
  // small: amax has at most 11 bits, so a quotient that is not a scale lies 2^-11
  // or more from one, and the reciprocal is off by 2^-23.
  const float t = amax * (1.f / 7.f) * (1.f - 0x1p-20f);
  int s = max(static_cast<int>(__float_as_uint(t) >> 20) - 113 * 8, 0);
  if (7.f * scale_value<I4>(min(s, SV_KV_I4_MAX_SCALE)) < amax) ++s;
  r.over = s > SV_KV_I4_MAX_SCALE;
  r.s = min(s, SV_KV_I4_MAX_SCALE);
  r.f = scale_value<I4>(r.s);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.inv) : "f"(r.f));   // 2^-23 off
  return r;
}
__device__ __forceinline__ void limit8(float (&x)[8], float f, bool odd) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = odd ? 0.f : fminf(fmaxf(x[i], -7.f * f), 7.f * f);
}

// Codes of eight elements: x / f rounded to the nearest whole number, by the addition of
// 1.5 * 2^23 + 8, whose sum's low bits are the code; one multiply-add moves it to its
// place.  Quotients are whole numbers and a half, or 2^-12 or more away from those (x has
// at most 11 bits): rounded to 2^-13 first, by the sum with 1536, the former are exact
// and go to the even one, and the others stay on their side.
__device__ __forceinline__ uint32_t codes4(const float (&x)[8], float inv) {
  const uint64_t inv2 = f2_pack(inv, inv), one2 = f2_pack(1.f, 1.f), fine2 = f2_pack(1536.f, 1536.f);
  const uint64_t up2 = f2_pack(12582920.f - 1536.f, 12582920.f - 1536.f);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const uint64_t y = f2_fma(f2_fma(f2_pack(x[2 * i], x[2 * i + 1]), inv2, fine2), one2, up2);
    codes = (codes * 16u + static_cast<uint32_t>(y >> 32)) * 16u + static_cast<uint32_t>(y);
  }
  return codes - 0x4b400000u * 0x11111111u;      // the sums' upper bits; the codes are 1 .. 15
}

template <typename Q>
__device__ __forceinline__ uint32_t quantise8(const uint4 &raw, uint32_t &codes) {
  uint32_t big = largest8(raw);
  big = max(big, __shfl_xor_sync(kFull, big, 1));
  big = max(big, __shfl_xor_sync(kFull, big, 2));
  const Scale4 sc = scale4<Q>(big);
  float x[8];
  unpack8<Q>(&raw, x);
  if (__any_sync(kFull, sc.over)) limit8(x, sc.f, sc.odd);
  codes = codes4(x, sc.inv);
  return sc.odd ? 255u : static_cast<uint32_t>(sc.s);
}

// Four rows at once: each of the four lanes of a group finds one row's scale, whose byte
// it returns, lane 4 g + j that of row j.  Bound by instructions, so their number is
// what counts: two shuffles join the largest of four rows, 16 bits each (8 prompts of up
// to 8192 tokens: kv_write 56 us, 4.6 TB/s; 65 us with each row by itself, quotients corrected by
// their remainders; 77 us with a conversion and comparisons for each element).
template <typename Q>
__device__ __forceinline__ uint32_t quantise4x8(const uint4 *raw, uint32_t (&codes)[4]) {
  uint32_t two[2];                               // rows 0 and 1, rows 2 and 3
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = halves8(raw[2 * i]), b = halves8(raw[2 * i + 1]);
    two[i] = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
  }
  const int lane = threadIdx.x & 31;
  uint32_t big = lane & 2 ? two[1] : two[0];
  big = __vmaxu2(big, __shfl_xor_sync(kFull, lane & 2 ? two[0] : two[1], 2));
  big = __vmaxu2(big, __shfl_xor_sync(kFull, big, 1));
  const Scale4 sc = scale4<Q>(lane & 1 ? big >> 16 : big & 0xffffu);
  const bool over = __any_sync(kFull, sc.over);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float x[8];
    unpack8<Q>(&raw[j], x);
    if (over) {
      const float f = __shfl_sync(kFull, sc.f, j, 4);
      limit8(x, f, __shfl_sync(kFull, static_cast<int>(sc.odd), j, 4));
    }
    codes[j] = codes4(x, __shfl_sync(kFull, sc.inv, j, 4));
  }
  return sc.odd ? 255u : static_cast<uint32_t>(sc.s);
}

// 16 bytes from the dense side, whatever its alignment (2-byte elements).
__device__ __forceinline__ uint4 load16(const uint8_t *s, bool vec) {
  if (vec) return ld128(s);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = ld16(s + 4 * k) | (ld16(s + 4 * k + 2) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace svp
