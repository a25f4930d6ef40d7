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

// Quantises 32 elements that 4 adjacent lanes hold (8 each); returns the
// scale byte.  Every lane of the warp takes part.  Magnitudes are compared as
// 16-bit integers, two at a time, and only a warp that meets an infinity or NaN
// looks at its elements one by one (8 prompts of up to 8192 tokens: 58 us, 5.3 TB/s;
// 68 us with comparisons of single fp32 magnitudes).
template <typename Q>
__device__ __forceinline__ uint32_t largest8(const uint4 &raw) {
  uint32_t big = 0;
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) big = __vmaxu2(big, u[i] & 0x7fff7fffu);
  return max(big & 0xffffu, big >> 16);
}

template <typename Q>
__device__ __forceinline__ uint32_t quantise8(const uint4 &raw, uint2 &codes) {
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
  constexpr uint32_t kInf = Q::kIsBf16 ? 0x7f80u : 0x7c00u;
  uint32_t big = largest8<Q>(raw);
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

// Two fp32 at once.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float lower(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float upper(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The same as codes of 4 bits: x / f rounded to the nearest whole number, f the
// smallest scale with amax <= 7 f.  An infinity or NaN makes the group's scale NaN.
// Bound by instructions, so each element takes about five: products of pairs,
// rounding by the addition of 1.5 * 2^23 + 8, whose sum's low bits are the code, and
// one multiply-add that moves it to its place (8 prompts of up to 8192 tokens: kv_write
// 65 us, 4.0 TB/s; 77 us with a conversion and comparisons for each element).
template <typename Q>
__device__ __forceinline__ uint32_t quantise8(const uint4 &raw, uint32_t &codes) {
  constexpr uint32_t kInf = Q::kIsBf16 ? 0x7f80u : 0x7c00u;
  uint32_t big = largest8<Q>(raw);
  big = max(big, __shfl_xor_sync(kFull, big, 1));
  big = max(big, __shfl_xor_sync(kFull, big, 2));
  const bool odd = big >= kInf;
  const uint32_t big16 = big;
  float amax;
  if constexpr (Q::kIsBf16) amax = __uint_as_float(big << 16);
  else amax = __half2float(*reinterpret_cast<const __half *>(&big16));
  // The quotient's upper bits are the byte, moved by 113 * 8, unless 7 f is too
  // small: amax has at most 11 bits, so a quotient that is not a scale lies 2^-11
  // or more from one, and the reciprocal is off by 2^-23.
  const float t = amax * (1.f / 7.f) * (1.f - 0x1p-20f);
  int s = max(static_cast<int>(__float_as_uint(t) >> 20) - 113 * 8, 0);
  if (7.f * scale_value<I4>(min(s, SV_KV_I4_MAX_SCALE)) < amax) ++s;
  const bool over = s > SV_KV_I4_MAX_SCALE;      // or not finite
  s = min(s, SV_KV_I4_MAX_SCALE);
  const float f = scale_value<I4>(s);
  float inv;                                     // 2^-23 off: the remainder below makes up for it
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(f));
  float x[8];
  unpack8<Q>(&raw, x);
  if (__any_sync(kFull, over)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = odd ? 0.f : fminf(fmaxf(x[i], -7.f * f), 7.f * f);
  }
  // The quotient once more by its remainder: one that is a whole number and a half
  // comes out exactly, so that it goes to the even one.
  const uint64_t inv2 = pair2(inv, inv), f2 = pair2(-f, -f), one2 = pair2(1.f, 1.f), up2 = pair2(12582920.f, 12582920.f);
  codes = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const uint64_t v = pair2(x[2 * i], x[2 * i + 1]);
    uint64_t y = mul_pair(v, inv2);
    y = fma_pair(fma_pair(y, f2, v), inv2, y);
    y = fma_pair(y, one2, up2);
    codes = (codes * 16u + static_cast<uint32_t>(y >> 32)) * 16u + static_cast<uint32_t>(y);
  }
  codes -= 0x4b400000u * 0x11111111u;            // the sums' upper bits; the codes are 1 .. 15
  return odd ? 255u : static_cast<uint32_t>(s);
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
