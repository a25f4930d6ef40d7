// sv_paged_common.cuh -- what the paged-cache kernels share: the cache's
// layout, page lookups, the batch's lengths and the 8-element vector of each
// element type.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "sv_paged.h"

// The verification kernels' device helpers, with internal linkage: this is
// the library's second translation unit that compiles them.
namespace {
#include "sv_device.cuh"
}

namespace svp {

using sv::kFull;

// Element tags.  kScaled: codes, with a scale byte for SV_KV_GROUP of them.
// Eight elements take kBits bytes.
struct BF16 { using raw = __nv_bfloat16; static constexpr int kBits = 16, kBytes = 2; static constexpr bool kIsBf16 = true, kScaled = false; };
struct F16 { using raw = __half; static constexpr int kBits = 16, kBytes = 2; static constexpr bool kIsBf16 = false, kScaled = false; };
struct F32 { using raw = float; static constexpr int kBits = 32, kBytes = 4; };
struct E4M3 { using raw = uint8_t; static constexpr int kBits = 8, kBytes = 1; static constexpr bool kScaled = true; };
struct I4 { using raw = uint8_t; static constexpr int kBits = 4; static constexpr bool kScaled = true; };

struct Cache {
  uint8_t *k, *v;
  uint8_t *ks, *vs;               // scale bytes or NULL
  int64_t layer_bytes, block_bytes, slayer_bytes, sblock_bytes;
  const int32_t *tables;
  int num_layers, num_blocks, heads, bs, D, max_blocks;
};

struct Batch {
  const int32_t *seq_lens, *new_lens;
  int B, T;
  uint32_t *status;
};

// Loads that stay behind griddepcontrol.wait: the kernel before may still be
// writing until then, and a load through the read-only path could be moved.
__device__ __forceinline__ int ld32(const int32_t *p) {
  int v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld16(const void *p) {
  uint16_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld8(const void *p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld128(const void *p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld64(const void *p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
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
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Eight elements as they lie in the cache, in the vector's first kBits bytes.
template <typename C>
__device__ __forceinline__ uint4 load8(const void *p) {
  if constexpr (C::kBits == 4) {
    return make_uint4(static_cast<uint32_t>(ld32(static_cast<const int32_t *>(p))), 0, 0, 0);
  } else if constexpr (C::kBits == 8) {
    const uint2 w = ld64(p);
    return make_uint4(w.x, w.y, 0, 0);
  } else {
    return ld128(p);
  }
}

__device__ __forceinline__ void report(uint32_t *status, uint32_t bits) {
  if (status && bits) atomicOr(status, bits);
}

// Block of position `pos` of request b, or -1 with the reason in `st`.
__device__ __forceinline__ int block_of(const Cache &c, int b, int pos, uint32_t &st) {
  const int j = pos / c.bs;
  if (j >= c.max_blocks) {
    st |= SV_KV_TABLE_SHORT;
    return -1;
  }
  const int id = ld32(c.tables + static_cast<size_t>(b) * c.max_blocks + j);
  if (id >= 0 && id < c.num_blocks) return id;
  st |= id == -1 ? SV_KV_MISSING_BLOCK : SV_KV_BAD_BLOCK;
  return -1;
}

// Committed and new tokens of request b; false (nothing to do) where they
// are out of range.  L + n stays below 2^31.
__device__ __forceinline__ bool lengths(const Batch &bt, int b, int &L, int &n, uint32_t &st) {
  L = ld32(bt.seq_lens + b);
  n = bt.new_lens ? ld32(bt.new_lens + b) : bt.T;
  if (L < 0 || n < 0 || n > bt.T || L > 0x7fffffff - n) {
    st |= SV_KV_BAD_LENGTH;
    n = 0;
    return false;
  }
  return true;
}

// A scale byte's value.
template <typename C>
__device__ __forceinline__ float scale_value(uint32_t s);

// 2^(s - 127), with E8M0's NaN at 255.
template <>
__device__ __forceinline__ float scale_value<E4M3>(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7fc00000u : s << 23);
}

// 2^(s / 8 - 14) * (1 + s % 8 / 8): the byte is the exponent and three fraction
// bits of a float, moved by 113.
template <>
__device__ __forceinline__ float scale_value<I4>(uint32_t s) {
  return __uint_as_float(s > SV_KV_I4_MAX_SCALE ? 0x7fc00000u : (s << 20) + (113u << 23));
}

// Eight elements as fp32.
template <typename E>
__device__ __forceinline__ void unpack8(const void *p, float (&f)[8]);

template <>
__device__ __forceinline__ void unpack8<BF16>(const void *p, float (&f)[8]) {
  const uint4 w = *reinterpret_cast<const uint4 *>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = sv::bf16_lo(u[i]);
    f[2 * i + 1] = sv::bf16_hi(u[i]);
  }
}

template <>
__device__ __forceinline__ void unpack8<F16>(const void *p, float (&f)[8]) {
  const uint4 w = *reinterpret_cast<const uint4 *>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

template <>
__device__ __forceinline__ void unpack8<E4M3>(const void *p, float (&f)[8]) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(u[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

template <>
__device__ __forceinline__ void unpack8<I4>(const void *p, float (&f)[8]) {
  const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float((w >> (4 * i) & 15u) | 0x4b000000u) - 8388616.f;   // 2^23 + c
}

template <typename E>
__device__ __forceinline__ void pack8(void *p, const float (&f)[8]);

template <>
__device__ __forceinline__ void pack8<BF16>(void *p, const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

template <>
__device__ __forceinline__ void pack8<F16>(void *p, const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

template <>
__device__ __forceinline__ void pack8<F32>(void *p, const float (&f)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

template <typename E>
__device__ __forceinline__ float load1(const void *p);
template <>
__device__ __forceinline__ float load1<BF16>(const void *p) {
  return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(p));
}
template <>
__device__ __forceinline__ float load1<F16>(const void *p) {
  return __half2float(*reinterpret_cast<const __half *>(p));
}

template <typename E>
__device__ __forceinline__ void store1(void *p, float x);
template <>
__device__ __forceinline__ void store1<BF16>(void *p, float x) {
  *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ void store1<F16>(void *p, float x) {
  *reinterpret_cast<__half *>(p) = __float2half_rn(x);
}
template <>
__device__ __forceinline__ void store1<F32>(void *p, float x) {
  *reinterpret_cast<float *>(p) = x;
}

}  // namespace svp
