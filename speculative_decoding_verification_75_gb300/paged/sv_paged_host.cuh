// sv_paged_host.cuh -- what the entry points of the paged-cache operators share
// on the host: checks of a cache and of strides, launches, tensor maps.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda.h>

#include "sv_paged_common.cuh"

namespace svp {
namespace {

bool aligned(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

int elem_bytes(int64_t dtype) {
  return dtype == SV_F32 ? 4 : dtype == SV_BF16 || dtype == SV_F16 ? 2 : 0;
}

// Bits of a cache's element.
int cache_bits(int64_t dtype) {
  return dtype == SV_E4M3 ? 8 : dtype == SV_I4 ? 4 : 16;
}

// Whether a cache holds codes and scales, which any 16-bit query reads.
bool scaled(int64_t dtype) {
  return dtype == SV_E4M3 || dtype == SV_I4;
}

constexpr int64_t kMaxStride = int64_t{1} << 46;  // elements; far past any memory

// Checks a cache and its block tables (B rows) and lays it out in bytes.
sv_status take_cache(const sv_kv_cache &c, int64_t B, bool layered, Cache &o) {
  if (c.dtype != SV_BF16 && c.dtype != SV_F16 && !scaled(c.dtype))
    return SV_ERR_UNSUPPORTED_DTYPE;
  const bool codes = scaled(c.dtype);
  const int64_t bits = cache_bits(c.dtype);
  if (c.num_blocks < 0 || c.num_blocks > INT_MAX || c.num_kv_heads < 1 ||
      c.num_kv_heads > 65536 || c.block_size < 1 || c.block_size > (1 << 20) ||
      c.head_dim < 8 || c.head_dim > SV_KV_MAX_HEAD_DIM || c.head_dim % (codes ? 32 : 8) ||
      c.num_layers < 1 || c.num_layers > (layered ? 65536 : 1) || c.max_blocks < 0 ||
      c.max_blocks > INT_MAX)
    return SV_ERR_INVALID_ARG;
  const int64_t rows = c.num_kv_heads * c.block_size;
  if (rows * c.head_dim > INT_MAX || c.max_blocks * c.block_size > INT_MAX) return SV_ERR_INVALID_ARG;
  // A pool or a table may be empty (then every position is reported missing).
  if ((c.num_blocks > 0 && (!c.k || !c.v || (codes && (!c.k_scale || !c.v_scale)))) ||
      (c.max_blocks > 0 && B > 0 && !c.block_tables))
    return SV_ERR_INVALID_ARG;
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.block_tables, 4)) return SV_ERR_INVALID_ARG;
  const auto stride_ok = [](int64_t s, int64_t least, int64_t unit, bool used) {
    return !used || (s >= least && s <= kMaxStride && s % unit == 0);
  };
  const bool many = c.num_blocks > 1, deep = c.num_layers > 1;
  if (!stride_ok(c.block_stride, rows * c.head_dim, 128 / bits, many) ||
      !stride_ok(c.layer_stride, rows * c.head_dim, 128 / bits, deep))
    return SV_ERR_INVALID_ARG;
  if (codes) {
    if (!aligned(c.k_scale, 16) || !aligned(c.v_scale, 16) ||
        !stride_ok(c.scale_block_stride, rows * c.head_dim / SV_KV_GROUP, 1, many) ||
        !stride_ok(c.scale_layer_stride, rows * c.head_dim / SV_KV_GROUP, 1, deep))
      return SV_ERR_INVALID_ARG;
  }
  o.k = static_cast<uint8_t *>(c.k);
  o.v = static_cast<uint8_t *>(c.v);
  o.ks = codes ? c.k_scale : nullptr;
  o.vs = codes ? c.v_scale : nullptr;
  o.block_bytes = many ? c.block_stride / 8 * bits : 0;
  o.layer_bytes = deep ? c.layer_stride / 8 * bits : 0;
  o.sblock_bytes = codes && many ? c.scale_block_stride : 0;
  o.slayer_bytes = codes && deep ? c.scale_layer_stride : 0;
  o.tables = c.block_tables;
  o.num_layers = static_cast<int>(c.num_layers);
  o.num_blocks = static_cast<int>(c.num_blocks);
  o.heads = static_cast<int>(c.num_kv_heads);
  o.bs = static_cast<int>(c.block_size);
  o.D = static_cast<int>(c.head_dim);
  o.max_blocks = static_cast<int>(c.max_blocks);
  return SV_OK;
}

// Strides of a dense side [B, T, heads, D] with dense rows, in bytes.
bool take_strides(const int64_t (&s)[3], int esz, int64_t &b, int64_t &t, int64_t &h) {
  for (int64_t x : s)
    if (x < 0 || x > kMaxStride) return false;
  b = s[0] * esz;
  t = s[1] * esz;
  h = s[2] * esz;
  return true;
}

// Whether k and v are one array; false where their scales say otherwise.
bool one_array(const Cache &c, bool &same) {
  same = c.num_blocks > 0 && c.k == c.v;
  return !c.ks || c.num_blocks == 0 || (c.ks == c.vs) == same;
}

bool batch_ok(int64_t B, int64_t T) {
  return B >= 0 && T >= 0 && B <= INT_MAX && T <= INT_MAX && (B == 0 || T <= INT_MAX / B);
}

template <typename K, typename... P>
sv_status launch(K kernel, dim3 grid, int threads, size_t smem, sv_stream_t stream, const P &...p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p...) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

constexpr int kMaxDevices = 64;

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once per process.
EncodeTiled encode_tiled() {
  static std::atomic<void *> fn{nullptr};
  void *f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(f);
}

// A cache side as [block][head][row][element]; boxes of `box` rows, 128
// bytes wide for 16-bit types (swizzled, as the tensor cores read them), a
// whole row for codes (of 4 bits swizzled by its size, 64 or 32 bytes).
bool make_map(CUtensorMap &m, const Cache &c, const void *base, int64_t dtype, int box) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return false;
  const bool codes = scaled(dtype);
  const cuuint64_t bits = cache_bits(dtype), row = c.D * bits / 8, head = row * c.bs;
  const cuuint64_t dims[4] = {codes ? row : c.D, static_cast<cuuint64_t>(c.bs),
                              static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.num_blocks)};
  const cuuint64_t strides[3] = {row, head,
                                 c.block_bytes ? static_cast<cuuint64_t>(c.block_bytes) : head * c.heads};
  const cuuint32_t boxes[4] = {codes ? static_cast<cuuint32_t>(row) : 64u, static_cast<cuuint32_t>(box), 1, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return enc(&m,
             codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                : dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             4, const_cast<void *>(base), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             bits == 16 ? CU_TENSOR_MAP_SWIZZLE_128B
             : bits == 8 ? CU_TENSOR_MAP_SWIZZLE_NONE : row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace svp
