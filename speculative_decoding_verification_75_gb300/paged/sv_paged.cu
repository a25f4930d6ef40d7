// sv_paged.cu -- C ABI of the paged-cache operators (include/sv_paged.h):
// argument checks, the choice of a kernel and the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "sv_paged.h"
#include "sv_paged_common.cuh"
#include "sv_paged_cache.cuh"
#include "sv_attn_general.cuh"
#include "sv_attn_tc.cuh"

namespace svp {
namespace {

bool aligned(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

int elem_bytes(int64_t dtype) {
  return dtype == SV_F32 ? 4 : dtype == SV_BF16 || dtype == SV_F16 ? 2 : dtype == SV_E4M3 ? 1 : 0;
}

constexpr int64_t kMaxStride = int64_t{1} << 46;  // elements; far past any memory

// Checks a cache and its block tables (B rows) and lays it out in bytes.
sv_status take_cache(const sv_kv_cache &c, int64_t B, bool layered, Cache &o) {
  if (c.dtype != SV_BF16 && c.dtype != SV_F16 && c.dtype != SV_E4M3)
    return SV_ERR_UNSUPPORTED_DTYPE;
  const bool f8 = c.dtype == SV_E4M3;
  const int64_t esz = elem_bytes(c.dtype);
  if (c.num_blocks < 0 || c.num_blocks > INT_MAX || c.num_kv_heads < 1 ||
      c.num_kv_heads > 65536 || c.block_size < 1 || c.block_size > (1 << 20) ||
      c.head_dim < 8 || c.head_dim > SV_KV_MAX_HEAD_DIM || c.head_dim % (f8 ? 32 : 8) ||
      c.num_layers < 1 || c.num_layers > (layered ? 65536 : 1) || c.max_blocks < 0 ||
      c.max_blocks > INT_MAX)
    return SV_ERR_INVALID_ARG;
  const int64_t rows = c.num_kv_heads * c.block_size;
  if (rows * c.head_dim > INT_MAX || c.max_blocks * c.block_size > INT_MAX) return SV_ERR_INVALID_ARG;
  // A pool or a table may be empty (then every position is reported missing).
  if ((c.num_blocks > 0 && (!c.k || !c.v || (f8 && (!c.k_scale || !c.v_scale)))) ||
      (c.max_blocks > 0 && B > 0 && !c.block_tables))
    return SV_ERR_INVALID_ARG;
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.block_tables, 4)) return SV_ERR_INVALID_ARG;
  const auto stride_ok = [](int64_t s, int64_t least, int64_t unit, bool used) {
    return !used || (s >= least && s <= kMaxStride && s % unit == 0);
  };
  const bool many = c.num_blocks > 1, deep = c.num_layers > 1;
  if (!stride_ok(c.block_stride, rows * c.head_dim, 16 / esz, many) ||
      !stride_ok(c.layer_stride, rows * c.head_dim, 16 / esz, deep))
    return SV_ERR_INVALID_ARG;
  if (f8) {
    if (!aligned(c.k_scale, 16) || !aligned(c.v_scale, 16) ||
        !stride_ok(c.scale_block_stride, rows * c.head_dim / SV_KV_GROUP, 1, many) ||
        !stride_ok(c.scale_layer_stride, rows * c.head_dim / SV_KV_GROUP, 1, deep))
      return SV_ERR_INVALID_ARG;
  }
  o.k = static_cast<uint8_t *>(c.k);
  o.v = static_cast<uint8_t *>(c.v);
  o.ks = f8 ? c.k_scale : nullptr;
  o.vs = f8 ? c.v_scale : nullptr;
  o.block_bytes = many ? c.block_stride * esz : 0;
  o.layer_bytes = deep ? c.layer_stride * esz : 0;
  o.sblock_bytes = f8 && many ? c.scale_block_stride : 0;
  o.slayer_bytes = f8 && deep ? c.scale_layer_stride : 0;
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

// The dense side of kv_write and kv_read and their grid.
sv_status take_move(MoveParams &p, const void *key, const void *value, const int64_t (&ks)[3],
                    const int64_t (&vs)[3], int64_t B, int64_t T, int esz, dim3 &grid) {
  if (!key || !value || !aligned(key, esz) || !aligned(value, esz)) return SV_ERR_INVALID_ARG;
  p.key = static_cast<uint8_t *>(const_cast<void *>(key));
  p.value = static_cast<uint8_t *>(const_cast<void *>(value));
  if (!take_strides(ks, esz, p.ksb, p.kst, p.ksh) || !take_strides(vs, esz, p.vsb, p.vst, p.vsh))
    return SV_ERR_INVALID_ARG;
  // Strides of dimensions of one element are never used.
  const int64_t used = (B > 1 ? p.ksb | p.vsb : 0) | (T > 1 ? p.kst | p.vst : 0) |
                       (p.c.heads > 1 ? p.ksh | p.vsh : 0);
  p.vec = aligned(key, 16) && aligned(value, 16) && used % 16 == 0;
  p.groups = static_cast<int>((T + kMoveTokens - 1) / kMoveTokens);
  const int64_t blocks = B * p.groups;
  const int64_t cols = 2ll * p.c.heads * (p.c.D / 8);
  const int64_t gy = (cols + kMoveThreads - 1) / kMoveThreads;
  if (blocks > INT_MAX || gy > 65535) return SV_ERR_INVALID_ARG;
  grid = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(gy));
  return SV_OK;
}

sv_status kv_write(const sv_kv_write_args *a, sv_stream_t stream) {
  if (!a || a->struct_bytes != sizeof *a || !batch_ok(a->B, a->T)) return SV_ERR_INVALID_ARG;
  if (a->dtype != SV_BF16 && a->dtype != SV_F16) return SV_ERR_UNSUPPORTED_DTYPE;
  MoveParams p = {};
  if (const sv_status s = take_cache(a->cache, a->B, false, p.c)) return s;
  if (a->cache.dtype != SV_E4M3 && a->cache.dtype != a->dtype) return SV_ERR_UNSUPPORTED_DTYPE;
  if (a->B == 0 || a->T == 0) return SV_OK;
  if (!a->seq_lens) return SV_ERR_INVALID_ARG;
  p.bt = Batch{a->seq_lens, a->new_lens, static_cast<int>(a->B), static_cast<int>(a->T), a->status};
  dim3 grid;
  if (const sv_status s = take_move(p, a->key, a->value, a->key_stride, a->value_stride, a->B,
                                    a->T, 2, grid))
    return s;
  bool same;
  if (!one_array(p.c, same) ||
      (same && (p.key != p.value || p.ksb != p.vsb || p.kst != p.vst || p.ksh != p.vsh)))
    return SV_ERR_INVALID_ARG;
  if (a->cache.dtype != SV_E4M3)  // a copy: the two 16-bit types are one
    return launch(sv_kv_write_kernel<BF16, BF16>, grid, kMoveThreads, 0, stream, p);
  return a->dtype == SV_BF16
             ? launch(sv_kv_write_kernel<BF16, E4M3>, grid, kMoveThreads, 0, stream, p)
             : launch(sv_kv_write_kernel<F16, E4M3>, grid, kMoveThreads, 0, stream, p);
}

template <typename C>
sv_status read_as(int64_t dtype, dim3 grid, sv_stream_t stream, const MoveParams &p) {
  if (dtype == SV_BF16) return launch(sv_kv_read_kernel<C, BF16>, grid, kMoveThreads, 0, stream, p);
  if (dtype == SV_F16) return launch(sv_kv_read_kernel<C, F16>, grid, kMoveThreads, 0, stream, p);
  return launch(sv_kv_read_kernel<C, F32>, grid, kMoveThreads, 0, stream, p);
}

sv_status kv_read(const sv_kv_read_args *a, sv_stream_t stream) {
  if (!a || a->struct_bytes != sizeof *a || !batch_ok(a->B, a->T)) return SV_ERR_INVALID_ARG;
  if (a->dtype != SV_BF16 && a->dtype != SV_F16 && a->dtype != SV_F32)
    return SV_ERR_UNSUPPORTED_DTYPE;
  MoveParams p = {};
  if (const sv_status s = take_cache(a->cache, a->B, false, p.c)) return s;
  if (a->B == 0 || a->T == 0) return SV_OK;
  if (!a->lens) return SV_ERR_INVALID_ARG;
  p.starts = a->starts;
  p.bt = Batch{nullptr, a->lens, static_cast<int>(a->B), static_cast<int>(a->T), a->status};
  dim3 grid;
  if (const sv_status s = take_move(p, a->key, a->value, a->key_stride, a->value_stride, a->B,
                                    a->T, elem_bytes(a->dtype), grid))
    return s;
  if (p.key == p.value) return SV_ERR_INVALID_ARG;
  if (a->cache.dtype == SV_BF16) return read_as<BF16>(a->dtype, grid, stream, p);
  if (a->cache.dtype == SV_F16) return read_as<F16>(a->dtype, grid, stream, p);
  return read_as<E4M3>(a->dtype, grid, stream, p);
}

sv_status kv_compact(const sv_kv_compact_args *a, sv_stream_t stream) {
  if (!a || a->struct_bytes != sizeof *a || !batch_ok(a->B, a->P)) return SV_ERR_INVALID_ARG;
  CompactParams p = {};
  if (const sv_status s = take_cache(a->cache, a->B, true, p.c)) return s;
  if (a->B == 0) return SV_OK;
  if (!a->num_accepted || !a->seq_lens || (a->P > 0 && !a->path)) return SV_ERR_INVALID_ARG;
  p.path = a->path;
  p.num_accepted = a->num_accepted;
  p.seq_lens = a->seq_lens;
  p.B = static_cast<int>(a->B);
  p.P = static_cast<int>(a->P);
  p.esz = elem_bytes(a->cache.dtype);
  p.status = a->status;
  bool same;
  if (!one_array(p.c, same)) return SV_ERR_INVALID_ARG;
  p.sides = same ? 1 : 2;
  const int64_t units = static_cast<int64_t>(p.sides) * p.c.heads * (p.c.D * p.esz / 16 + (p.esz == 1 ? p.c.D / SV_KV_GROUP : 0));
  // As many layers to a block as make all blocks run at once, four to an SM.
  const int64_t gy = (units + kMoveThreads - 1) / kMoveThreads;
  p.layers = static_cast<int>(std::max<int64_t>(
      std::min<int64_t>((a->B * p.c.num_layers * gy + 4 * kMaxGrid - 1) / (4 * kMaxGrid), p.c.num_layers), 1));
  p.groups = (p.c.num_layers + p.layers - 1) / p.layers;
  const int64_t blocks = a->B * p.groups;
  if (blocks > INT_MAX || gy > 65535) return SV_ERR_INVALID_ARG;
  return launch(sv_kv_compact_kernel,
                dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(gy)), kMoveThreads, 0,
                stream, p);
}

template <typename Q>
sv_status attn_general(int64_t cache_dtype, const AttnParams &p, sv_stream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.bt.B) * p.bt.T * p.Hq;
  if (rows > INT_MAX) return SV_ERR_INVALID_ARG;
  const dim3 grid(static_cast<unsigned>(rows));
  return cache_dtype == SV_E4M3
             ? launch(sv_attn_general_kernel<Q, E4M3>, grid, 32 * kGenWarps, 0, stream, p)
             : launch(sv_attn_general_kernel<Q, Q>, grid, 32 * kGenWarps, 0, stream, p);
}

// ------------------------------------------- tensor-core attention ----

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
// whole row for e4m3.
bool make_map(CUtensorMap &m, const Cache &c, const void *base, int64_t dtype, int box) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return false;
  const bool f8 = dtype == SV_E4M3;
  const cuuint64_t esz = f8 ? 1 : 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.bs),
                              static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.num_blocks)};
  const cuuint64_t row = c.D * esz, head = row * c.bs;
  const cuuint64_t strides[3] = {row, head,
                                 c.block_bytes ? static_cast<cuuint64_t>(c.block_bytes) : head * c.heads};
  const cuuint32_t boxes[4] = {f8 ? static_cast<cuuint32_t>(c.D) : 64u, static_cast<cuuint32_t>(box), 1, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return enc(&m,
             f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                : dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             4, const_cast<void *>(base), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             f8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as [request][token][head][element]; boxes of `tokens` tokens of
// the G heads that share a KV head, 64 elements wide.
bool make_query_map(CUtensorMap &m, const AttnParams &p, int64_t dtype, int tokens) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.c.D), static_cast<cuuint64_t>(p.Hq),
                              static_cast<cuuint64_t>(p.bt.T), static_cast<cuuint64_t>(p.bt.B)};
  const cuuint64_t row = p.c.D * 2;  // stands for strides that are never used
  const cuuint64_t strides[3] = {p.Hq > 1 ? static_cast<cuuint64_t>(p.qsh) : row,
                                 p.bt.T > 1 ? static_cast<cuuint64_t>(p.qst) : row,
                                 p.bt.B > 1 ? static_cast<cuuint64_t>(p.qsb) : row};
  const cuuint32_t boxes[4] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(tokens), 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return enc(&m, dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<uint8_t *>(p.q), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace of the tensor-core path.
struct TcLayout {
  size_t cuts, err, slots, total;
  int TT, MP, slot_rows, slot_floats;
};

TcLayout tc_layout(int64_t T, int64_t G, int64_t D) {
  const auto up = [](size_t x, size_t a) { return (x + a - 1) / a * a; };
  TcLayout w;
  w.TT = static_cast<int>(std::max<int64_t>(kTile / G, 1));  // tokens of a row tile
  const bool pair = T > w.TT;
  const int64_t unit = pair ? 2 * w.TT : w.TT;
  w.MP = static_cast<int>(std::max<int64_t>((T + unit - 1) / unit, 1));
  w.slot_rows = pair ? 2 * kTile
                     : static_cast<int>(up(std::min<int64_t>(std::max<int64_t>(T * G, 1), kTile), 32));
  // A pair's slot is two of a full single tile: a workspace for many tokens
  // serves few ones too.
  const auto slot = [&](int rows) { return static_cast<int>(up((D + 2) * rows + 1, 32)); };
  w.slot_floats = pair ? 2 * slot(kTile) : slot(w.slot_rows);
  w.cuts = 0;
  w.err = up(2 * kMaxGrid * sizeof(Cut), 256);
  w.slots = w.err + 256;
  w.total = w.slots + up(static_cast<size_t>(kMaxGrid) * (pair ? 1 : 2) * 2 * w.slot_floats * 4, 256);
  return w;
}

// Key tiles of a request whose table is full.
int64_t tc_tiles(const Cache &c) {
  return std::max<int64_t>((static_cast<int64_t>(c.max_blocks) * c.bs + kKeys - 1) / kKeys, 1);
}

// What the tensor-core kernel takes: whole 8-row swizzle atoms per page,
// query rows on 16-byte boundaries and a token's heads within a tile, sizes
// within TMA's and int32's.  It is
// the faster one at every size of these: one request of 500 keys 9 us, 33 by
// the general kernel; 8 of up to 4000 keys 28 and 827; 131071 keys 92 and 18377.
bool tc_takes(const sv_tree_attention_args *a, const AttnParams &p, const TcLayout &w) {
  if (p.c.D != 64 && p.c.D != 128) return false;
  if (p.c.bs % 8 || p.c.num_blocks < 1 || p.G > kTile || !p.qvec) return false;
  if (a->cache.dtype == SV_E4M3 && p.c.sblock_bytes % 16) return false;
  if (p.c.block_bytes >= (int64_t{1} << 40) || p.c.sblock_bytes > INT_MAX ||
      static_cast<int64_t>(p.c.heads) * p.c.bs * (p.c.D / SV_KV_GROUP) > INT_MAX)
    return false;
  const int64_t units = static_cast<int64_t>(p.bt.B) * p.c.heads * w.MP;
  return units <= INT_MAX / tc_tiles(p.c);
}

template <typename Q, typename C, int D, bool kPair>
sv_status tc_launch(const TcParams &p, int64_t units, int dev, sv_stream_t stream) {
  using S = Shape<Q, C, D, kPair>;
  static std::atomic<uint64_t> done{0};
  auto *k = sv_attn_tc_kernel<Q, C, D, kPair>;
  const uint64_t bit = 1ull << (dev % kMaxDevices);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) != cudaSuccess)
      return SV_ERR_CUDA;
    done.fetch_or(bit, std::memory_order_acq_rel);
  }
  if (const sv_status s = launch(k, dim3(static_cast<unsigned>(std::min(p.ranges, p.grid))), S::kThreads, S::kSmem,
                                 stream, p))
    return s;
  if (p.ranges < 2) return SV_OK;  // nothing is cut
  // Few units are cut into many parts: then more threads share an output, and
  // so do those of a block that would have none.
  const int outputs = std::min(p.a.bt.T, p.TT * S::kTilesPerUnit) * p.a.G * (D / 4 / kJoinCols);
  int K = 1;
  while (K < 8 && K * units <= p.ranges && (K * 4 * units <= p.ranges || outputs * 2 * K <= kJoinThreads)) K *= 2;
  const int per = kJoinThreads / K;
  return launch(sv_attn_join_kernel<Q, C, D, kPair>,
                dim3(static_cast<unsigned>(p.ranges - 1), static_cast<unsigned>((outputs + per - 1) / per)), kJoinThreads,
                0, stream, p, K);
}

template <typename Q, typename C>
sv_status tc_pick(const TcParams &p, bool pair, int64_t units, int dev, sv_stream_t stream) {
  if (p.a.c.D == 64)
    return pair ? tc_launch<Q, C, 64, true>(p, units, dev, stream) : tc_launch<Q, C, 64, false>(p, units, dev, stream);
  return pair ? tc_launch<Q, C, 128, true>(p, units, dev, stream) : tc_launch<Q, C, 128, false>(p, units, dev, stream);
}

sv_status attn_tc(const sv_tree_attention_args *a, const AttnParams &ap, const TcLayout &w,
                  sv_stream_t stream, bool *taken) {
  int dev = 0, nsm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SV_ERR_CUDA;
  TcParams p = {};
  p.a = ap;
  uint8_t *ws = static_cast<uint8_t *>(a->workspace);
  p.cuts = reinterpret_cast<Cut *>(ws + w.cuts);
  p.err = a->status ? a->status : reinterpret_cast<uint32_t *>(ws + w.err);
  p.slots = reinterpret_cast<float *>(ws + w.slots);
  p.slot_rows = w.slot_rows;
  p.slot_floats = w.slot_floats;
  const bool pair = ap.bt.T > w.TT;
  p.box = 8;  // a power of two that divides the block size, at most a stage
  while (p.box < kKeys && ap.c.bs % (2 * p.box) == 0) p.box *= 2;
  p.c = std::max(std::fabs(ap.scale_log2), kLeast);
  p.negate = ap.scale_log2 < 0.f;
  p.TT = w.TT;
  p.qbox = std::min(w.TT, ap.bt.T);
  *taken = make_map(p.kmap, ap.c, ap.c.k, a->cache.dtype, p.box) &&
           make_map(p.vmap, ap.c, ap.c.v, a->cache.dtype, p.box) &&
           make_query_map(p.qmap, ap, a->dtype, p.qbox);
  if (!*taken) return SV_OK;  // strides that no tensor map describes
  // At most one range per tile that the table has room for.
  const int64_t units = static_cast<int64_t>(ap.bt.B) * ap.c.heads * w.MP;
  const int64_t tiles = units * tc_tiles(ap.c);
  p.grid = std::min(nsm, kMaxGrid);
  p.ranges = static_cast<int>(std::min<int64_t>(p.grid * (pair ? 1 : 2), tiles));
  p.mvec = ap.mask && ap.bt.T % 4 == 0 && aligned(ap.mask, 4) && ap.msb % 4 == 0;
  if (a->cache.dtype == SV_E4M3)
    return a->dtype == SV_BF16 ? tc_pick<BF16, E4M3>(p, pair, units, dev, stream)
                               : tc_pick<F16, E4M3>(p, pair, units, dev, stream);
  return a->dtype == SV_BF16 ? tc_pick<BF16, BF16>(p, pair, units, dev, stream)
                             : tc_pick<F16, F16>(p, pair, units, dev, stream);
}

bool attn_sizes_ok(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D) {
  return batch_ok(B, T) && Hkv >= 1 && Hkv <= 65536 && Hq >= Hkv && Hq <= 65536 && Hq % Hkv == 0 &&
         D >= 8 && D <= SV_KV_MAX_HEAD_DIM && D % 8 == 0 && (B * T == 0 || Hq <= INT_MAX / (B * T));
}

sv_status tree_attention(const sv_tree_attention_args *a, sv_stream_t stream) {
  if (!a || a->struct_bytes != sizeof *a || !batch_ok(a->B, a->T)) return SV_ERR_INVALID_ARG;
  if (a->dtype != SV_BF16 && a->dtype != SV_F16) return SV_ERR_UNSUPPORTED_DTYPE;
  AttnParams p = {};
  if (const sv_status s = take_cache(a->cache, a->B, false, p.c)) return s;
  if (a->cache.dtype != SV_E4M3 && a->cache.dtype != a->dtype) return SV_ERR_UNSUPPORTED_DTYPE;
  if (!attn_sizes_ok(a->B, a->T, a->num_heads, p.c.heads, p.c.D) || !std::isfinite(a->scale) ||
      a->cache.max_blocks * a->cache.block_size > SV_ATTN_MAX_KEYS)  // a tile of keys ends below 2^31
    return SV_ERR_INVALID_ARG;
  const double sl2 = a->scale * 1.4426950408889634;
  if (std::fabs(sl2) > 3.4e38) return SV_ERR_INVALID_ARG;
  if (a->B == 0 || a->T == 0) return SV_OK;
  if (!a->seq_lens || !a->query || !a->out || !a->workspace) return SV_ERR_INVALID_ARG;
  if (!aligned(a->query, 2) || !aligned(a->out, 16) || !aligned(a->workspace, 256) ||
      !aligned(a->lse, 4) || a->mask_batch_stride < 0)
    return SV_ERR_INVALID_ARG;
  if (a->workspace_bytes < sv_tree_attention_workspace_bytes(a->B, a->T, a->num_heads, p.c.heads, p.c.D))
    return SV_ERR_WORKSPACE_TOO_SMALL;
  p.bt = Batch{a->seq_lens, a->new_lens, static_cast<int>(a->B), static_cast<int>(a->T), a->status};
  p.q = static_cast<const uint8_t *>(a->query);
  if (!take_strides(a->query_stride, 2, p.qsb, p.qst, p.qsh)) return SV_ERR_INVALID_ARG;
  const int64_t used = (a->B > 1 ? p.qsb : 0) | (a->T > 1 ? p.qst : 0) | (a->num_heads > 1 ? p.qsh : 0);
  p.qvec = aligned(a->query, 16) && used % 16 == 0;
  p.mask = a->tree_mask;
  p.msb = a->mask_batch_stride;
  p.out = static_cast<uint8_t *>(a->out);
  p.lse = a->lse;
  p.scale_log2 = static_cast<float>(sl2);
  p.Hq = static_cast<int>(a->num_heads);
  p.G = p.Hq / p.c.heads;
  const TcLayout w = tc_layout(a->T, p.G, p.c.D);
  if (tc_takes(a, p, w)) {
    bool taken = false;
    const sv_status s = attn_tc(a, p, w, stream, &taken);
    if (taken || s != SV_OK) return s;
  }
  return a->dtype == SV_BF16 ? attn_general<BF16>(a->cache.dtype, p, stream)
                             : attn_general<F16>(a->cache.dtype, p, stream);
}

}  // namespace
}  // namespace svp

extern "C" {

sv_status sv_kv_write(const sv_kv_write_args *args, sv_stream_t stream) {
  return svp::kv_write(args, stream);
}

sv_status sv_kv_read(const sv_kv_read_args *args, sv_stream_t stream) {
  return svp::kv_read(args, stream);
}

sv_status sv_kv_compact(const sv_kv_compact_args *args, sv_stream_t stream) {
  return svp::kv_compact(args, stream);
}

sv_status sv_tree_attention(const sv_tree_attention_args *args, sv_stream_t stream) {
  return svp::tree_attention(args, stream);
}

size_t sv_tree_attention_workspace_bytes(int64_t B, int64_t T, int64_t num_heads,
                                         int64_t num_kv_heads, int64_t head_dim) {
  if (!svp::attn_sizes_ok(B, T, num_heads, num_kv_heads, head_dim)) return 0;
  return svp::tc_layout(T, num_heads / num_kv_heads, head_dim).total;
}

}  // extern "C"
