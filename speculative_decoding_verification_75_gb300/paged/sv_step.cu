// sv_step.cu -- C ABI of what a step does before its attention (include/sv_paged.h):
// places for the new tokens, and queries, keys and values on their way to them.
#include "sv_paged.h"
#include "sv_paged_host.cuh"
#include "sv_reserve.cuh"
#include "sv_rope.cuh"

namespace svp {
namespace {

sv_status kv_reserve(const sv_kv_reserve_args *a, sv_stream_t stream) {
  if (!a || a->struct_bytes != sizeof *a || !batch_ok(a->B, a->T)) return SV_ERR_INVALID_ARG;
  if (a->block_size < 1 || a->block_size > (1 << 20) || a->max_blocks < 0 || a->max_blocks > INT_MAX ||
      a->max_blocks * a->block_size > INT_MAX || a->free_capacity < 0 || a->free_capacity > INT_MAX ||
      a->mask_batch_stride < 0 || a->mask_batch_stride > kMaxStride ||
      a->B > int64_t{kReserveCluster} * kReserveRequests)
    return SV_ERR_INVALID_ARG;
  if (a->B == 0) return SV_OK;
  if (!a->seq_lens || !a->free_count || !a->reserved || (a->max_blocks > 0 && !a->block_tables) ||
      (a->free_capacity > 0 && !a->free_list) || (a->T > 0 && (!a->slots || !a->positions)))
    return SV_ERR_INVALID_ARG;
  if (!aligned(a->seq_lens, 4) || !aligned(a->new_lens, 4) || !aligned(a->block_tables, 4) ||
      !aligned(a->free_list, 4) || !aligned(a->free_count, 4) || !aligned(a->reserved, 4) ||
      !aligned(a->slots, 8) || !aligned(a->positions, 4))
    return SV_ERR_INVALID_ARG;
  ReserveParams p = {};
  p.seq_lens = a->seq_lens;
  p.new_lens = a->new_lens;
  p.free_list = a->free_list;
  p.tables = a->block_tables;
  p.free_count = a->free_count;
  p.positions = a->positions;
  p.reserved = a->reserved;
  p.slots = a->slots;
  p.mask = a->tree_mask;
  p.msb = a->mask_batch_stride;
  p.B = static_cast<int>(a->B);
  p.T = static_cast<int>(a->T);
  p.max_blocks = static_cast<int>(a->max_blocks);
  p.bs = static_cast<int>(a->block_size);
  p.capacity = static_cast<int>(a->free_capacity);
  p.mvec = a->T % 4 == 0 && aligned(a->tree_mask, 4) && a->mask_batch_stride % 4 == 0;
  p.status = a->status;
  // A lane for each entry that a request may lack, 32 at most; as many thread blocks
  // as give each lane one request.
  const int64_t entries = std::min<int64_t>(a->T / a->block_size + 2, 32);
  p.lanes = 1;
  while (p.lanes < entries) p.lanes *= 2;
  int ranks = 1;
  while (ranks < kReserveCluster && ranks * (kReserveThreads / p.lanes) < p.B) ranks *= 2;
  while (ranks < kReserveCluster && (p.B + ranks - 1) / ranks > kReserveRequests) ranks *= 2;
  const int64_t tokens = a->B * a->T;
  p.per = (p.B + ranks - 1) / ranks;
  p.fused = tokens <= static_cast<int64_t>(kReserveThreads * ranks * (p.mask ? kFusedNodes : kFusedTokens));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kReserveThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.per) * sizeof(int2);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, sv_reserve_kernel, p) != cudaSuccess) return SV_ERR_CUDA;
  if (p.fused) return SV_OK;
  return launch(sv_place_kernel, dim3(static_cast<unsigned>((tokens + kReserveThreads - 1) / kReserveThreads)),
                kReserveThreads, 0, stream, p);
}

template <typename Q, typename C>
sv_status rope_as(bool pairs, unsigned grid, sv_stream_t stream, const RopeParams &p) {
  return pairs ? launch(sv_rope_kernel<Q, C, true>, dim3(grid), kRopeThreads, 0, stream, p)
               : launch(sv_rope_kernel<Q, C, false>, dim3(grid), kRopeThreads, 0, stream, p);
}

template <typename Q>
sv_status rope_into(int64_t cache, bool pairs, unsigned grid, sv_stream_t stream, const RopeParams &p) {
  if (cache == SV_E4M3) return rope_as<Q, E4M3>(pairs, grid, stream, p);
  if (cache == SV_I4) return rope_as<Q, I4>(pairs, grid, stream, p);
  return rope_as<Q, Q>(pairs, grid, stream, p);
}

sv_status qk_norm_rope(const sv_qk_norm_rope_args *a, sv_stream_t stream) {
  if (!a || a->struct_bytes != sizeof *a || !batch_ok(a->B, a->T)) return SV_ERR_INVALID_ARG;
  if (a->dtype != SV_BF16 && a->dtype != SV_F16) return SV_ERR_UNSUPPORTED_DTYPE;
  const int64_t D = a->head_dim, R = a->rotary_dim;
  if (a->num_heads < 0 || a->num_heads > 65536 || a->num_kv_heads < 0 || a->num_kv_heads > 65536 || D < 8 ||
      D > SV_KV_MAX_HEAD_DIM || D % 8 || R < 0 || R > D || R % (a->interleaved ? 2 : 16) || a->num_positions < 0 ||
      a->num_positions > INT_MAX || !(a->eps >= 0) || !(a->eps <= 1e30))
    return SV_ERR_INVALID_ARG;
  RopeParams p = {};
  const bool cached = a->slots != nullptr;
  if (cached) {
    sv_kv_cache c = a->cache;
    c.block_tables = nullptr;
    c.max_blocks = 0;
    if (const sv_status s = take_cache(c, 0, false, p.c)) return s;
    if (!scaled(a->cache.dtype) && a->cache.dtype != a->dtype) return SV_ERR_UNSUPPORTED_DTYPE;
    if (a->cache.num_kv_heads != a->num_kv_heads || a->cache.head_dim != D) return SV_ERR_INVALID_ARG;
    bool same;  // keys turn, values do not
    if (!one_array(p.c, same) || same) return SV_ERR_INVALID_ARG;
  }
  if (a->B == 0 || a->T == 0) return SV_OK;
  const bool any_q = a->num_heads > 0, any_k = a->num_kv_heads > 0;
  if (!a->positions || (R > 0 && !a->cos_sin) || (any_q && (!a->query || !a->out)) ||
      (any_k && (!a->key || (cached ? !a->value : !a->key_out))))
    return SV_ERR_INVALID_ARG;
  const void *const rows[] = {a->query, a->key, cached ? a->value : nullptr, a->out, a->key_out};
  bool vec = true;
  for (const void *x : rows) {
    if (!aligned(x, 2)) return SV_ERR_INVALID_ARG;
    vec = vec && aligned(x, 16);
  }
  // In place, or apart: other threads still read what a result written elsewhere covers.
  const auto apart = [&](const void *x, const int64_t (&sx)[3], const void *y, const int64_t (&sy)[3], int64_t heads) {
    return x != y || ((a->B == 1 || sx[0] == sy[0]) && (a->T == 1 || sx[1] == sy[1]) && (heads == 1 || sx[2] == sy[2]));
  };
  if ((any_q && !apart(a->out, a->out_stride, a->query, a->query_stride, a->num_heads)) ||
      (any_k && a->key_out && !apart(a->key_out, a->key_out_stride, a->key, a->key_stride, a->num_kv_heads)) ||
      (any_q && any_k && (a->out == a->key || a->out == a->key_out || a->key_out == a->query)) ||
      (cached && any_k && ((any_q && a->out == a->value) || a->key_out == a->value)))
    return SV_ERR_INVALID_ARG;
  // Vectors of four angles, where a lane's eight are adjacent.
  if (!aligned(a->positions, 4) || !aligned(a->slots, 8) || !aligned(a->cos_sin, a->interleaved ? 4 : 16) ||
      !aligned(a->q_weight, 16) || !aligned(a->k_weight, 16))
    return SV_ERR_INVALID_ARG;
  p.q = static_cast<const uint8_t *>(a->query);
  p.k = static_cast<const uint8_t *>(a->key);
  p.v = static_cast<const uint8_t *>(a->value);
  p.qo = static_cast<uint8_t *>(a->out);
  p.ko = static_cast<uint8_t *>(a->key_out);
  int64_t used = 0;
  const auto strides = [&](const int64_t (&s)[3], int64_t heads, int64_t &sb, int64_t &st, int64_t &sh) {
    if (!take_strides(s, 2, sb, st, sh)) return false;
    used |= (a->B > 1 ? sb : 0) | (a->T > 1 ? st : 0) | (heads > 1 ? sh : 0);
    return true;
  };
  if ((any_q && (!strides(a->query_stride, a->num_heads, p.qsb, p.qst, p.qsh) ||
                 !strides(a->out_stride, a->num_heads, p.qosb, p.qost, p.qosh))) ||
      (any_k && (!strides(a->key_stride, a->num_kv_heads, p.ksb, p.kst, p.ksh) ||
                 (cached && !strides(a->value_stride, a->num_kv_heads, p.vsb, p.vst, p.vsh)) ||
                 (a->key_out && !strides(a->key_out_stride, a->num_kv_heads, p.kosb, p.kost, p.kosh)))))
    return SV_ERR_INVALID_ARG;
  p.vec = vec && used % 16 == 0;
  p.qw = static_cast<const uint8_t *>(a->q_weight);
  p.kw = static_cast<const uint8_t *>(a->k_weight);
  p.cos_sin = a->cos_sin;
  p.positions = a->positions;
  p.slots = a->slots;
  p.eps = static_cast<float>(a->eps);
  p.root_eps = static_cast<float>(std::sqrt(a->eps));
  p.least = p.eps < kLeastEps ? kLeastSquares : 0.f;
  p.B = static_cast<int>(a->B);
  p.T = static_cast<int>(a->T);
  p.Hq = static_cast<int>(a->num_heads);
  p.Hkv = static_cast<int>(a->num_kv_heads);
  p.D = static_cast<int>(D);
  p.inv_d = 1.f / static_cast<float>(D);
  p.R = static_cast<int>(R);
  p.P = static_cast<int>(a->num_positions);
  p.status = a->status;
  p.lanes = 1;
  while (p.lanes < D / 8) p.lanes *= 2;
  // Steps of whole rows of a kind; a warp's: as many as leave kRopeWarps warps, rounded
  // down and then to whole turns of kRopeRows.  (128 x 6 tokens of 40 steps: 8 of 8.4, 3840
  // warps, 9.7 us; rounded up 10, fewer than kRopeWarps warps, 10.7 us.)
  const int group = 32 / p.lanes;
  p.steps_q = (p.Hq + group - 1) / group;
  p.steps_k = (p.Hkv + group - 1) / group;
  p.steps = p.steps_q + p.steps_k * (cached ? 2 : 1);
  if (p.steps == 0) return SV_OK;
  const int64_t tokens = a->B * a->T;
  int64_t per = std::min<int64_t>(std::max<int64_t>(tokens * p.steps / kRopeWarps, 1), p.steps);
  if (per > kRopeRows) per = (per + kRopeRows - 1) / kRopeRows * kRopeRows;
  p.per = static_cast<int>(per);
  p.runs = (p.steps + p.per - 1) / p.per;
  const int64_t blocks = (tokens * p.runs + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (blocks > INT_MAX) return SV_ERR_INVALID_ARG;
  const int64_t cache = cached ? a->cache.dtype : a->dtype;
  const unsigned grid = static_cast<unsigned>(blocks);
  return a->dtype == SV_BF16 ? rope_into<BF16>(cache, a->interleaved != 0, grid, stream, p)
                             : rope_into<F16>(cache, a->interleaved != 0, grid, stream, p);
}

}  // namespace
}  // namespace svp

extern "C" {

sv_status sv_kv_reserve(const sv_kv_reserve_args *args, sv_stream_t stream) {
  return svp::kv_reserve(args, stream);
}

sv_status sv_qk_norm_rope(const sv_qk_norm_rope_args *args, sv_stream_t stream) {
  return svp::qk_norm_rope(args, stream);
}

}  // extern "C"
