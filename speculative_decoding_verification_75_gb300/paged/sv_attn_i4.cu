// sv_attn_i4.cu -- launches of tree attention over a cache of 4 bits.
#include "sv_attn_host.cuh"
#include "sv_attn_i4.cuh"

namespace svp {
namespace {

template <typename Q, int D>
sv_status i4_launch(const TcParams &p, int64_t units, int dev, sv_stream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto *k = i4::sv_attn_i4_kernel<Q, D>;
  constexpr int smem = i4::Shape<D>::kSmem;
  if (!shared_memory(k, smem, dev, done)) return SV_ERR_CUDA;
  if (const sv_status s = launch(k, dim3(static_cast<unsigned>(p.ranges)), i4::kThreads, smem, stream, p)) return s;
  return join_launch<Q, I4, D, false>(p, p.unit_rows, units, stream);
}

}  // namespace

sv_status attn_i4(const sv_tree_attention_args *a, const AttnParams &ap, sv_stream_t stream, bool *taken) {
  *taken = false;
  const Cache &c = ap.c;
  // Whole swizzle atoms of rows per page, scales of 4 keys on 16-byte boundaries,
  // query rows too, sizes within TMA's and int32's.
  if ((c.D != 64 && c.D != 128) || c.bs % 8 || c.num_blocks < 1 || !ap.qvec || c.sblock_bytes % 16 ||
      c.block_bytes >= (int64_t{1} << 40))
    return SV_OK;
  // Rows of a request and KV head in equal units, whole steps of N.
  const int64_t rows = static_cast<int64_t>(ap.bt.T) * ap.G;
  const int64_t parts = (rows + i4::kRows - 1) / i4::kRows;
  const int64_t units = static_cast<int64_t>(ap.bt.B) * c.heads * parts;
  const int64_t most = tc_tiles(c, i4::kT);
  if (units > INT_MAX / most) return SV_OK;
  int dev = 0, nsm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SV_ERR_CUDA;
  TcParams p = {};
  p.a = ap;
  p.unit_rows = static_cast<int>(((rows + parts - 1) / parts + i4::kUnit - 1) / i4::kUnit * i4::kUnit);
  // The workspace of the wider rows of the other types, which has room for these.
  const TcLayout w = tc_layout(a->T, ap.G, c.D);
  uint8_t *ws = static_cast<uint8_t *>(a->workspace);
  p.cuts = reinterpret_cast<Cut *>(ws + w.cuts);
  p.err = a->status ? a->status : reinterpret_cast<uint32_t *>(ws + w.err);
  p.slots = reinterpret_cast<float *>(ws + w.slots);
  p.slot_rows = p.unit_rows;
  p.slot_floats = ((c.D + 2) * p.slot_rows + 1 + 31) / 32 * 32;
  p.box = 8;  // a power of two that divides the block size, at most a tile
  while (p.box < i4::kT && c.bs % (2 * p.box) == 0) p.box *= 2;
  if (!make_map(p.kmap, c, c.k, SV_I4, p.box) || !make_map(p.vmap, c, c.v, SV_I4, p.box)) return SV_OK;
  p.c = std::max(std::fabs(ap.scale_log2), kLeast);
  p.negate = ap.scale_log2 < 0.f;
  // Scores are taken in units of kUndo: an infinite factor would make NaN of those of 0.
  if (a->dtype == SV_F16 && !std::isfinite(p.c * i4::kUndo<F16>)) return SV_OK;
  *taken = true;
  p.grid = std::min(nsm, kMaxGrid);
  p.ranges = static_cast<int>(std::min<int64_t>(p.grid, units * most));
  if (static_cast<size_t>(p.ranges) * 2 * p.slot_floats * 4 > w.total - w.slots) return SV_ERR_WORKSPACE_TOO_SMALL;
  if (a->dtype == SV_BF16)
    return c.D == 64 ? i4_launch<BF16, 64>(p, units, dev, stream) : i4_launch<BF16, 128>(p, units, dev, stream);
  return c.D == 64 ? i4_launch<F16, 64>(p, units, dev, stream) : i4_launch<F16, 128>(p, units, dev, stream);
}

}  // namespace svp
