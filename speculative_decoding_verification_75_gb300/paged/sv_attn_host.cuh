// sv_attn_host.cuh -- what the tensor-core attention kernels share on the host:
// the workspace, a kernel's shared memory, the launch of the second kernel.
#pragma once

#include "sv_attn_tc.cuh"
#include "sv_paged_host.cuh"

namespace svp {

// The kernel for caches of 4 bits (sv_attn_i4.cu): takes the call, or leaves it to
// the general kernel.
sv_status attn_i4(const sv_tree_attention_args *a, const AttnParams &ap, sv_stream_t stream, bool *taken);

namespace {

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
int64_t tc_tiles(const Cache &c, int keys = kKeys) {
  return std::max<int64_t>((static_cast<int64_t>(c.max_blocks) * c.bs + keys - 1) / keys, 1);
}

// Allows a kernel its dynamic shared memory, once per device.
template <typename K>
bool shared_memory(K kernel, int bytes, int dev, std::atomic<uint64_t> &done) {
  const uint64_t bit = 1ull << (dev % kMaxDevices);
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_acq_rel);
  return true;
}

// Joins the units that range ends cut; a unit has `rows` rows at most.
template <typename Q, typename C, int D, bool kPair>
sv_status join_launch(const TcParams &p, int rows, int64_t units, sv_stream_t stream) {
  if (p.ranges < 2) return SV_OK;  // nothing is cut
  // Few units are cut into many parts: then more threads share an output, and
  // so do those of a block that would have none.
  const int outputs = rows * (D / 4 / kJoinCols);
  int K = 1;
  while (K < 8 && K * units <= p.ranges && (K * 4 * units <= p.ranges || outputs * 2 * K <= kJoinThreads)) K *= 2;
  const int per = kJoinThreads / K;
  return launch(sv_attn_join_kernel<Q, C, D, kPair>,
                dim3(static_cast<unsigned>(p.ranges - 1), static_cast<unsigned>((outputs + per - 1) / per)), kJoinThreads,
                0, stream, p, K);
}

}  // namespace
}  // namespace svp
