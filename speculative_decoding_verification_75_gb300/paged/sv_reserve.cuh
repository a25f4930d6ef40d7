// sv_reserve.cuh -- places for a step's new tokens: blocks from the free list
// into the block tables, and each new token's slot and position.
//
// Request b lacks need_b blocks: the entries [ceil(L / bs), ceil((L + n) / bs)) of
// its table that are -1.  Requests are served in order: b gets its blocks where the
// sum of the needs up to it is at most the number of free blocks, and the blocks
// are numbered by request and position, so that results do not depend on timing.
//
// Bound by latencies (lengths -> table -> sum over the requests -> free list ->
// table -> slots): one launch, whose thread blocks form one cluster and exchange
// their sums through shared memory, and which also places the tokens while its threads
// have few; else a second kernel on all SMs does.  In a graph of calls: 8 requests of 6
// tokens 3.0 us, 256 trees of 64 nodes 7.6 us (38 us by the one kernel).
#pragma once

#include "sv_paged_common.cuh"

namespace svp {

constexpr int kReserveThreads = 512;
constexpr int kReserveCluster = 8;        // thread blocks at most
constexpr int kReserveRequests = 4096;    // of a thread block
// Tokens of a thread, at most, where the same kernel places them: one kernel against two
// takes 3.0 and 3.9 us for 48 tokens, 3.7 and 4.5 for 2 on each thread, 4.5 for 4, 6.1 and
// 4.8 for 8; of trees, whose nodes read a row of the mask each, 3.4 and 4.3 us for 48, 4.4
// and 4.8 for 1.5, 7.7 and 6.6 for 2 (of 64 nodes), 5.5 and 5.1 for 3 (of 6).
constexpr float kFusedTokens = 4, kFusedNodes = 1.5f;

struct ReserveParams {
  const int32_t *seq_lens, *new_lens, *free_list;
  int32_t *tables, *free_count, *positions, *reserved;
  int64_t *slots;
  const uint8_t *mask;                    // NULL: a chain
  int64_t msb;                            // bytes between requests
  int B, T, max_blocks, bs, capacity;
  int per, lanes;                         // requests of a thread block; lanes that share one
  int fused;                              // slots and positions by the same kernel
  int mvec;                               // mask rows are whole 4-byte words
  uint32_t *status;
};

// New token i of a request with n places behind L committed tokens.
__device__ __forceinline__ void place(const ReserveParams &p, int b, int i, int L, int n) {
  int64_t slot = -1;
  int at = 0;
  if (i < n) {
    const int pos = L + i, j = pos / p.bs;
    const int id = ld32(p.tables + static_cast<size_t>(b) * p.max_blocks + j);
    if (id >= 0) slot = static_cast<int64_t>(id) * p.bs + (pos - j * p.bs);
    at = pos;
    if (p.mask) {                         // the number of visible tokens: ancestors and itself
      const uint8_t *row = p.mask + b * p.msb + static_cast<int64_t>(i) * p.T;
      int seen = 0;
      if (p.mvec) {
#pragma unroll 4
        for (int c = 0; c < n; c += 4) {
          uint32_t v = static_cast<uint32_t>(ld32(reinterpret_cast<const int32_t *>(row + c)));
          if (n - c < 4) v &= (1u << (8 * (n - c))) - 1u;
          seen += __popc((((v & 0x7f7f7f7fu) + 0x7f7f7f7fu) | v) & 0x80808080u);
        }
      } else {
#pragma unroll 4
        for (int c = 0; c < n; ++c) seen += ld8(row + c) != 0;
      }
      at = L + max(seen - 1, 0);
    }
  }
  const size_t o = static_cast<size_t>(b) * p.T + i;
  p.slots[o] = slot;
  p.positions[o] = at;
}

// Committed and new tokens of request b and the entries [j0, j1) of its table that
// the new ones need.  False where nothing can be reserved.
__device__ __forceinline__ bool wanted(const ReserveParams &p, int b, int &L, int &n, int &j0, int &j1, uint32_t &st) {
  L = ld32(p.seq_lens + b);
  n = p.new_lens ? ld32(p.new_lens + b) : p.T;
  j0 = j1 = 0;
  if (L < 0 || n < 0 || n > p.T || L > 0x7fffffff - n) {
    st |= SV_KV_BAD_LENGTH;
    return false;
  }
  const auto blocks = [&](int x) { return x / p.bs + (x % p.bs ? 1 : 0); };
  j0 = blocks(L);
  j1 = blocks(L + n);
  if (n > 0 && j1 > p.max_blocks) {
    j1 = j0;
    st |= SV_KV_TABLE_SHORT;
    return false;
  }
  return true;
}

__global__ void __launch_bounds__(kReserveThreads) sv_reserve_kernel(const ReserveParams p) {
  extern __shared__ int2 req[];           // need, then the tokens reserved; blocks before it
  __shared__ int sums[kReserveCluster];   // of the cluster's thread blocks
  __shared__ int warp_sums[kReserveThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.x), ranks = static_cast<int>(gridDim.x);
  const int b0 = rank * p.per, cnt = max(min(p.per, p.B - b0), 0);
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  sv::pdl_wait();
  sv::pdl_launch_dependents();
  const int count = min(max(ld32(p.free_count), 0), p.capacity);
  const int groups = kReserveThreads / p.lanes, group = tid / p.lanes, sub = tid & (p.lanes - 1);
  uint32_t st = 0;

  // What each request lacks.
  for (int base = 0; base < cnt; base += groups) {
    const int r = base + group, b = b0 + r;
    int need = 0;
    bool ok = false;
    if (r < cnt) {
      int L, n, j0, j1;
      uint32_t mine = 0;
      ok = wanted(p, b, L, n, j0, j1, mine);
      const int32_t *row = p.tables + static_cast<size_t>(b) * p.max_blocks;
      if (ok && n > 0 && L % p.bs) {      // the last committed tokens' block
        const int id = ld32(row + j0 - 1);
        if (id < 0) mine |= id == -1 ? SV_KV_MISSING_BLOCK : SV_KV_BAD_BLOCK;
      }
#pragma unroll 4
      for (int j = j0 + sub; j < j1; j += p.lanes) {
        const int id = ld32(row + j);
        need += id == -1;
        if (id < -1) mine |= SV_KV_BAD_BLOCK;
      }
      ok = mine == 0;
      st |= mine;
    }
    int bad = ok ? 0 : 1;
    for (int o = 1; o < p.lanes; o <<= 1) {
      need += __shfl_xor_sync(kFull, need, o);
      bad |= __shfl_xor_sync(kFull, bad, o);
    }
    if (r < cnt && sub == 0) req[r] = make_int2(bad ? -1 : need, 0);
  }
  __syncthreads();

  // Blocks before each request, in order.
  int total = 0;
  for (int base = 0; base < cnt; base += kReserveThreads) {
    const int r = base + tid, need = r < cnt ? max(req[r].x, 0) : 0;
    int incl = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kReserveThreads / 32; ++w) {
      before += w < warp ? warp_sums[w] : 0;
      all += warp_sums[w];
    }
    if (r < cnt) req[r].y = total + before + incl - need;
    total += all;
    __syncthreads();
  }
  int first = 0;
  if (ranks > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // every peer has begun
    if (tid < ranks) {
      uint32_t at;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(sv::smem_addr(&sums[rank])), "r"(tid));
      asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(at), "r"(total) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int i = 0; i < rank; ++i) first += sums[i];
  }

  // Blocks for those that get them.
  int taken = 0;                          // blocks up to the last request served
  for (int base = 0; base < cnt; base += groups) {
    const int r = base + group, b = b0 + r;
    int need = 0, at = 0, j0 = 0, j1 = 0, n = 0;
    if (r < cnt) {
      const int2 q = req[r];
      int L;
      uint32_t none = 0;
      need = q.x;
      at = first + q.y;
      if (need >= 0) wanted(p, b, L, n, j0, j1, none);
      if (need > 0 && need > count - at) {
        st |= SV_KV_NO_BLOCKS;
        need = -1;
      }
      if (need > 0) taken = at + need;
    }
    const int32_t *row = p.tables + static_cast<size_t>(r < cnt ? b : 0) * p.max_blocks;
    const int steps = need > 0 ? (j1 - j0 + p.lanes - 1) / p.lanes : 0;
    const int most = __reduce_max_sync(kFull, steps);
    for (int k = 0; k < most; ++k) {
      const int j = j0 + k * p.lanes + sub;
      const bool lacks = k < steps && j < j1 && ld32(row + j) == -1;
      const uint32_t same = __ballot_sync(kFull, lacks) >> (lane - sub) & (p.lanes == 32 ? kFull : (1u << p.lanes) - 1u);
      if (lacks) {
        const int i = at + __popc(same & ((1u << sub) - 1u));
        p.tables[static_cast<size_t>(b) * p.max_blocks + j] = ld32(p.free_list + (count - 1 - i));
      }
      at += __popc(same);
    }
    __syncwarp();
    if (r < cnt && sub == 0) {
      req[r].x = need >= 0 ? n : 0;
      p.reserved[b] = need >= 0 ? n : 0;
    }
  }
  // Every thread block has read the number of free blocks by now.
  taken = __reduce_max_sync(kFull, taken);
  if (lane == 0 && taken > 0) atomicMin(p.free_count, count - taken);
  report(p.status, st);
  if (!p.fused) return;
  __syncthreads();
  for (int k = tid; k < cnt * p.T; k += kReserveThreads) {
    const int r = k / p.T;
    place(p, b0 + r, k - r * p.T, ld32(p.seq_lens + b0 + r), req[r].x);
  }
}

// The same places by as many thread blocks as there are tokens for.
__global__ void __launch_bounds__(kReserveThreads) sv_place_kernel(const ReserveParams p) {
  sv::pdl_wait();
  sv::pdl_launch_dependents();
  const int64_t k = static_cast<int64_t>(blockIdx.x) * kReserveThreads + threadIdx.x;
  if (k >= static_cast<int64_t>(p.B) * p.T) return;
  const int b = static_cast<int>(k / p.T);
  place(p, b, static_cast<int>(k - static_cast<int64_t>(b) * p.T), ld32(p.seq_lens + b), ld32(p.reserved + b));
}

}  // namespace svp
