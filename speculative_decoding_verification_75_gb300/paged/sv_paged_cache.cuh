// sv_paged_cache.cuh -- writing new tokens into the paged cache, reading
// sequences back, and moving an accepted tree path together.
//
// All three move bytes and compute next to nothing: long sequences are bound
// by HBM, a step's few tokens by the chain lengths -> block table -> data.
#pragma once

#include "sv_paged_quant.cuh"

namespace svp {

constexpr int kMoveThreads = 256;
// Tokens a thread block handles at once: a thread owns one 8-element column
// (of one head of k or v) and keeps its loads for all of them in flight.
constexpr int kMoveTokens = 8;

struct MoveParams {
  Cache c;
  Batch bt;                              // read: new_lens are the lengths
  const int32_t *starts;                 // read: first positions, may be NULL
  uint8_t *key, *value;                  // dense side
  int64_t ksb, kst, ksh, vsb, vst, vsh;  // its strides in bytes
  int groups;                            // token groups of a request
  int vec;                               // dense side on 16-byte boundaries
};

// Byte offsets of a token's row of head 0 in the cache and in the scales;
// data < 0 marks a token that has no place.
struct Slot {
  int64_t data, scale;
};

__device__ __forceinline__ Slot slot_at(const Cache &c, int id, int pos, int row_bytes) {
  const int r = pos % c.bs;
  Slot s;
  s.data = id < 0 ? -1 : id * c.block_bytes + static_cast<int64_t>(r) * row_bytes;
  s.scale = id < 0 ? -1 : id * c.sblock_bytes + static_cast<int64_t>(r) * (c.D / SV_KV_GROUP);
  return s;
}

// Looks up the block's tokens (its first threads do); returns how many it has.
template <bool kRead>
__device__ __forceinline__ int find_slots(const MoveParams &p, int b, int t0, int row_bytes,
                                          Slot *slot) {
  uint32_t st = 0;
  int L = 0, n = 0;
  if (kRead) {
    n = ld32(p.bt.new_lens + b);
    L = p.starts ? ld32(p.starts + b) : 0;
    if (L < 0 || n < 0 || n > p.bt.T || L > 0x7fffffff - n) {
      st = SV_KV_BAD_LENGTH;
      n = 0;
    }
  } else {
    lengths(p.bt, b, L, n, st);
  }
  const int cnt = min(max(n - t0, 0), kMoveTokens);
  const int i = threadIdx.x;
  if (i < cnt) {
    const int pos = L + t0 + i;
    slot[i] = slot_at(p.c, block_of(p.c, b, pos, st), pos, row_bytes);
  }
  if (i < kMoveTokens) report(p.bt.status, st);
  return cnt;
}

// What a thread moves: side (k or v), head and 8-element column.
struct Column {
  bool on, is_v;
  int h, d8;
};

__device__ __forceinline__ Column column_of(const Cache &c, int i) {
  const int per_head = c.D / 8, per_side = c.heads * per_head;
  Column q;
  q.on = i < 2 * per_side;
  q.is_v = q.on && i >= per_side;
  const int cc = q.on ? i - (q.is_v ? per_side : 0) : 0;
  q.h = cc / per_head;
  q.d8 = cc - q.h * per_head;
  return q;
}

// kv_write.  Q: type of the new tokens, C: the cache's.  Grid: (requests x
// token groups, column groups).
template <typename Q, typename C>
__global__ void __launch_bounds__(kMoveThreads) sv_kv_write_kernel(const MoveParams p) {
  __shared__ Slot slot[kMoveTokens];
  sv::pdl_wait();
  sv::pdl_launch_dependents();
  const int b = blockIdx.x / p.groups, t0 = (blockIdx.x - b * p.groups) * kMoveTokens;
  const int row_bytes = p.c.D / 8 * C::kBits;
  const int cnt = find_slots<false>(p, b, t0, row_bytes, slot);
  const Column q = column_of(p.c, blockIdx.y * kMoveThreads + threadIdx.x);
  const int64_t step = q.is_v ? p.vst : p.kst;
  const uint8_t *src = (q.is_v ? p.value + b * p.vsb + q.h * p.vsh : p.key + b * p.ksb + q.h * p.ksh) +
                       t0 * step + q.d8 * 16;
  uint4 raw[kMoveTokens];
#pragma unroll
  for (int i = 0; i < kMoveTokens; ++i)
    raw[i] = q.on && i < cnt ? load16(src + i * step, p.vec) : make_uint4(0, 0, 0, 0);
  __syncthreads();
  uint8_t *dst = (q.is_v ? p.c.v : p.c.k) + static_cast<int64_t>(q.h) * p.c.bs * row_bytes +
                 q.d8 * C::kBits;
  const int srow = p.c.D / SV_KV_GROUP;
  uint8_t *dsc = C::kScaled
                     ? (q.is_v ? p.c.vs : p.c.ks) + static_cast<int64_t>(q.h) * p.c.bs * srow + q.d8 / 4
                     : nullptr;
  if constexpr (C::kBits == 4) {
#pragma unroll
    for (int i = 0; i < kMoveTokens; i += 4) {
      if (i >= cnt) break;  // the same for every thread
      uint32_t codes[4];
      const uint32_t sc = quantise4x8<Q>(raw + i, codes);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!q.on || i + j >= cnt) continue;
        const int64_t at = slot[i + j].data;
        if (at >= 0) *reinterpret_cast<uint32_t *>(dst + at) = codes[j];
      }
      const int mine = i + (threadIdx.x & 3);
      if (q.on && mine < cnt && slot[mine].scale >= 0) dsc[slot[mine].scale] = static_cast<uint8_t>(sc);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kMoveTokens; ++i) {
      if (i >= cnt) break;  // the same for every thread
      const Slot s = slot[i];
      const bool put = q.on && s.data >= 0;
      if constexpr (C::kScaled) {
        typename Codes<C>::type codes;
        const uint32_t sc = quantise8<Q>(raw[i], codes);
        if (put) {
          *reinterpret_cast<typename Codes<C>::type *>(dst + s.data) = codes;
          if ((q.d8 & 3) == 0) dsc[s.scale] = static_cast<uint8_t>(sc);
        }
      } else {
        if (put) *reinterpret_cast<uint4 *>(dst + s.data) = raw[i];
      }
    }
  }
}

// Eight 4-bit codes times their scale as 16-bit numbers, exactly: a code's bits are a
// fraction of 64 (bf16: 16), pairs are 16 bits apart.  (8 x 16000 tokens to bf16: 85 us,
// 5.9 TB/s, HBM; 92 us through fp32.)
template <typename O>
__device__ __forceinline__ uint4 values8(uint32_t w, uint32_t s) {
  const uint32_t sv2 = s > SV_KV_I4_MAX_SCALE ? 0x7fff7fffu : O::kIsBf16 ? s * 0x00100010u + 0x38803880u : s * 0x00800080u + 0x04000400u;
  constexpr uint32_t mask = O::kIsBf16 ? 0x00780078u : 0x00f000f0u, base = O::kIsBf16 ? 0x41804180u : 0x54005400u;
  uint32_t y[4];                                   // elements i and i + 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int up = (O::kIsBf16 ? 3 : 4) - 4 * i;
    const uint32_t x = up > 0 ? w << up : w >> -up;
    uint32_t u;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(u) : "r"(x), "n"(mask), "r"(base));
    if constexpr (O::kIsBf16) {
      asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(u) : "r"(u), "r"(0xc1c0c1c0u));     // - 24
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y[i]) : "r"(u), "r"(sv2));
    } else {
      asm("add.rn.f16x2 %0, %1, %2;" : "=r"(u) : "r"(u), "r"(0xd480d480u));      // - 72
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y[i]) : "r"(u), "r"(sv2));
    }
  }
  return make_uint4(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410), __byte_perm(y[0], y[1], 0x7632),
                    __byte_perm(y[2], y[3], 0x7632));
}

// kv_read.  C: the cache's type, O: the output's.
template <typename C, typename O>
__global__ void __launch_bounds__(kMoveThreads) sv_kv_read_kernel(const MoveParams p) {
  __shared__ Slot slot[kMoveTokens];
  sv::pdl_wait();
  sv::pdl_launch_dependents();
  const int b = blockIdx.x / p.groups, t0 = (blockIdx.x - b * p.groups) * kMoveTokens;
  const int row_bytes = p.c.D / 8 * C::kBits;
  const int cnt = find_slots<true>(p, b, t0, row_bytes, slot);
  const Column q = column_of(p.c, blockIdx.y * kMoveThreads + threadIdx.x);
  __syncthreads();
  if (!q.on) return;
  const uint8_t *src = (q.is_v ? p.c.v : p.c.k) + static_cast<int64_t>(q.h) * p.c.bs * row_bytes +
                       q.d8 * C::kBits;
  const int srow = p.c.D / SV_KV_GROUP;
  const uint8_t *ssc = C::kScaled ? (q.is_v ? p.c.vs : p.c.ks) +
                                            static_cast<int64_t>(q.h) * p.c.bs * srow + q.d8 / 4
                                      : nullptr;
  uint4 raw[kMoveTokens];
  uint32_t sc[kMoveTokens];
#pragma unroll
  for (int i = 0; i < kMoveTokens; ++i) {
    if (i < cnt && slot[i].data >= 0) {
      raw[i] = load8<C>(src + slot[i].data);
      if constexpr (C::kScaled) sc[i] = ld8(ssc + slot[i].scale);
    }
  }
  const int64_t step = q.is_v ? p.vst : p.kst;
  uint8_t *dst = (q.is_v ? p.value + b * p.vsb + q.h * p.vsh : p.key + b * p.ksb + q.h * p.ksh) +
                 t0 * step + q.d8 * 8 * O::kBytes;
#pragma unroll
  for (int i = 0; i < kMoveTokens; ++i) {
    if (i >= cnt) break;
    if (slot[i].data < 0) continue;
    uint8_t *d = dst + i * step;
    if constexpr (C::kBits == 4 && O::kBits == 16) {
      if (p.vec) {
        *reinterpret_cast<uint4 *>(d) = values8<O>(raw[i].x, sc[i]);
        continue;
      }
    }
    float f[8];
    unpack8<C>(&raw[i], f);
    if constexpr (C::kScaled) {
      const float m = scale_value<C>(sc[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= m;
    }
    if (p.vec) {
      pack8<O>(d, f);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) store1<O>(d + k * O::kBytes, f[k]);
    }
  }
}

// ------------------------------------------------------------- compaction ----
struct CompactParams {
  Cache c;
  const int32_t *path, *num_accepted, *seq_lens;
  int B, P, bits, sides;  // bits of an element; sides: 1 where k and v are one array
  int layers, groups;  // layers of a thread block, groups of them
  uint32_t *status;
};

constexpr int kPathChunk = 64;  // path entries looked up at once
constexpr int kPathBatch = 8;   // rows a thread holds between loads and stores

struct Move {
  int64_t from, to, sfrom, sto;  // byte offsets; from == to: nothing to do
};

__device__ __forceinline__ Move move_of(const CompactParams &p, int from, int from_pos, int to, int to_pos) {
  const int row_bytes = p.c.D / 8 * p.bits;
  const Slot f = slot_at(p.c, from, from_pos, row_bytes), t = slot_at(p.c, to, to_pos, row_bytes);
  return Move{f.data, t.data, f.scale, t.scale};
}

template <typename V>
__device__ __forceinline__ void move_rows(uint8_t *base, const Move *mv, int cnt, bool scales) {
  for (int i0 = 0; i0 < cnt; i0 += kPathBatch) {
    V w[kPathBatch];
#pragma unroll
    for (int i = 0; i < kPathBatch; ++i)
      if (i0 + i < cnt)
        w[i] = *reinterpret_cast<const V *>(base + (scales ? mv[i0 + i].sfrom : mv[i0 + i].from));
#pragma unroll
    for (int i = 0; i < kPathBatch; ++i)
      if (i0 + i < cnt)
        *reinterpret_cast<V *>(base + (scales ? mv[i0 + i].sto : mv[i0 + i].to)) = w[i];
  }
}

// Grid: (requests x groups of layers, column groups).  A thread moves the same 16
// bytes of every row of the path, in path order and in batches that are read
// before they are written.  The path increases strictly from >= 0, so
// path[i] >= i: a row that a batch writes is read by no later entry, and by
// an earlier one only in this batch or before, by the same thread.
//
// Bound by latencies: lengths, path, table, rows.  The first three are the same
// in every layer, so a block moves several where there are more blocks than run
// at once (32 layers of 64 requests: 16.6 us with four, 18.1 with one, 18.8 with
// eight).
__global__ void __launch_bounds__(kMoveThreads, 4) sv_kv_compact_kernel(const CompactParams p) {
  __shared__ Move mv[kPathChunk];
  sv::pdl_wait();
  sv::pdl_launch_dependents();
  const int b = blockIdx.x / p.groups, l0 = (blockIdx.x - b * p.groups) * p.layers;
  const int l1 = min(l0 + p.layers, p.c.num_layers);
  const int L = ld32(p.seq_lens + b), k = ld32(p.num_accepted + b);
  if (k <= 0) return;
  const int32_t *path = p.path + static_cast<int64_t>(b) * p.P;
  // The whole path is checked before anything moves; its first rows are looked
  // up on the way.
  uint32_t st = 0;
  if (L < 0 || k > p.P) {
    st = SV_KV_BAD_LENGTH;
  } else {
    for (int i = threadIdx.x; i < k; i += kMoveThreads) {
      const int a = ld32(path + i), before = i ? ld32(path + i - 1) : -1;
      if (a <= before || a < 0) st |= SV_KV_BAD_PATH;
      else if (a > 0x7fffffff - L) st |= SV_KV_BAD_LENGTH;
      else {
        const int ib = block_of(p.c, b, L + a, st), jb = block_of(p.c, b, L + i, st);
        if (i < kPathChunk) mv[i] = move_of(p, ib, L + a, jb, L + i);
      }
    }
  }
  if (blockIdx.y == 0 && l0 == 0) report(p.status, st);
  if (__syncthreads_or(static_cast<int>(st))) return;

  const int row_bytes = p.c.D / 8 * p.bits, per_head = row_bytes / 16, per_side = p.c.heads * per_head;
  const int srow = p.bits < 16 ? p.c.D / SV_KV_GROUP : 0, sper_side = p.c.heads * srow;
  const int u = blockIdx.y * kMoveThreads + threadIdx.x;
  const bool data = u < p.sides * per_side, scales = !data && u - p.sides * per_side < p.sides * sper_side;
  uint8_t *base = nullptr;
  if (data) {
    const bool is_v = u >= per_side;
    const int cc = u - (is_v ? per_side : 0), h = cc / per_head;
    base = (is_v ? p.c.v : p.c.k) +
           static_cast<int64_t>(h) * p.c.bs * row_bytes + (cc - h * per_head) * 16;
  } else if (scales) {
    const int s = u - p.sides * per_side;
    const bool is_v = s >= sper_side;
    const int cc = s - (is_v ? sper_side : 0), h = cc / srow;
    base = (is_v ? p.c.vs : p.c.ks) +
           static_cast<int64_t>(h) * p.c.bs * srow + (cc - h * srow);
  }
  for (int i0 = 0; i0 < k; i0 += kPathChunk) {
    const int cnt = min(k - i0, kPathChunk);
    if (i0 > 0) {
      __syncthreads();
      if (threadIdx.x < cnt) {
        const int i = i0 + threadIdx.x, a = ld32(path + i);
        uint32_t none = 0;
        const int ib = block_of(p.c, b, L + a, none), jb = block_of(p.c, b, L + i, none);
        mv[threadIdx.x] = move_of(p, ib, L + a, jb, L + i);
      }
      __syncthreads();
    }
    // Entries that are in place already come first (path[i] == i holds for a
    // prefix, since the path increases strictly).
    int first = 0;
    while (first < cnt && mv[first].from == mv[first].to) ++first;
    for (int layer = l0; layer < l1; ++layer) {
      if (data) move_rows<uint4>(base + layer * p.c.layer_bytes, mv + first, cnt - first, false);
      if (scales) move_rows<uint8_t>(base + layer * p.c.slayer_bytes, mv + first, cnt - first, true);
    }
  }
}

}  // namespace svp
