// sv_paged_cache.cuh -- writing new tokens into the paged cache, reading
// sequences back, and moving an accepted tree path together.
//
// All three move bytes and compute next to nothing: long sequences are bound
// by HBM, a step's few tokens by the chain lengths -> block table -> data.
#pragma once

#include "sv_paged_common.cuh"

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

// Quantises 32 elements that 4 adjacent lanes hold (8 each); returns the
// scale byte.  Every lane of the warp takes part.  Magnitudes are compared as
// 16-bit integers, two at a time, and only a warp that meets an infinity or NaN
// looks at its elements one by one (8 prompts of up to 8192 tokens: 58 us, 5.3 TB/s;
// 68 us with comparisons of single fp32 magnitudes).
template <typename Q>
__device__ __forceinline__ uint32_t quantise8(const uint4 &raw, uint2 &codes) {
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
  constexpr uint32_t kInf = Q::kIsBf16 ? 0x7f80u : 0x7c00u;
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) big = __vmaxu2(big, u[i] & 0x7fff7fffu);
  big = max(big & 0xffffu, big >> 16);
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

// 16 bytes from the dense side, whatever its alignment (2-byte elements).
__device__ __forceinline__ uint4 load16(const uint8_t *s, bool vec) {
  if (vec) return ld128(s);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = ld16(s + 4 * k) | (ld16(s + 4 * k + 2) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// kv_write.  Q: type of the new tokens, C: the cache's.  Grid: (requests x
// token groups, column groups).
template <typename Q, typename C>
__global__ void __launch_bounds__(kMoveThreads) sv_kv_write_kernel(const MoveParams p) {
  __shared__ Slot slot[kMoveTokens];
  sv::pdl_wait();
  sv::pdl_launch_dependents();
  const int b = blockIdx.x / p.groups, t0 = (blockIdx.x - b * p.groups) * kMoveTokens;
  const int row_bytes = p.c.D * C::kBytes;
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
                 q.d8 * 8 * C::kBytes;
  const int srow = p.c.D / SV_KV_GROUP;
  uint8_t *dsc = C::kBytes == 1
                     ? (q.is_v ? p.c.vs : p.c.ks) + static_cast<int64_t>(q.h) * p.c.bs * srow + q.d8 / 4
                     : nullptr;
#pragma unroll
  for (int i = 0; i < kMoveTokens; ++i) {
    if (i >= cnt) break;  // the same for every thread
    const Slot s = slot[i];
    const bool put = q.on && s.data >= 0;
    if constexpr (C::kBytes == 1) {
      uint2 codes;
      const uint32_t sc = quantise8<Q>(raw[i], codes);
      if (put) {
        *reinterpret_cast<uint2 *>(dst + s.data) = codes;
        if ((q.d8 & 3) == 0) dsc[s.scale] = static_cast<uint8_t>(sc);
      }
    } else {
      if (put) *reinterpret_cast<uint4 *>(dst + s.data) = raw[i];
    }
  }
}

// kv_read.  C: the cache's type, O: the output's.
template <typename C, typename O>
__global__ void __launch_bounds__(kMoveThreads) sv_kv_read_kernel(const MoveParams p) {
  __shared__ Slot slot[kMoveTokens];
  sv::pdl_wait();
  sv::pdl_launch_dependents();
  const int b = blockIdx.x / p.groups, t0 = (blockIdx.x - b * p.groups) * kMoveTokens;
  const int row_bytes = p.c.D * C::kBytes;
  const int cnt = find_slots<true>(p, b, t0, row_bytes, slot);
  const Column q = column_of(p.c, blockIdx.y * kMoveThreads + threadIdx.x);
  __syncthreads();
  if (!q.on) return;
  const uint8_t *src = (q.is_v ? p.c.v : p.c.k) + static_cast<int64_t>(q.h) * p.c.bs * row_bytes +
                       q.d8 * 8 * C::kBytes;
  const int srow = p.c.D / SV_KV_GROUP;
  const uint8_t *ssc = C::kBytes == 1 ? (q.is_v ? p.c.vs : p.c.ks) +
                                            static_cast<int64_t>(q.h) * p.c.bs * srow + q.d8 / 4
                                      : nullptr;
  uint4 raw[kMoveTokens];
  uint32_t sc[kMoveTokens];
#pragma unroll
  for (int i = 0; i < kMoveTokens; ++i) {
    if (i < cnt && slot[i].data >= 0) {
      if constexpr (C::kBytes == 1) {
        const uint2 w = ld64(src + slot[i].data);
        raw[i] = make_uint4(w.x, w.y, 0, 0);
        sc[i] = ld8(ssc + slot[i].scale);
      } else {
        raw[i] = ld128(src + slot[i].data);
      }
    }
  }
  const int64_t step = q.is_v ? p.vst : p.kst;
  uint8_t *dst = (q.is_v ? p.value + b * p.vsb + q.h * p.vsh : p.key + b * p.ksb + q.h * p.ksh) +
                 t0 * step + q.d8 * 8 * O::kBytes;
#pragma unroll
  for (int i = 0; i < kMoveTokens; ++i) {
    if (i >= cnt) break;
    if (slot[i].data < 0) continue;
    float f[8];
    unpack8<C>(&raw[i], f);
    if constexpr (C::kBytes == 1) {
      const float m = scale_value(sc[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= m;
    }
    uint8_t *d = dst + i * step;
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
  int B, P, esz, sides;  // sides: 1 where k and v are one array
  int layers, groups;  // layers of a thread block, groups of them
  uint32_t *status;
};

constexpr int kPathChunk = 64;  // path entries looked up at once
constexpr int kPathBatch = 8;   // rows a thread holds between loads and stores

struct Move {
  int64_t from, to, sfrom, sto;  // byte offsets; from == to: nothing to do
};

__device__ __forceinline__ Move move_of(const CompactParams &p, int from, int from_pos, int to, int to_pos) {
  const Slot f = slot_at(p.c, from, from_pos, p.c.D * p.esz), t = slot_at(p.c, to, to_pos, p.c.D * p.esz);
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

  const int row_bytes = p.c.D * p.esz, per_head = row_bytes / 16, per_side = p.c.heads * per_head;
  const int srow = p.esz == 1 ? p.c.D / SV_KV_GROUP : 0, sper_side = p.c.heads * srow;
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
