/*
 * sv_paged.h -- C ABI of the paged KV cache around the verification step:
 * part of libspecverify.so, with the conventions of spec_verify.h (device
 * pointers owned by the caller, nothing allocated, work enqueued on `stream`,
 * host-side argument checks before anything is enqueued, invalid data never
 * traps).
 *
 * The target model's side of one speculative step (P3 §5.4: the KV of the
 * drafted tokens is written first and marked tentative):
 *   sv_kv_write        the step's new tokens (the last emitted token and the
 *                      drafts, or a prompt) go into the cache, quantised if
 *                      the cache is e4m3;
 *   sv_tree_attention  every new token attends to the committed tokens and to
 *                      the new tokens that its tree mask names;
 *   spec_verify        accepts drafts (spec_verify.h);
 *   sv_kv_compact      the entries of an accepted tree path move together;
 *   sv_kv_rollback     cuts the sequence behind them (spec_verify.h);
 *   sv_kv_read         reads a sequence back as dense tensors.
 * The entries to keep are those of the last emitted token and of the accepted
 * drafts: where both were written in the step, sv_kv_compact and sv_kv_rollback
 * take spec_verify's num_accepted + 1 (0 for a request that it marked invalid),
 * and sv_kv_rollback's draft_lens are the new tokens, n.
 *
 * The cache.  k and v are arrays [num_layers][num_blocks][num_kv_heads]
 * [block_size][head_dim]; the innermost three dimensions are dense, blocks
 * and layers may be further apart (block_stride, layer_stride, in elements,
 * the same for k and v).  Position p of request b is row p % block_size of
 * block block_tables[b][p / block_size]; -1 is no block.  Element types:
 * SV_BF16, SV_F16, or SV_E4M3 with one scale byte s per 32 elements of
 * head_dim (k_scale, v_scale: [num_layers][num_blocks][num_kv_heads]
 * [block_size][head_dim / 32], E8M0: value = code * 2^(s - 127), 255 is NaN).
 * k and v do not overlap, or are one array for both, as are then the scales.
 * k, v and the scales start on 16-byte boundaries; block_stride and
 * layer_stride in bytes, scale_block_stride and scale_layer_stride are
 * multiples of 16 where they are used.
 *
 * Quantising.  For each 32 elements, e is the smallest whole number with
 * amax <= 448 * 2^e, at least -120, where amax is the largest finite
 * magnitude; s = e + 127, and a code is x / 2^e rounded to the nearest e4m3
 * (ties to even).  The scale is a power of two, so that the division is
 * exact and the only error is the code's rounding (2^-4 relative, or 2^(e-10)
 * for codes below 2^-6).  A value that is not finite becomes the NaN code.
 *
 * The batch.  seq_lens[b] = L is the number of committed tokens, new_lens[b]
 * = n in [0, T] (NULL: T) the number of new ones, which stand at positions
 * L .. L+n-1.  Rows i >= n of a request are not touched.
 *
 * Problems in the data set bits in the device word `status` (OR-ed; may be
 * NULL; the caller zeroes it) and never fault:
 *   SV_KV_BAD_LENGTH     L or n (or k, a start) out of range: the request is
 *                        skipped, its outputs are left as they were
 *   SV_KV_TABLE_SHORT    positions behind the table's max_blocks are skipped
 *                        (write, read) or not seen (attention)
 *   SV_KV_MISSING_BLOCK  positions whose block is -1: the same
 *   SV_KV_BAD_BLOCK      positions whose block is < -1 or >= num_blocks: the same
 *   SV_KV_BAD_PATH       a path that is not strictly increasing from >= 0:
 *                        the request is left unchanged
 * sv_kv_compact leaves a request unchanged on any of them.
 */
#ifndef SV_PAGED_H
#define SV_PAGED_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types besides SV_F32 and SV_BF16 of spec_verify.h. */
enum { SV_F16 = 2, SV_E4M3 = 3 };

/* Bits of `status` besides those of sv_kv_rollback. */
#define SV_KV_BAD_BLOCK 0x10u
#define SV_KV_BAD_PATH 0x20u

#define SV_KV_GROUP 32        /* elements that share a scale byte */
#define SV_KV_MAX_HEAD_DIM 256
#define SV_ATTN_MAX_KEYS 0x7ffff000  /* positions of a table, for attention */

/* Every field is 8 bytes wide. */
typedef struct {
    void *k, *v;
    uint8_t *k_scale, *v_scale;   /* SV_E4M3 only */
    int64_t layer_stride, block_stride;              /* elements */
    int64_t scale_layer_stride, scale_block_stride;  /* bytes; SV_E4M3 only */
    int64_t num_layers;           /* 1 unless the entry point says otherwise */
    int64_t num_blocks, num_kv_heads, block_size, head_dim;
    int64_t dtype;                /* SV_BF16, SV_F16 or SV_E4M3 */
    const int32_t *block_tables;  /* [B, max_blocks], dense */
    int64_t max_blocks;
} sv_kv_cache;

/*
 * New tokens into the cache.
 *   key, value [B, T, num_kv_heads, head_dim] of `dtype` (SV_BF16 or SV_F16;
 *   the cache's own type, or any of the two for SV_E4M3), head_dim dense, the
 *   other strides free (in elements: a view of a fused projection).
 * head_dim is a multiple of 8 (of 32 for SV_E4M3), at most 256.  No two
 * positions written by one call may share a cache row (two requests that
 * share a block hold it below both of their L).  Where k and v are one array,
 * so are key and value.
 */
typedef struct {
    uint64_t struct_bytes;        /* sizeof(sv_kv_write_args) */
    sv_kv_cache cache;            /* num_layers = 1 */
    const int32_t *seq_lens, *new_lens;
    const void *key, *value;
    int64_t key_stride[3], value_stride[3];  /* of b, t, head */
    int64_t B, T, dtype;
    uint32_t *status;
} sv_kv_write_args;
SV_API sv_status sv_kv_write(const sv_kv_write_args *args, sv_stream_t stream);

/*
 * Cached tokens as dense tensors: positions starts[b] + i (NULL: i) for
 * i < lens[b] go to key[b, i], value[b, i] ([B, T, num_kv_heads, head_dim] of
 * `dtype`: SV_BF16, SV_F16 or SV_F32, strides as in sv_kv_write; two tensors
 * that do not overlap).  Values of
 * an e4m3 cache are code * 2^(s-127) rounded to `dtype`, to nearest.
 */
typedef struct {
    uint64_t struct_bytes;
    sv_kv_cache cache;            /* num_layers = 1 */
    const int32_t *starts, *lens; /* [B]; starts may be NULL */
    void *key, *value;
    int64_t key_stride[3], value_stride[3];
    int64_t B, T, dtype;
    uint32_t *status;
} sv_kv_read_args;
SV_API sv_status sv_kv_read(const sv_kv_read_args *args, sv_stream_t stream);

/*
 * The accepted path of a tree, moved together in every layer: for i < k =
 * num_accepted[b] the entry at position seq_lens[b] + path[b, i] moves to
 * seq_lens[b] + i.  k counts entries: the accepted drafts and, where it is the
 * tree's node 0, the last emitted token.  path [B, P] holds strictly increasing
 * node numbers (a parent is numbered before its children), so path[b, i] >= i;
 * entries at i >= k are not read.  k <= 0 moves nothing, k > P is
 * SV_KV_BAD_LENGTH.  seq_lens is not changed: sv_kv_rollback does that.  Rows that are read or written must belong to one
 * request alone.
 */
typedef struct {
    uint64_t struct_bytes;
    sv_kv_cache cache;            /* any num_layers >= 1 */
    const int32_t *path, *num_accepted, *seq_lens;
    int64_t B, P;
    uint32_t *status;
} sv_kv_compact_args;
SV_API sv_status sv_kv_compact(const sv_kv_compact_args *args, sv_stream_t stream);

/*
 * Attention of the new tokens over the paged cache (which holds them already,
 * see sv_kv_write):
 *   out[b, i, h] = sum_j p_j v_j,  p = softmax over the visible positions j of
 *   scale * q[b, i, h] . k_j, with k, v of KV head h / (num_heads /
 *   num_kv_heads).
 * Visible to new token i of request b: every j < L, and j = L + c with c < n
 * and tree_mask[b, i, c] != 0 (no mask: c <= i, a chain or a prompt).  What is
 * not visible has no influence, whatever it holds.  A row that sees nothing,
 * or nothing but scores of -inf, is 0, its lse -inf.  A row that sees another
 * NaN or infinity follows the formula in IEEE arithmetic.
 *
 *   query     [B, T, num_heads, head_dim] of `dtype` (SV_BF16 or SV_F16; the
 *             cache's own type, or any of the two for SV_E4M3), strides as in
 *             sv_kv_write.  num_heads is a multiple of num_kv_heads.
 *   tree_mask [B, T, T] or NULL; rows of T bytes, dense; mask_batch_stride
 *             bytes between requests (0: one mask for all).
 *   out       [B, T, num_heads, head_dim] of `dtype`, dense, 16-byte aligned.
 *   lse       [B, T, num_heads] fp32 or NULL: the natural logarithm of the
 *             softmax's denominator (to merge with another cache's result).
 *   workspace sv_tree_attention_workspace_bytes() bytes, 256-byte aligned, no
 *             initialisation needed; calls that share one are ordered on one
 *             stream.
 * head_dim is a multiple of 8 (of 32 for SV_E4M3), at most 256, and max_blocks *
 * block_size at most SV_ATTN_MAX_KEYS.  Statistics and sums are fp32;
 * probabilities may be rounded to the query's type, over an e4m3 cache to fp16,
 * before their product with v; over an e4m3 cache elements of a bf16 query row
 * below 2^-31 of its largest may lose bits.  A bounded wait that gives up sets
 * SV_FAULT_TIMEOUT in `status`.  Results are deterministic.
 *
 * Fast for head_dim 64 and 128, block_size a multiple of 8 and query rows on
 * 16-byte boundaries; other batches take 25 to 200 times as long.  Rows of one
 * KV head and request (128 or 256 at a time) are computed at that rate too where
 * one of their blocks is missing, a new token's value is not finite, or, e4m3,
 * scales lie further apart than 2^15 (k: of 64 keys, v: below the first ones',
 * or 2^7 above); zeros with s = 7, as sv_kv_write leaves them, do not count.
 */
typedef struct {
    uint64_t struct_bytes;
    sv_kv_cache cache;            /* num_layers = 1 */
    const int32_t *seq_lens, *new_lens;
    const void *query;
    int64_t query_stride[3];      /* of b, t, head */
    const uint8_t *tree_mask;
    int64_t mask_batch_stride;
    void *out;
    float *lse;
    double scale;
    int64_t B, T, num_heads, dtype;
    void *workspace;
    uint64_t workspace_bytes;
    uint32_t *status;
} sv_tree_attention_args;
SV_API sv_status sv_tree_attention(const sv_tree_attention_args *args, sv_stream_t stream);

/* Workspace of sv_tree_attention: what it returns serves every smaller B, T,
 * num_heads and head_dim, and more KV heads (the cache's type and block size do
 * not matter); 0 for invalid sizes. */
SV_API size_t sv_tree_attention_workspace_bytes(int64_t B, int64_t T, int64_t num_heads,
                                                int64_t num_kv_heads, int64_t head_dim);

#ifdef __cplusplus
}
#endif

#endif /* SV_PAGED_H */
