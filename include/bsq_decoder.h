/*
 * bsq_decoder.h -- further entry points of libbsq_serving, those around the
 * cache and the experts of bsq_serving.h in a decoder's step: norms and
 * rotation of queries and keys, attention over the cache for trees of drafted
 * tokens and for windows with first tokens that stay visible, routing and the
 * grouped rows that the grouped quantizer and GEMM of bsq.h take, and log
 * probabilities of tokens.
 *
 * Conventions are those of bsq_serving.h, bsq_serving_last_error() included.
 */
#ifndef BSQ_DECODER_H
#define BSQ_DECODER_H

#include <stdint.h>

#include "bsq_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of inputs that may be either (any other value:
   BSQ_ERR_UNSUPPORTED). */
enum bsq_dtype { BSQ_BF16 = 0, BSQ_FP32 = 1 };

/*
 * Norms of queries and keys for each head, and their rotation by position, in
 * one pass over a projection's output:
 *
 *   y = x * w / sqrt(mean over the head of x^2 + eps)    (no weights: y = x)
 *   with a = positions[row] * inv_freq[i], for i < rotary_dim / 2:
 *   (out_p, out_r) = (y_p cos a - y_r sin a, y_r cos a + y_p sin a),
 *   p, r = i, i + rotary_dim / 2, or 2 i, 2 i + 1 with interleaved != 0;
 *   elements from rotary_dim on: out = y.
 *
 *   dtype         of q, k and v: BSQ_BF16 or BSQ_FP32 (what the GEMMs of
 *                 bsq.h write).  Outputs are BF16, rounded once.
 *   q, k          [num_rows][num_q_heads / num_heads][head_dim], ldq / ldk
 *                 elements from a row to the next (multiples of 8, so slices
 *                 of one projection's output do), 16-byte aligned.
 *   v, v_out      as k, rounded to BF16 only; or both NULL.
 *   head_dim      a multiple of 8, at most 256 (others: BSQ_ERR_UNSUPPORTED).
 *   q_weight, k_weight   fp32 [head_dim], or NULL: not normalised.
 *   eps           finite, >= 0.
 *   positions     int32 [num_rows]; rows that share a place (siblings in a
 *                 tree of drafted tokens) share their number.
 *   inv_freq      fp64 [rotary_dim / 2], radians a token.  The angle and its
 *                 reduction are computed in 64 bits.
 *   rotary_dim    0 (no rotation) or a multiple of 16 up to head_dim (others:
 *                 BSQ_ERR_UNSUPPORTED).
 *   num_q_heads, num_heads   1 .. 65535.
 * An output may be its BF16 input itself, with the same stride; else they may
 * not overlap.  Squares are summed in fp32.
 */
int qk_norm_rope(int dtype, const void* q, int64_t ldq, int64_t num_q_heads, const void* k,
                 int64_t ldk, int64_t num_heads, const void* v, int64_t ldv, int64_t head_dim,
                 int64_t num_rows, const float* q_weight, const float* k_weight, float eps,
                 const int32_t* positions, const double* inv_freq, int64_t rotary_dim,
                 int interleaved, void* q_out, int64_t ldqo, void* k_out, int64_t ldko, void* v_out,
                 int64_t ldvo, void* stream);

/*
 * kv_cache_attention (bsq_serving.h) with two more masks.  Of a sequence with
 * n rows and L tokens, the rows being its last tokens, base = L - n tokens
 * lie before them.
 *
 * masks NULL: row i is at place P = base + i and sees the tokens j <= P with
 *     j > P - window or j < sinks   (window 0: all of them).
 * masks given: the rows are nodes of a tree of drafted tokens.  Row i sees
 *     the rows (token base + x) whose bit x is set in its mask, bit x % 64 of
 *     word x / 64, itself only if its own is; and of the tokens before them
 *     j >= base - (window - c) or j < sinks   (window 0: all of them), where c
 *     is the number of rows it sees: base + c - 1 is then the place of the
 *     last node of a path of c.  Bits from n on are ignored.
 *
 *   masks         uint64 [num_rows][mask_words] without gaps, 8-byte aligned, or
 *                 NULL.  max_q is at most 64 * mask_words.
 *   window        0, or the number of tokens seen beside the sinks.
 *   sinks         first tokens that stay visible, 0 .. 2^31 - 1.
 * Pages of which no row sees a token are not read, and neither are their
 * table entries.  All else as for kv_cache_attention: rows that see nothing,
 * NaN scales, pages outside the cache, sums and their order, and the
 * workspace, of kv_cache_attention_masked_workspace(...) bytes (-1 for sizes
 * that the call would refuse).
 */
int kv_cache_attention_masked(const bsq_kv_cache* cache, const void* q, int64_t ldq,
                              int64_t num_q_heads, const uint32_t* row_offsets,
                              const int32_t* kv_lens, const int32_t* block_table,
                              int64_t table_stride, int64_t max_pages, int64_t num_seqs,
                              int64_t num_rows, int64_t max_q, int64_t max_kv, float scale,
                              int64_t window, int64_t sinks, const uint64_t* masks,
                              int64_t mask_words, void* out, int64_t ldo, float* lse,
                              void* workspace, int64_t workspace_bytes, void* stream);
int64_t kv_cache_attention_masked_workspace(int64_t num_heads, int64_t head_dim,
                                            int64_t num_q_heads, int64_t num_seqs,
                                            int64_t num_rows, int64_t max_q, int64_t max_kv,
                                            int64_t window, int64_t sinks);

#ifdef __cplusplus
}
#endif

#endif /* BSQ_DECODER_H */
