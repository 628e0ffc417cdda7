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

#ifdef __cplusplus
}
#endif

#endif /* BSQ_DECODER_H */
