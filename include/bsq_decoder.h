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
 * workspace, of kv_cache_attention_masked_workspace(...) bytes (mask_words 0
 * without masks; -1 for sizes that the call would refuse).
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
                                            int64_t window, int64_t sinks, int64_t mask_words);

/*
 * Experts of each token from a router's logits z, and their weights.
 *
 *   s = softmax(z) (BSQ_SCORE_SOFTMAX) or 1 / (1 + exp(-z)) (BSQ_SCORE_SIGMOID)
 *   c = s + bias   (the bias takes part in the choice alone)
 *   of num_groups groups of num_experts / num_groups consecutive experts, the
 *     topk_groups with the largest sum of their group_top (1 or 2) largest c
 *     are kept;
 *   the topk largest c of the kept groups' experts are chosen, the largest
 *     first; equal groups and experts go by their number, the lower first;
 *   weight = factor * s, with renormalize != 0 divided by the sum of the
 *     chosen s.
 *
 * The choice is that of c in 64-bit arithmetic: values that 32 bits cannot
 * tell apart are computed again.  (Without a bias c goes by z, and z is
 * compared instead, but for sums of two.)  A logit of -inf or NaN, or a bias
 * of -inf or NaN, makes c -inf: chosen only where nothing else is left, with
 * weight 0.  Under softmax a logit of +inf takes the whole score, shared with
 * its equals.  Where the chosen s are all 0, so are the weights.
 *
 *   dtype         of the logits [num_tokens][num_experts], ldl elements from
 *                 a row to the next, aligned to their size.
 *   num_experts   1 .. 1024;  topk 1 .. 16 and at most the experts kept.
 *   bias          fp32 [num_experts], or NULL.
 *   num_groups    1 .. 64, a divisor of num_experts;  topk_groups 1 ..
 *                 num_groups.  group_top above a group's size counts as it.
 *   factor        finite.
 *   topk_ids, topk_weights   int32 / fp32 [num_tokens][topk], as
 *                 moe_few_tokens takes them.
 */
enum bsq_score { BSQ_SCORE_SOFTMAX = 0, BSQ_SCORE_SIGMOID = 1 };
int moe_route(int dtype, const void* logits, int64_t ldl, int64_t num_tokens, int64_t num_experts,
              int64_t topk, int score, const float* bias, int64_t num_groups, int64_t topk_groups,
              int group_top, int renormalize, float factor, int32_t* topk_ids, float* topk_weights,
              void* stream);

/*
 * The routed rows of each expert, as the grouped calls of bsq.h take them:
 * entry (token t, place j) of topk_ids goes to the group of its expert, the
 * entries of an expert in their order (t, then j).
 *
 *   topk_ids        int32 [num_tokens][topk]; an entry outside num_experts has
 *                   no row.
 *   pad             1 .. 65536: scale rows of a group are its rows rounded up
 *                   to a multiple of pad (the MFMA scale layout takes 16).
 *   row_offsets, scales_offsets   uint32 [num_experts + 1].
 *   row_indices     int32 [num_tokens * topk]: the token of each routed row,
 *                   -1 past the last.
 *   entry_rows      int32 [num_tokens][topk]: the routed row of each entry, -1
 *                   for none; or NULL.
 *   num_experts     1 .. 1024;  num_tokens * topk at most 2^31 - 1, and with
 *                   num_experts * (pad - 1) at most 2^32 - 1.
 *   workspace       16-byte aligned, moe_group_rows_workspace(...) bytes (0: may
 *                   be NULL).
 * expert_ids of the grouped calls are the numbers 0 .. num_experts - 1.
 * No tokens: the offsets are written, all 0.
 */
int moe_group_rows(const int32_t* topk_ids, int64_t num_tokens, int64_t topk, int64_t num_experts,
                   int64_t pad, uint32_t* row_offsets, uint32_t* scales_offsets,
                   int32_t* row_indices, int32_t* entry_rows, void* workspace,
                   int64_t workspace_bytes, void* stream);
int64_t moe_group_rows_workspace(int64_t num_tokens, int64_t topk, int64_t num_experts);

/*
 * Log probabilities under softmax(logits), with its entropy and the likeliest
 * tokens, in one pass over the logits.
 *
 *   lse = log of the sum of exp(z);   logprobs = z_token - lse;
 *   entropy = - sum of p log p;   top_ids: the `top` largest z, the largest
 *   first, equal ones by their number, the lower first;   top_logprobs theirs.
 *
 * NaN counts as -inf.  A logit of +inf takes the whole probability, shared
 * with its equals.  A row whose logits are all -inf has log probabilities of
 * -inf and entropy 0.  A token outside the vocabulary has -inf.
 *
 *   dtype           of the logits [num_rows][vocab], ldl elements from a row
 *                   to the next, aligned to their size.
 *   vocab           1 .. 2^19 - 8 (more: BSQ_ERR_UNSUPPORTED).
 *   tokens          int32 [num_rows][num_tokens]; logprobs fp32, as tokens;
 *                   num_tokens 0 .. 2^30 (0: both may be NULL).
 *   entropy         fp32 [num_rows], or NULL.
 *   top             0 .. 64, at most vocab.  top_ids, top_logprobs: int32 /
 *                   fp32 [num_rows][top].
 *   workspace       16-byte aligned, token_logprobs_workspace(...) bytes (0:
 *                   may be NULL; -1 for sizes that the call would refuse).
 * Sums are fp32, of exp(z - the row's largest), in a fixed order.
 */
int token_logprobs(int dtype, const void* logits, int64_t ldl, int64_t num_rows, int64_t vocab,
                   const int32_t* tokens, int64_t num_tokens, int64_t top, float* logprobs,
                   float* entropy, int32_t* top_ids, float* top_logprobs, void* workspace,
                   int64_t workspace_bytes, void* stream);
int64_t token_logprobs_workspace(int64_t num_rows, int64_t vocab, int64_t top);

#ifdef __cplusplus
}
#endif

#endif /* BSQ_DECODER_H */
