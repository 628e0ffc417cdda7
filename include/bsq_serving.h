/*
 * bsq_serving.h -- C ABI of libbsq_serving, the operators of a decode step
 * that keep their state and weights in the block-scaled formats of bsq.h, on
 * AMD Instinct MI355X (gfx950): a paged key/value cache in 8 bits with the
 * attention that reads it and the management of its pages, and a mixture-of-
 * experts layer for a few tokens over MX weights.
 *
 * Conventions are those of bsq.h: device pointers owned by the caller,
 * nothing allocated, kernels only on `stream` (so a sequence of calls can be
 * captured in a HIP graph), every argument validated on the host before any
 * HIP call, a bsq_status returned and bsq_serving_last_error() describing a
 * failure.  Sizes of zero are no-ops that return BSQ_OK.  Device-array
 * contents (offsets, lengths, page and expert numbers) are not read on the
 * host; a number that falls outside the sizes given makes the kernels skip
 * what it names, never access memory outside the buffers.
 * bsq_time_next_launch does not see this library's kernels.
 */
#ifndef BSQ_SERVING_H
#define BSQ_SERVING_H

#include <stdint.h>

#include "bsq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The cache.  A page holds BSQ_KV_PAGE = 64 tokens of every head.  For each
 * (page, head), K and V each have one E8M0 scale byte b (2^(b - 127); 255:
 * NaN), and a value is its E4M3 code times that scale, as in bsq.h's MXFP8.
 *
 *   k_codes   uint8 [num_pages][num_heads][head_dim / 16][64][16]: element d
 *             of the page's token t at (d / 16) * 1024 + t * 16 + d % 16 of
 *             its (page, head).
 *   v_codes   uint8 [num_pages][num_heads][head_dim][64]: element d of token
 *             t = 16 j + 4 g + e (j, g, e in 0..3) at d * 64 + 16 g + 4 j + e.
 *             Both orders are those in which the matrix instruction takes its
 *             operands: every 16-byte load of a wave covers whole cache lines
 *             and no value is moved between lanes.
 *   page_stride    bytes from a page to the next in k_codes and in v_codes:
 *             a multiple of 16, at least num_heads * head_dim * 64.
 *   k_scales, v_scales   uint8 [num_pages][num_heads], scale_stride bytes
 *             from a page to the next, at least num_heads.
 *   num_pages at most 2^31 - 1;  num_heads 1 .. 65535;  head_dim 64, 128 or
 *             256 (others: BSQ_ERR_UNSUPPORTED).
 * k_codes and v_codes are 16-byte aligned.
 */
#define BSQ_KV_PAGE 64

typedef struct bsq_kv_cache {
    void* k_codes;
    void* v_codes;
    uint8_t* k_scales;
    uint8_t* v_scales;
    int64_t num_pages;
    int64_t page_stride;
    int64_t scale_stride;
    int32_t num_heads;
    int32_t head_dim;
} bsq_kv_cache;

/*
 * Sequences, the same for every cache call.  Sequence s has kv_lens[s]
 * tokens; token p of it is token p % 64 of page block_table[s][p / 64].
 *   block_table  int32 [num_seqs][max_pages], table_stride elements from a
 *                row to the next.  Entries past the last token are not read.
 *   kv_lens      int32 [num_seqs].
 * In a call with new tokens (append) or queries (attention), sequence s owns
 * the rows [row_offsets[s], row_offsets[s + 1]) of the row-major inputs
 * (uint32 [num_seqs + 1], nondecreasing, the last at most num_rows), which
 * are its LAST tokens: kv_lens counts them.  The same arrays serve both
 * calls of a step: append first, then attend.
 */

/*
 * Write new tokens into the cache.
 *
 *   k, v     BF16 [num_rows][num_heads][head_dim]: heads contiguous in a row,
 *            ldk / ldv elements from a row to the next (multiples of 8, so
 *            slices of one projection's output do), 16-byte aligned.
 *   max_new  host-side bound on the rows of one sequence (sizes the grid;
 *            rows past it are not written).
 * The pages written must be in the table already (kv_pages_reserve) and be
 * no other sequence's.
 *
 * For each (page, head) touched, of K and of V: X = max(floor(log2 amax) - 8,
 * -127) over the new tokens (bsq.h's MX rule); when the page held tokens of
 * the sequence before, X is at least their scale's, and where it grew their
 * codes are written again as RNE(code * 2^(X_old - X)).  New codes are
 * RNE_sat_E4M3(x * 2^-X).  A NaN or Inf among the new tokens, or the NaN
 * scale of the tokens before, gives the (page, head) the NaN scale and zero
 * codes for all its tokens.  Codes of tokens past the sequence's end are not
 * written.
 */
int kv_cache_append(const bsq_kv_cache* cache, const void* k, int64_t ldk, const void* v,
                    int64_t ldv, const uint32_t* row_offsets, const int32_t* kv_lens,
                    const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                    int64_t num_seqs, int64_t num_rows, int64_t max_new, void* stream);

/*
 * Attention of query rows over the cache (causal, the queries being their
 * sequence's last tokens): row i of a sequence with n rows and L tokens is
 * at place P = L - n + i and sees the tokens j with j <= P and, with
 * window > 0, j > P - window.  Query head h reads cache head
 * h / (num_q_heads / num_heads).
 *
 *   out[row, h] = sum over j of softmax_j(scale * q . k_j) v_j      (BF16)
 *   lse[row, h] = log of the sum of exp(scale * q . k_j)            (fp32)
 * A row that sees no token (L = 0, or P < 0) gets zeros and -inf.  A token
 * whose (page, head) has the NaN scale makes NaN of the rows that see it and
 * of no others; bytes past a sequence's end are never used.  E4M3 NaN codes
 * inside a sequence's length (which kv_cache_append never writes) make the
 * result of that sequence's head unspecified.  A page number outside the
 * cache leaves its tokens unseen.  Where the V scales of a head's pages lie
 * more than 2^60 apart, the smaller ones count as 0.
 *
 * Scores, softmax statistics and sums are fp32; K and V codes enter the
 * matrix cores exactly (K as BF16 beside the BF16 queries, V as FP16), and
 * the softmax weights as FP16 numbers between 2^11 and 2^15 for the largest
 * (11 bits down to 2^-25 of it, an absolute 2^-36 of it below that).  The
 * order of every sum is fixed: equal inputs and sizes give equal bits.
 *
 *   q             BF16 [num_rows][num_q_heads][head_dim], ldq elements from a
 *                 row to the next (a multiple of 8), 16-byte aligned.
 *   num_q_heads   a multiple of cache->num_heads, at most 65535.
 *   max_q         host-side bound on the rows of one sequence (rows past it
 *                 are not computed); max_kv on kv_lens (only a hint of how to
 *                 split the work: results hold for any lengths).
 *   scale         the factor of the scores, finite.
 *   window        0: every token up to the row's own; else the number of
 *                 tokens seen, the row's own included.
 *   out, ldo      BF16, as q.  lse: fp32 [num_rows][num_q_heads], or NULL.
 *   workspace     device memory, 16-byte aligned, at least
 *                 kv_cache_attention_workspace(...) bytes (may be NULL when
 *                 that is 0).
 * Rows of `out` and `lse` that no sequence owns are not written.
 */
int kv_cache_attention(const bsq_kv_cache* cache, const void* q, int64_t ldq,
                       int64_t num_q_heads, const uint32_t* row_offsets, const int32_t* kv_lens,
                       const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                       int64_t num_seqs, int64_t num_rows, int64_t max_q, int64_t max_kv,
                       float scale, int64_t window, void* out, int64_t ldo, float* lse,
                       void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace of a kv_cache_attention call of these sizes (partial
   results of work split over the tokens; 0 when none is needed), or -1 for
   sizes that the call would refuse. */
int64_t kv_cache_attention_workspace(int64_t num_heads, int64_t head_dim, int64_t num_q_heads,
                                     int64_t num_seqs, int64_t num_rows, int64_t max_q,
                                     int64_t max_kv, int64_t window);

/*
 * Pages.  refcounts (int32 [num_pages]) counts the table entries that name a
 * page; a page of count 0 is free.  Pages are given out lowest number first,
 * to the requests of a call in their order, so the result is a function of
 * the inputs alone.  Slot numbers index the rows of block_table and kv_lens
 * (num_seqs of them); a request with a slot outside them fails.
 * Status codes (int32, one per request): 0 done, 1 not enough free pages or
 * table entries (its length and the counts stay as they were; table entries
 * past its end may be written), 2 a slot outside the table.  One call names a
 * slot once (children of a fork: distinct slots that no request names as a
 * parent).
 *
 * No call shortens a sequence.  A caller that takes back its last tokens (a
 * proposal that was not accepted) writes the smaller number to kv_lens itself.
 * Where fewer pages hold it then, ceil(kv_lens / 64), it first takes 1 off the
 * counts of the pages that are given up: the last entries of the sequence's
 * table row.  Left counted they are free for no one, and the next reserve
 * writes over the entries that name them.  The next append then writes over
 * the tokens taken back; in a page where others stay, the scale is at least
 * what they had made it.  A page that is partly filled afterwards must be the
 * sequence's own, as for any append: one that a fork shares (a count above 1)
 * is first exchanged for a copy, a free page with count 1 (kv_pages_copy, its
 * number in the table, and 1 off the shared page's count).
 *
 * kv_pages_copy     page dst[i] becomes a copy of page src[i] (codes and
 *     scales of every head).  Distinct destinations, none of them a source
 *     of another pair.  Pairs outside the cache are skipped.
 * kv_pages_reserve  lengthens sequence slots[i] by add_tokens[i] >= 0 tokens
 *     (kv_lens grows) and gives it the pages that this takes.
 * kv_pages_fork     slot children[i], which holds nothing, becomes a copy of
 *     slot parents[i]: full pages are shared (their counts grow), a partly
 *     filled last page is copied to a page of the child's own, so that both
 *     can be appended to.  A request that fails leaves the child's kv_lens 0.
 * kv_pages_free     sequence slots[i] gives its pages back (their counts
 *     shrink) and its kv_lens becomes 0; its table row is left as it was.
 * kv_pages_compact  with n pages in use, moves each page in use numbered n
 *     or above to a free one below n (the lowest to the lowest), writes the
 *     table with the new numbers to table_out and the counts to
 *     refcounts_out, and n to num_live[0].  Either output may be the input
 *     itself; the moved pages' old places keep their bytes.  Every user of
 *     the cache's pages must be in block_table.
 *
 * kv_pages_compact's workspace: 16-byte aligned, at least
 * kv_pages_compact_workspace(num_pages) bytes.
 * kv_pages_fork's and kv_pages_reserve's status may not be NULL.
 */
int kv_pages_copy(const bsq_kv_cache* cache, const int32_t* src, const int32_t* dst, int64_t n,
                  void* stream);
int kv_pages_reserve(int32_t* block_table, int64_t table_stride, int64_t max_pages,
                     int64_t num_seqs, int32_t* kv_lens, int32_t* refcounts, int64_t num_pages,
                     const int32_t* slots, const int32_t* add_tokens, int64_t n, int32_t* status,
                     void* stream);
int kv_pages_fork(const bsq_kv_cache* cache, int32_t* block_table, int64_t table_stride,
                  int64_t max_pages, int64_t num_seqs, int32_t* kv_lens, int32_t* refcounts,
                  const int32_t* parents, const int32_t* children, int64_t n, int32_t* status,
                  void* stream);
int kv_pages_free(const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                  int64_t num_seqs, int32_t* kv_lens, int32_t* refcounts, int64_t num_pages,
                  const int32_t* slots, int64_t n, void* stream);
int kv_pages_compact(const bsq_kv_cache* cache, const int32_t* block_table, int64_t table_stride,
                     int64_t max_pages, int64_t num_seqs, const int32_t* kv_lens,
                     const int32_t* refcounts, int32_t* table_out, int64_t table_out_stride,
                     int32_t* refcounts_out, int32_t* num_live, void* workspace,
                     int64_t workspace_bytes, void* stream);
int64_t kv_pages_compact_workspace(int64_t num_pages);

/*
 * A mixture-of-experts layer for a few tokens.  With at most 16 (token,
 * expert) entries it is two kernels: routing (of at most 4 tokens),
 * gate and up products with the SiLU gate, then the down products summed over
 * each token's experts.  More entries keep their parts of the down products
 * apart, which a third kernel sums; more tokens are routed by one before.
 *
 *   y[t] = sum over the token's experts e of w_te * W2_e h_te   (BF16)
 *   h_te = silu(W1_e x_t) * (W3_e x_t)
 *
 *   x            BF16 [num_tokens][hidden], ldx elements from a row to the
 *                next (a multiple of 8), 16-byte aligned.
 *   format       BSQ_MXFP4 or BSQ_MXFP8 weights, as the grouped GEMM takes
 *                them: codes row-major (16-byte aligned rows without gaps),
 *                scales in BSQ_SCALES_MFMA16 (256 * ceil(K / 512) bytes per
 *                16 rows, without gaps).
 *   w13_codes, w13_scales   [num_experts * 2 * inter] rows of `hidden`
 *                elements: expert e's W1 in rows 2 e inter .., its W3 in the
 *                inter rows after them.
 *   w2_codes, w2_scales     [num_experts * hidden] rows of `inter` elements.
 *   router_logits   fp32 [num_tokens][num_experts] without gaps, or NULL.
 *                Given: the token's experts are the topk largest logits (ties
 *                to the lower expert; NaN counts as -inf), and its weights
 *                their softmax over all experts or, with renormalize != 0,
 *                over the topk; both are written to topk_ids and
 *                topk_weights.  A token whose logits are all -inf or NaN gets
 *                weights 0, and so does an expert whose logit is.  A logit
 *                of +inf takes the whole weight, shared with its equals.
 *                NULL: topk_ids and topk_weights are inputs.
 *   topk_ids, topk_weights  int32 / fp32 [num_tokens][topk].  An entry with
 *                weight 0 or an expert outside num_experts contributes
 *                nothing, whatever the expert's weights hold.
 *   num_tokens   0 .. 64 (more: BSQ_ERR_UNSUPPORTED -- take those through the
 *                quantizers and grouped_block_scaled_matmul_mfma).  topk
 *                1 .. 16, at most num_experts; num_experts 1 .. 1024.  hidden and inter:
 *                multiples of 128, at most 2^17.
 *   y            BF16 [num_tokens][hidden], ldy as ldx.
 *   workspace    16-byte aligned, moe_few_tokens_workspace(...) bytes.
 * Products are summed in fp32, weights enter the matrix cores exactly (as
 * BF16), and h as the sum of two BF16 numbers (16 bits).
 * The order of every sum is fixed.
 */
int moe_few_tokens(int format, const void* x, int64_t ldx, int64_t num_tokens, int64_t hidden,
                   int64_t inter, int64_t num_experts, int64_t topk, const void* w13_codes,
                   const void* w13_scales, const void* w2_codes, const void* w2_scales,
                   const float* router_logits, int renormalize, int32_t* topk_ids,
                   float* topk_weights, void* y, int64_t ldy, void* workspace,
                   int64_t workspace_bytes, void* stream);

/* Bytes of moe_few_tokens' workspace, or -1 for sizes it would refuse. */
int64_t moe_few_tokens_workspace(int64_t num_tokens, int64_t hidden, int64_t inter, int64_t topk);

/* Message of the calling thread's most recent failed call into this library
   ("" after a call that returned BSQ_OK). */
const char* bsq_serving_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* BSQ_SERVING_H */
