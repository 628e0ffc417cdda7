// bsq_serving_internal.h -- launch interface between the host layer of
// libbsq_serving (bsq_serving_api.cpp) and its gfx950 kernels (bsq_kv.hip,
// bsq_pages.hip, bsq_moe.hip, bsq_rope.hip, bsq_route.hip,
// bsq_logprobs.hip).  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bsq {

constexpr int kKvPage = 64;          // tokens of a cache page

struct KvCache {
    uint8_t* k_codes;
    uint8_t* v_codes;
    uint8_t* k_scales;
    uint8_t* v_scales;
    int64_t page_stride;             // bytes
    int64_t scale_stride;            // bytes
    int32_t num_pages;
    int32_t num_heads;
    int32_t head_dim;
};

struct KvSeqs {
    const uint32_t* row_offsets;     // [num_seqs + 1]
    const int32_t* kv_lens;          // [num_seqs]
    const int32_t* table;
    int64_t table_stride;
    int64_t num_rows;
    int32_t max_pages;
    int32_t num_seqs;
};

struct AppendArgs {
    KvCache cache;
    KvSeqs seqs;
    const uint16_t* x[2];            // K, V
    int64_t ldx[2];                  // elements
    int32_t max_new;                 // tokens of a sequence at most
    int32_t pages_per_seq;           // grid bound on the pages that they touch
};
// Threads for a page and head: up to 5 tokens lie in two groups of 4, one wave's work (64
// sequences of 5 tokens, 8 heads of 128: 6.2 us a call, with 256 threads 8.1).
constexpr int append_threads(int64_t max_new) { return max_new <= 5 ? 64 : 256; }
hipError_t launch_kv_append(const AppendArgs& a, hipStream_t stream);

struct AttendArgs {
    KvCache cache;
    KvSeqs seqs;
    const uint16_t* q;
    int64_t ldq;
    uint16_t* out;
    int64_t ldo;
    float* lse;                      // nullable
    float* part_o;                   // [splits][num_rows][num_q_heads][head_dim]
    float* part_ml;                  // [splits][num_rows][num_q_heads][2]
    int64_t window;                  // 0: none
    const uint64_t* masks;           // nullable; [num_rows][mask_words]
    int32_t mask_words, sinks;       // sinks: of account with a window alone
    float scale;
    int32_t num_q_heads;
    int32_t group;                   // num_q_heads / num_heads
    int32_t max_q;
    int32_t col_blocks;              // workgroups over (row, head of the group) pairs, and
    int32_t block_cols;              // pairs of each
    int32_t splits;
    int32_t split_pages;             // pages of a split
};
// How a call's work is cut; also what the workspace is sized by.
struct AttendPlan {
    bool rows_form;                  // waves share the pages and split the columns (many rows)
    int32_t col_blocks;
    int32_t block_cols;
    int32_t splits;
    int32_t split_pages;
    bool wide;                       // eight waves a workgroup instead of four (both forms)
    int32_t threads;                 // of a workgroup
    bool masked;                     // the kernels that know trees and sinks
};
AttendPlan plan_attend(int64_t num_heads, int64_t head_dim, int64_t num_q_heads, int64_t num_seqs,
                       int64_t max_q, int64_t max_kv, int64_t window, int64_t sinks, bool tree);
hipError_t launch_kv_attend(const AttendArgs& a, const AttendPlan& p, hipStream_t stream);

struct PageArgs {
    KvCache cache;                   // of kv_pages_reserve and kv_pages_free: num_pages alone
    int32_t* table;
    int64_t table_stride;
    int32_t* kv_lens;
    int32_t* refcounts;
    const int32_t* a;                // sources, slots or parents
    const int32_t* b;                // destinations, tokens to add or children
    int32_t* status;
    int32_t max_pages;
    int32_t num_seqs;
    int32_t n;                       // requests
};
hipError_t launch_pages_copy(const PageArgs& p, hipStream_t stream);
hipError_t launch_pages_reserve(const PageArgs& p, hipStream_t stream);
hipError_t launch_pages_fork(const PageArgs& p, hipStream_t stream);
hipError_t launch_pages_free(const PageArgs& p, hipStream_t stream);

struct CompactArgs {
    KvCache cache;
    const int32_t* table;
    int64_t table_stride;
    const int32_t* kv_lens;
    const int32_t* refs;
    int32_t* table_out;
    int64_t table_out_stride;
    int32_t* refs_out;
    int32_t* num_live;
    int32_t* moves;                  // workspace: number of moves, then their sources, then their
                                     // destinations (num_pages / 2 + 1 each), then new numbers
    int32_t max_pages;
    int32_t num_seqs;
};
hipError_t launch_pages_compact(const CompactArgs& p, hipStream_t stream);

struct MoeArgs {
    const uint16_t* x;
    int64_t ldx;                     // elements
    const uint8_t* w13;
    const uint8_t* w13_scales;
    const uint8_t* w2;
    const uint8_t* w2_scales;
    const float* logits;             // nullable
    int32_t* ids;
    float* weights;
    uint16_t* h;                     // [num_tokens * topk][2][inter] BF16, workspace: h is the
                                     // sum of the two
    float* part;                     // [num_tokens * topk][hidden], workspace of many entries
    uint16_t* y;
    int64_t ldy;
    int32_t tokens, hidden, inter, experts, topk;
    int32_t renormalize;
};
constexpr int kMoeMaxTokens = 64, kMoeMaxExperts = 1024, kMoeMaxTopk = 16;
// Entries (a token's choices of an expert) that one wave's lanes hold, one block of matrix
// columns: so few take the kernels without LDS tables and partial results, which save a launch
// or two but whose down products have a workgroup for 16 columns only.  Both forms, with 8
// experts a token of 128 (2048 x 768, FP4): 8 entries 17.3 and 26.3 us, 16 23.7 and 28.5, 24
// 32.6 and 31.7, 32 37.9 and 33.1.
constexpr int kFewEntries = 16;
inline bool moe_is_few(int64_t tokens, int64_t topk) { return tokens * topk <= kFewEntries; }
hipError_t launch_moe(int fmt, const MoeArgs& a, hipStream_t stream);

struct RopeArgs {
    const void* x[3];                // q, k, v
    uint16_t* out[3];
    int64_t ldx[3], ldo[3];          // elements
    int32_t heads[3];                // v: 0 where there is none
    const float* weight[2];          // nullable
    const int32_t* positions;
    const double* inv_freq;
    int64_t num_rows;
    float eps, inv_dim;
    int32_t head_dim, rotary_dim;
    int32_t seg_steps[3], all_steps; // steps (of as many heads as a wave takes at once) of a row
    int32_t steps, parts;            // of a wave; waves of a row
    bool once;                       // loads past the caches
};
void plan_rope(RopeArgs& a, bool f32);   // seg_steps and what follows, from the sizes
hipError_t launch_rope(const RopeArgs& a, bool f32, bool pairs, hipStream_t stream);

struct RouteArgs {
    const void* logits;
    int64_t ldl;                     // elements
    const float* bias;               // nullable
    int32_t* ids;
    float* weights;
    int64_t tokens;
    float factor;
    int32_t experts, topk, groups, keep, group_top;
    int32_t sigmoid, renormalize;
    int32_t group_size;              // experts of a group,
    uint32_t group_magic;            // e * group_magic >> 20 = e / group_size for every expert e,
    int32_t group_lanes;             // lanes that look at a group: a power of two
};
void plan_route(RouteArgs& a);       // group_size and what follows
hipError_t launch_route(const RouteArgs& a, bool f32, hipStream_t stream);

struct GroupArgs {
    const int32_t* ids;
    int64_t entries;
    uint32_t* row_offsets;
    uint32_t* scales_offsets;
    int32_t* row_indices;
    int32_t* entry_rows;             // nullable
    int32_t* counts;                 // [tiles][experts], workspace of more than one tile,
    int32_t* ranks;                  // and behind it [entries]: within the tile
    int32_t topk, experts;
    uint32_t pad;
    int64_t tile;                    // entries of a workgroup
    int32_t tiles, bits;             // bits of the numbers 0 .. experts
    int32_t count_lanes;             // threads that read consecutive counts of a tile
};
void plan_group(GroupArgs& a);       // tile and what follows
hipError_t launch_group(const GroupArgs& a, hipStream_t stream);

struct LogprobArgs {
    const void* logits;
    int64_t ldl, rows;               // elements
    const int32_t* tokens;           // [rows][num_tokens]
    float* logprobs;
    float* entropy;                  // nullable
    int32_t* top_ids;                // [rows][top]
    float* top_logprobs;
    float* sums;                     // [rows][slices][3], workspace of more than one slice
    uint64_t* best;                  // [rows][slices][top], before them
    int32_t vocab, num_tokens, top;
    int32_t slices, per_thread;      // of a row; elements of a thread and chunk
    int32_t chunks;                  // of a slice
};
constexpr int kMostTop = 64, kMostVocab = (1 << 19) - 8;
void plan_logprobs(LogprobArgs& a);  // slices and what follows, from rows and vocab
hipError_t launch_logprobs(const LogprobArgs& a, bool f32, hipStream_t stream);

}  // namespace bsq
