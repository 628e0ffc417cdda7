// bsq_serving_api.cpp -- the C ABI of libbsq_serving (declared in
// include/bsq_serving.h): argument validation, launch geometry and error
// reporting.  Every check runs on the host before any HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "bsq_serving.h"
#include "bsq_serving_internal.h"

namespace {

thread_local char g_last_error[512] = "";

int fail(int status, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return status;
}

int ok() {
    g_last_error[0] = 0;
    return BSQ_OK;
}

int launched(hipError_t e) {
    if (e != hipSuccess) return fail(BSQ_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
    return ok();
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

constexpr int64_t kMaxInt = 0x7FFFFFFF;

// Whether a launch may have that many workgroups: its threads are counted in 32 bits.
bool fits(double workgroups, int threads) { return workgroups <= (double)(0xFFFFFFFFu / threads); }
constexpr int kPageThreads = 256;    // of every kernel with a workgroup per request

// Head count, head width and page count of a cache; with data, its buffers too.
int check_cache(const bsq_kv_cache* c, bsq::KvCache* out) {
    if (!c) return fail(BSQ_ERR_INVALID_ARG, "null pointer (cache)");
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(BSQ_ERR_UNSUPPORTED, "head_dim=%d is not provided (64, 128 or 256)", c->head_dim);
    if (c->num_heads < 1 || c->num_heads > 65535)
        return fail(BSQ_ERR_INVALID_ARG, "num_heads=%d must be in 1 .. 65535", c->num_heads);
    if (c->num_pages < 0 || c->num_pages > kMaxInt)
        return fail(BSQ_ERR_INVALID_ARG, "num_pages=%lld must be in 0 .. 2^31 - 1",
                    (long long)c->num_pages);
    const int64_t need = (int64_t)c->num_heads * c->head_dim * bsq::kKvPage;
    if (c->page_stride < need || c->page_stride % 16 != 0)
        return fail(BSQ_ERR_INVALID_ARG, "page_stride=%lld must be >= %lld and a multiple of 16",
                    (long long)c->page_stride, (long long)need);
    if (c->scale_stride < c->num_heads)
        return fail(BSQ_ERR_INVALID_ARG, "scale_stride=%lld must be >= num_heads=%d",
                    (long long)c->scale_stride, c->num_heads);
    if (c->num_pages > 0) {
        if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales)
            return fail(BSQ_ERR_INVALID_ARG, "null pointer in the cache");
        if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16))
            return fail(BSQ_ERR_INVALID_ARG, "k_codes and v_codes must be 16-byte aligned");
    }
    out->k_codes = static_cast<uint8_t*>(c->k_codes);
    out->v_codes = static_cast<uint8_t*>(c->v_codes);
    out->k_scales = c->k_scales;
    out->v_scales = c->v_scales;
    out->page_stride = c->page_stride;
    out->scale_stride = c->scale_stride;
    out->num_pages = (int32_t)c->num_pages;
    out->num_heads = c->num_heads;
    out->head_dim = c->head_dim;
    return BSQ_OK;
}

// The table's sizes, and its buffers when there are sequences.
int check_table(const void* table, int64_t table_stride, int64_t max_pages, int64_t num_seqs,
                const void* kv_lens) {
    if (num_seqs < 0 || num_seqs > kMaxInt || max_pages < 0 || max_pages > (kMaxInt >> 6))
        return fail(BSQ_ERR_INVALID_ARG,
                    "num_seqs=%lld must be in 0 .. 2^31 - 1 and max_pages=%lld in 0 .. 2^25 - 1",
                    (long long)num_seqs, (long long)max_pages);
    if (table_stride < max_pages)
        return fail(BSQ_ERR_INVALID_ARG, "table_stride=%lld must be >= max_pages=%lld",
                    (long long)table_stride, (long long)max_pages);
    if (num_seqs > 0 && (!kv_lens || (max_pages > 0 && !table)))
        return fail(BSQ_ERR_INVALID_ARG, "null pointer (block_table=%p kv_lens=%p)", table, kv_lens);
    return BSQ_OK;
}

int check_rows(const char* what, const void* p, int64_t ld, int64_t width) {
    if (!p) return fail(BSQ_ERR_INVALID_ARG, "null pointer (%s)", what);
    if (!aligned(p, 16)) return fail(BSQ_ERR_INVALID_ARG, "%s must be 16-byte aligned", what);
    if (ld < width || ld % 8 != 0)
        return fail(BSQ_ERR_INVALID_ARG, "the row stride %lld of %s must be >= %lld and a multiple of 8",
                    (long long)ld, what, (long long)width);
    return BSQ_OK;
}

int check_seqs(const uint32_t* row_offsets, const int32_t* kv_lens, const int32_t* table,
               int64_t table_stride, int64_t max_pages, int64_t num_seqs, int64_t num_rows,
               int64_t most, bsq::KvSeqs* out) {
    const int st = check_table(table, table_stride, max_pages, num_seqs, kv_lens);
    if (st != BSQ_OK) return st;
    if (num_rows < 0 || num_rows > kMaxInt || most < 0 || most > kMaxInt)
        return fail(BSQ_ERR_INVALID_ARG, "rows (%lld) and rows of a sequence (%lld) must be in "
                    "0 .. 2^31 - 1", (long long)num_rows, (long long)most);
    if (num_seqs > 0 && !row_offsets) return fail(BSQ_ERR_INVALID_ARG, "null pointer (row_offsets)");
    out->row_offsets = row_offsets;
    out->kv_lens = kv_lens;
    out->table = table;
    out->table_stride = table_stride;
    out->num_rows = num_rows;
    out->max_pages = (int32_t)max_pages;
    out->num_seqs = (int32_t)num_seqs;
    return BSQ_OK;
}

// The query heads and sizes of an attention call, and how its work is cut.
int plan(int64_t num_heads, int64_t head_dim, int64_t num_q_heads, int64_t num_seqs, int64_t max_q,
         int64_t max_kv, int64_t window, bsq::AttendPlan* p) {
    if (num_heads < 1 || num_q_heads < 1 || num_q_heads > 65535 || num_q_heads % num_heads != 0)
        return fail(BSQ_ERR_INVALID_ARG,
                    "num_q_heads=%lld must be in 1 .. 65535 and a multiple of num_heads=%lld",
                    (long long)num_q_heads, (long long)num_heads);
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return fail(BSQ_ERR_UNSUPPORTED, "head_dim=%lld is not provided (64, 128 or 256)",
                    (long long)head_dim);
    if (num_seqs < 0 || num_seqs > kMaxInt || max_q < 0 || max_q > kMaxInt || max_kv < 0 ||
        max_kv > kMaxInt || window < 0)
        return fail(BSQ_ERR_INVALID_ARG,
                    "num_seqs=%lld, max_q=%lld and max_kv=%lld must be in 0 .. 2^31 - 1, window=%lld "
                    ">= 0", (long long)num_seqs, (long long)max_q, (long long)max_kv,
                    (long long)window);
    if (max_q * (num_q_heads / num_heads) > 0x7FFFFE00LL)
        return fail(BSQ_ERR_INVALID_ARG, "max_q=%lld rows of %lld heads are too many",
                    (long long)max_q, (long long)num_q_heads);
    if (num_seqs == 0 || max_q == 0) {
        *p = bsq::AttendPlan{};
        return BSQ_OK;
    }
    *p = bsq::plan_attend(num_heads, head_dim, num_q_heads, num_seqs, max_q, max_kv, window);
    const double blocks = (double)num_seqs * (double)num_heads * (double)p->col_blocks * p->splits;
    const double pairs = (double)num_seqs * (double)max_q * (double)num_q_heads;
    // the join has at least a wave for each pair
    if (!fits(blocks, p->threads) || (p->splits > 1 && !fits(pairs, 64)))
        return fail(BSQ_ERR_INVALID_ARG, "problem too large for one launch");
    return BSQ_OK;
}

int64_t attend_workspace(const bsq::AttendPlan& p, int64_t num_rows, int64_t num_q_heads,
                         int64_t head_dim) {
    if (p.splits <= 1) return 0;
    return (int64_t)p.splits * num_rows * num_q_heads * (head_dim + 2) * (int64_t)sizeof(float);
}

int check_pages(const bsq_kv_cache* cache, const void* a, const void* b, int64_t n,
                bsq::PageArgs* p) {
    const int st = check_cache(cache, &p->cache);
    if (st != BSQ_OK) return st;
    if (n < 0 || n > kMaxInt) return fail(BSQ_ERR_INVALID_ARG, "n=%lld out of range", (long long)n);
    if (n > 0 && (!a || !b)) return fail(BSQ_ERR_INVALID_ARG, "null pointer in the requests");
    p->a = static_cast<const int32_t*>(a);
    p->b = static_cast<const int32_t*>(b);
    p->n = (int32_t)n;
    // one workgroup for each 16 KiB of a page and request
    const int64_t parts = 2 * (int64_t)p->cache.num_heads * p->cache.head_dim * bsq::kKvPage / 16384 + 2;
    if (!fits((double)(n * parts), kPageThreads))
        return fail(BSQ_ERR_INVALID_ARG, "problem too large for one launch");
    return BSQ_OK;
}

int check_slots(int64_t num_pages, const void* refcounts, const void* slots, int64_t n) {
    if (num_pages < 0 || num_pages > kMaxInt || n < 0 || n > kMaxInt)
        return fail(BSQ_ERR_INVALID_ARG, "num_pages=%lld and n=%lld must be in 0 .. 2^31 - 1",
                    (long long)num_pages, (long long)n);
    if (n > 0 && (!slots || (num_pages > 0 && !refcounts)))
        return fail(BSQ_ERR_INVALID_ARG, "null pointer (refcounts=%p slots=%p)", refcounts, slots);
    return BSQ_OK;
}

}  // namespace

extern "C" {

int kv_cache_append(const bsq_kv_cache* cache, const void* k, int64_t ldk, const void* v,
                    int64_t ldv, const uint32_t* row_offsets, const int32_t* kv_lens,
                    const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                    int64_t num_seqs, int64_t num_rows, int64_t max_new, void* stream) {
    bsq::AppendArgs a{};
    int st = check_cache(cache, &a.cache);
    if (st == BSQ_OK)
        st = check_seqs(row_offsets, kv_lens, block_table, table_stride, max_pages, num_seqs,
                        num_rows, max_new, &a.seqs);
    if (st != BSQ_OK) return st;
    if (num_seqs == 0 || num_rows == 0 || max_new == 0 || max_pages == 0 || cache->num_pages == 0)
        return ok();
    const int64_t width = (int64_t)cache->num_heads * cache->head_dim;
    if ((st = check_rows("k", k, ldk, width)) != BSQ_OK) return st;
    if ((st = check_rows("v", v, ldv, width)) != BSQ_OK) return st;
    a.x[0] = static_cast<const uint16_t*>(k);
    a.x[1] = static_cast<const uint16_t*>(v);
    a.ldx[0] = ldk;
    a.ldx[1] = ldv;
    // max_new tokens touch one page more than they fill when they start inside one
    int64_t pages = (max_new + bsq::kKvPage - 2) / bsq::kKvPage + 1;
    if (pages > max_pages) pages = max_pages;
    if (!fits((double)(num_seqs * pages), bsq::append_threads(max_new)))
        return fail(BSQ_ERR_INVALID_ARG, "problem too large for one launch");
    a.pages_per_seq = (int32_t)pages;
    a.max_new = (int32_t)max_new;
    return launched(bsq::launch_kv_append(a, static_cast<hipStream_t>(stream)));
}

int64_t kv_cache_attention_workspace(int64_t num_heads, int64_t head_dim, int64_t num_q_heads,
                                     int64_t num_seqs, int64_t num_rows, int64_t max_q,
                                     int64_t max_kv, int64_t window) {
    bsq::AttendPlan p;
    if (num_rows < 0 || num_rows > kMaxInt) {
        fail(BSQ_ERR_INVALID_ARG, "num_rows=%lld must be in 0 .. 2^31 - 1", (long long)num_rows);
        return -1;
    }
    if (plan(num_heads, head_dim, num_q_heads, num_seqs, max_q, max_kv, window, &p) != BSQ_OK)
        return -1;
    ok();
    return attend_workspace(p, num_rows, num_q_heads, head_dim);
}

int kv_cache_attention(const bsq_kv_cache* cache, const void* q, int64_t ldq, int64_t num_q_heads,
                       const uint32_t* row_offsets, const int32_t* kv_lens,
                       const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                       int64_t num_seqs, int64_t num_rows, int64_t max_q, int64_t max_kv,
                       float scale, int64_t window, void* out, int64_t ldo, float* lse,
                       void* workspace, int64_t workspace_bytes, void* stream) {
    bsq::AttendArgs a{};
    bsq::AttendPlan p;
    int st = check_cache(cache, &a.cache);
    if (st == BSQ_OK)
        st = check_seqs(row_offsets, kv_lens, block_table, table_stride, max_pages, num_seqs,
                        num_rows, max_q, &a.seqs);
    if (st == BSQ_OK)
        st = plan(cache->num_heads, cache->head_dim, num_q_heads, num_seqs, max_q, max_kv, window, &p);
    if (st != BSQ_OK) return st;
    if (!std::isfinite(scale)) return fail(BSQ_ERR_INVALID_ARG, "scale must be finite");
    if (num_seqs == 0 || num_rows == 0 || max_q == 0) return ok();
    const int64_t width = num_q_heads * cache->head_dim;
    if ((st = check_rows("q", q, ldq, width)) != BSQ_OK) return st;
    if ((st = check_rows("out", out, ldo, width)) != BSQ_OK) return st;
    const int64_t need = attend_workspace(p, num_rows, num_q_heads, cache->head_dim);
    if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
        return fail(BSQ_ERR_INVALID_ARG,
                    "workspace (%p, %lld bytes) must be 16-byte aligned and hold %lld bytes",
                    workspace, (long long)workspace_bytes, (long long)need);
    a.q = static_cast<const uint16_t*>(q);
    a.ldq = ldq;
    a.out = static_cast<uint16_t*>(out);
    a.ldo = ldo;
    a.lse = lse;
    a.part_o = static_cast<float*>(workspace);
    if (need > 0)
        a.part_ml = a.part_o + (int64_t)p.splits * num_rows * num_q_heads * cache->head_dim;
    a.window = window > kMaxInt ? 0 : window;      // longer than any sequence; its places stay in 64 bits
    a.scale = scale;
    a.num_q_heads = (int32_t)num_q_heads;
    a.group = (int32_t)(num_q_heads / cache->num_heads);
    a.max_q = (int32_t)max_q;
    a.col_blocks = p.col_blocks;
    a.block_cols = p.block_cols;
    a.splits = p.splits;
    a.split_pages = p.split_pages;
    return launched(bsq::launch_kv_attend(a, p, static_cast<hipStream_t>(stream)));
}

int kv_pages_copy(const bsq_kv_cache* cache, const int32_t* src, const int32_t* dst, int64_t n,
                  void* stream) {
    bsq::PageArgs p{};
    const int st = check_pages(cache, src, dst, n, &p);
    if (st != BSQ_OK) return st;
    if (n == 0) return ok();
    return launched(bsq::launch_pages_copy(p, static_cast<hipStream_t>(stream)));
}

int kv_pages_reserve(int32_t* block_table, int64_t table_stride, int64_t max_pages,
                     int64_t num_seqs, int32_t* kv_lens, int32_t* refcounts, int64_t num_pages,
                     const int32_t* slots, const int32_t* add_tokens, int64_t n, int32_t* status,
                     void* stream) {
    bsq::PageArgs p{};
    int st = check_table(block_table, table_stride, max_pages, num_seqs, kv_lens);
    if (st == BSQ_OK) st = check_slots(num_pages, refcounts, slots, n);
    if (st != BSQ_OK) return st;
    if (n == 0) return ok();
    if (!add_tokens || !status)
        return fail(BSQ_ERR_INVALID_ARG, "null pointer (add_tokens=%p status=%p)", add_tokens, status);
    p.cache.num_pages = (int32_t)num_pages;
    p.table = block_table;
    p.table_stride = table_stride;
    p.kv_lens = kv_lens;
    p.refcounts = refcounts;
    p.a = slots;
    p.b = add_tokens;
    p.status = status;
    p.max_pages = (int32_t)max_pages;
    p.num_seqs = (int32_t)num_seqs;
    p.n = (int32_t)n;
    return launched(bsq::launch_pages_reserve(p, static_cast<hipStream_t>(stream)));
}

int kv_pages_fork(const bsq_kv_cache* cache, int32_t* block_table, int64_t table_stride,
                  int64_t max_pages, int64_t num_seqs, int32_t* kv_lens, int32_t* refcounts,
                  const int32_t* parents, const int32_t* children, int64_t n, int32_t* status,
                  void* stream) {
    bsq::PageArgs p{};
    int st = check_pages(cache, parents, children, n, &p);
    if (st == BSQ_OK) st = check_table(block_table, table_stride, max_pages, num_seqs, kv_lens);
    if (st == BSQ_OK) st = check_slots(cache->num_pages, refcounts, parents, n);
    if (st != BSQ_OK) return st;
    if (n == 0) return ok();
    if (!status) return fail(BSQ_ERR_INVALID_ARG, "null pointer (status)");
    p.table = block_table;
    p.table_stride = table_stride;
    p.kv_lens = kv_lens;
    p.refcounts = refcounts;
    p.status = status;
    p.max_pages = (int32_t)max_pages;
    p.num_seqs = (int32_t)num_seqs;
    return launched(bsq::launch_pages_fork(p, static_cast<hipStream_t>(stream)));
}

int kv_pages_free(const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                  int64_t num_seqs, int32_t* kv_lens, int32_t* refcounts, int64_t num_pages,
                  const int32_t* slots, int64_t n, void* stream) {
    bsq::PageArgs p{};
    int st = check_table(block_table, table_stride, max_pages, num_seqs, kv_lens);
    if (st == BSQ_OK) st = check_slots(num_pages, refcounts, slots, n);
    if (st != BSQ_OK) return st;
    if (n == 0) return ok();
    if (!fits((double)n, kPageThreads))
        return fail(BSQ_ERR_INVALID_ARG, "problem too large for one launch");
    p.cache.num_pages = (int32_t)num_pages;
    p.table = const_cast<int32_t*>(block_table);   // read only
    p.table_stride = table_stride;
    p.kv_lens = kv_lens;
    p.refcounts = refcounts;
    p.a = slots;
    p.max_pages = (int32_t)max_pages;
    p.num_seqs = (int32_t)num_seqs;
    p.n = (int32_t)n;
    return launched(bsq::launch_pages_free(p, static_cast<hipStream_t>(stream)));
}

int64_t kv_pages_compact_workspace(int64_t num_pages) {
    if (num_pages < 0 || num_pages > kMaxInt) {
        fail(BSQ_ERR_INVALID_ARG, "num_pages=%lld must be in 0 .. 2^31 - 1", (long long)num_pages);
        return -1;
    }
    ok();
    return (int64_t)sizeof(int32_t) * (4 + 2 * (num_pages / 2 + 1) + num_pages);
}

int kv_pages_compact(const bsq_kv_cache* cache, const int32_t* block_table, int64_t table_stride,
                     int64_t max_pages, int64_t num_seqs, const int32_t* kv_lens,
                     const int32_t* refcounts, int32_t* table_out, int64_t table_out_stride,
                     int32_t* refcounts_out, int32_t* num_live, void* workspace,
                     int64_t workspace_bytes, void* stream) {
    bsq::CompactArgs p{};
    int st = check_cache(cache, &p.cache);
    if (st == BSQ_OK) st = check_table(block_table, table_stride, max_pages, num_seqs, kv_lens);
    if (st == BSQ_OK) st = check_table(table_out, table_out_stride, max_pages, num_seqs, kv_lens);
    if (st != BSQ_OK) return st;
    if (!num_live || (cache->num_pages > 0 && (!refcounts || !refcounts_out)))
        return fail(BSQ_ERR_INVALID_ARG, "null pointer (refcounts=%p refcounts_out=%p num_live=%p)",
                    refcounts, refcounts_out, num_live);
    if (table_out == block_table && table_out_stride != table_stride)
        return fail(BSQ_ERR_INVALID_ARG, "table_out is block_table with another stride");
    const int64_t need = kv_pages_compact_workspace(cache->num_pages);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < need)
        return fail(BSQ_ERR_INVALID_ARG,
                    "workspace (%p, %lld bytes) must be 16-byte aligned and hold %lld bytes",
                    workspace, (long long)workspace_bytes, (long long)need);
    p.table = block_table;
    p.table_stride = table_stride;
    p.kv_lens = kv_lens;
    p.refs = refcounts;
    p.table_out = table_out;
    p.table_out_stride = table_out_stride;
    p.refs_out = refcounts_out;
    p.num_live = num_live;
    p.moves = static_cast<int32_t*>(workspace);
    p.max_pages = (int32_t)max_pages;
    p.num_seqs = (int32_t)num_seqs;
    return launched(bsq::launch_pages_compact(p, static_cast<hipStream_t>(stream)));
}

int64_t moe_few_tokens_workspace(int64_t num_tokens, int64_t hidden, int64_t inter, int64_t topk) {
    if (num_tokens < 0 || num_tokens > bsq::kMoeMaxTokens || topk < 1 || topk > bsq::kMoeMaxTopk ||
        hidden < 0 || hidden > (int64_t(1) << 17) || hidden % 128 != 0 || inter < 0 ||
        inter > (int64_t(1) << 17) || inter % 128 != 0) {
        fail(BSQ_ERR_INVALID_ARG, "num_tokens=%lld hidden=%lld inter=%lld topk=%lld out of range",
             (long long)num_tokens, (long long)hidden, (long long)inter, (long long)topk);
        return -1;
    }
    ok();
    return num_tokens * topk * 4 * (inter + (bsq::moe_is_few(num_tokens, topk) ? 0 : hidden));
}

int moe_few_tokens(int format, const void* x, int64_t ldx, int64_t num_tokens, int64_t hidden,
                   int64_t inter, int64_t num_experts, int64_t topk, const void* w13_codes,
                   const void* w13_scales, const void* w2_codes, const void* w2_scales,
                   const float* router_logits, int renormalize, int32_t* topk_ids,
                   float* topk_weights, void* y, int64_t ldy, void* workspace,
                   int64_t workspace_bytes, void* stream) {
    if (format != BSQ_MXFP4 && format != BSQ_MXFP8)
        return fail(BSQ_ERR_UNSUPPORTED, "format %d is not provided (MXFP4 or MXFP8 weights)", format);
    if (num_tokens < 0) return fail(BSQ_ERR_INVALID_ARG, "negative size (num_tokens=%lld)",
                                    (long long)num_tokens);
    if (num_tokens > bsq::kMoeMaxTokens)
        return fail(BSQ_ERR_UNSUPPORTED, "num_tokens=%lld: at most %d are provided",
                    (long long)num_tokens, bsq::kMoeMaxTokens);
    if (num_experts < 1 || num_experts > bsq::kMoeMaxExperts || topk < 1 ||
        topk > bsq::kMoeMaxTopk || topk > num_experts)
        return fail(BSQ_ERR_INVALID_ARG,
                    "num_experts=%lld must be in 1 .. %d and topk=%lld in 1 .. %d, at most num_experts",
                    (long long)num_experts, bsq::kMoeMaxExperts, (long long)topk, bsq::kMoeMaxTopk);
    if (hidden < 0 || inter < 0 || hidden % 128 != 0 || inter % 128 != 0 ||
        hidden > (int64_t(1) << 17) || inter > (int64_t(1) << 17))
        return fail(BSQ_ERR_INVALID_ARG,
                    "hidden=%lld and inter=%lld must be multiples of 128, at most 2^17",
                    (long long)hidden, (long long)inter);
    if (num_tokens == 0 || hidden == 0) return ok();
    if (inter == 0) return fail(BSQ_ERR_INVALID_ARG, "inter must not be 0");
    int st = check_rows("x", x, ldx, hidden);
    if (st == BSQ_OK) st = check_rows("y", y, ldy, hidden);
    if (st != BSQ_OK) return st;
    if (!w13_codes || !w13_scales || !w2_codes || !w2_scales || !topk_ids || !topk_weights)
        return fail(BSQ_ERR_INVALID_ARG, "null pointer (weights, topk_ids or topk_weights)");
    if (!aligned(w13_codes, 16) || !aligned(w2_codes, 16) || !aligned(w13_scales, 4) ||
        !aligned(w2_scales, 4))
        return fail(BSQ_ERR_INVALID_ARG, "codes must be 16-byte and scales 4-byte aligned");
    const int64_t need = moe_few_tokens_workspace(num_tokens, hidden, inter, topk);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < need)
        return fail(BSQ_ERR_INVALID_ARG,
                    "workspace (%p, %lld bytes) must be 16-byte aligned and hold %lld bytes",
                    workspace, (long long)workspace_bytes, (long long)need);
    if (num_experts * (inter / 16) > kMaxInt)
        return fail(BSQ_ERR_INVALID_ARG, "problem too large for one launch");
    bsq::MoeArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.ldx = ldx;
    a.w13 = static_cast<const uint8_t*>(w13_codes);
    a.w13_scales = static_cast<const uint8_t*>(w13_scales);
    a.w2 = static_cast<const uint8_t*>(w2_codes);
    a.w2_scales = static_cast<const uint8_t*>(w2_scales);
    a.logits = router_logits;
    a.ids = topk_ids;
    a.weights = topk_weights;
    a.h = static_cast<uint16_t*>(workspace);
    a.part = static_cast<float*>(workspace) + num_tokens * topk * inter;   // behind h
    a.y = static_cast<uint16_t*>(y);
    a.ldy = ldy;
    a.tokens = (int32_t)num_tokens;
    a.hidden = (int32_t)hidden;
    a.inter = (int32_t)inter;
    a.experts = (int32_t)num_experts;
    a.topk = (int32_t)topk;
    a.renormalize = renormalize;
    return launched(bsq::launch_moe(format, a, static_cast<hipStream_t>(stream)));
}

const char* bsq_serving_last_error(void) { return g_last_error; }

}  // extern "C"
