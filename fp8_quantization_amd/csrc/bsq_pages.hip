// bsq_pages.hip -- gfx950 kernels that manage the pages of the key/value
// cache: copies, giving out, sharing, giving back and moving together
// (include/bsq_serving.h).
//
// Giving out pages is one workgroup's work: it sums the requests' needs in
// order and walks the reference counts until that many free pages are found,
// 4096 counts a step.  Everything that moves bytes runs on many workgroups.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bsq_serving_internal.h"

namespace bsq {
namespace {

constexpr int kScanThreads = 1024, kScanWaves = kScanThreads / 64;
constexpr int kCopyThreads = 256;
// bytes of a page that one workgroup copies (four 16-byte loads a thread in flight)
constexpr int kCopyBytes = kCopyThreads * 16 * 4;

__device__ __forceinline__ int pages_of(int tokens) { return (int)(((int64_t)tokens + kKvPage - 1) / kKvPage); }

// Exclusive prefix sum over the workgroup's threads; total gets the sum.  `tmp` holds
// kScanWaves numbers, free again when the call returns.
template <typename T>
__device__ __forceinline__ T block_prefix(T v, T* tmp, T& total) {
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    T x = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const T y = __shfl_up(x, off);
        if (lane >= off) x += y;
    }
    if (lane == 63) tmp[wave] = x;
    __syncthreads();
    T before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kScanWaves; ++w) {
        const T t = tmp[w];
        before += w < wave ? t : 0;
        all += t;
    }
    __syncthreads();
    total = all;
    return before + x - v;
}

// What a request asks for: `pages` pages to be written to table entries
// first .. of row `slot`; bad: its status when it cannot be served at all.
struct Request {
    int slot, first, pages, bad;
};
template <bool FORK>
__device__ __forceinline__ Request request(const PageArgs& p, int i) {
    Request r{0, 0, 0, 0};
    const int a = p.a[i], b = p.b[i];
    r.slot = FORK ? b : a;
    if (a < 0 || a >= p.num_seqs || r.slot < 0 || r.slot >= p.num_seqs) {
        r.bad = 2;
        return r;
    }
    const int len = p.kv_lens[a];
    const int64_t room = (int64_t)p.max_pages * kKvPage;
    if (len < 0 || len > room || (!FORK && (b < 0 || (int64_t)len + b > room))) {
        r.bad = 1;
        return r;
    }
    if constexpr (FORK) {
        r.first = len / kKvPage;
        r.pages = len % kKvPage != 0;
    } else {
        r.first = pages_of(len);
        r.pages = pages_of(len + b) - r.first;
    }
    return r;
}

// SMALL: at most kScanThreads requests, one a thread, which stay in LDS; others are read
// again where they are needed, their ranks kept in status (32 requests: 6.4 us against 7.9).
// A chain of dependent loads and barriers bounds it, not its bytes.
template <bool FORK, bool SMALL>
__global__ void __launch_bounds__(kScanThreads) give_out_kernel(const PageArgs p) {
    __shared__ int tmp[kScanWaves];
    __shared__ int64_t needs[kScanWaves];
    __shared__ Request kept[SMALL ? kScanThreads : 1];
    __shared__ int ranks[SMALL ? kScanThreads : 1];
    const int tid = (int)threadIdx.x;
    // the first step's counts, while the requests are read
    int ref[4];
    auto load_counts = [&](int64_t b0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t b = b0 + 4 * tid + k;
            ref[k] = b < p.cache.num_pages ? p.refcounts[b] : 1;
        }
    };
    load_counts(0);
    // the rank of request i's first page
    auto rank_of = [&](int i) { return SMALL ? ranks[i] : p.status[i]; };
    auto request_of = [&](int i) { return SMALL ? kept[i] : request<FORK>(p, i); };
    int64_t need = 0;
    for (int i0 = 0; i0 < p.n; i0 += kScanThreads) {
        const int i = i0 + tid;
        Request r{0, 0, 0, 0};
        if (i < p.n) r = request<FORK>(p, i);
        // in 64 bits: a step's requests may name 2^10 times 2^25 pages
        int64_t total;
        const int64_t before = block_prefix((int64_t)r.pages, needs, total);
        // ranks past every page stay past every page
        const int rank = (int)min(need + before, (int64_t)0x7FFFFFFF);
        if (SMALL) {
            kept[tid] = r;
            ranks[tid] = rank;
        } else if (i < p.n) {
            p.status[i] = rank;
        }
        need += total;
    }
    __syncthreads();
    int64_t found = 0;
    for (int64_t b0 = 0; b0 < p.cache.num_pages && found < need; b0 += 4 * kScanThreads) {
        if (b0 > 0) load_counts(b0);
        const int64_t b = b0 + 4 * tid;
        int v = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) v += ref[k] == 0;
        int total;
        int64_t rank = found + block_prefix(v, tmp, total);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (ref[k] != 0) continue;
            if (rank < need) {
                int lo = 0, hi = p.n;              // the last request whose rank is at most this one
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (rank_of(mid) <= rank) lo = mid; else hi = mid;
                }
                const Request r = request_of(lo);
                const int64_t at = r.first + (rank - rank_of(lo));
                if (!r.bad && at < p.max_pages) {
                    p.table[r.slot * p.table_stride + at] = (int32_t)(b + k);
                    p.refcounts[b + k] = 1;
                }
            }
            ++rank;
        }
        found += total;
    }
    __syncthreads();
    for (int i = tid; i < p.n; i += kScanThreads) {
        const Request r = request_of(i);
        const int64_t start = rank_of(i);
        int st = r.bad;
        if (!st && r.pages > 0 && start + r.pages > found) {
            st = 1;                                // pages it was given already go back
            for (int64_t k = 0; k < r.pages && start + k < found; ++k) {
                const int page = p.table[r.slot * p.table_stride + r.first + k];
                if (page >= 0 && page < p.cache.num_pages) p.refcounts[page] = 0;
            }
        }
        p.status[i] = st;
        if constexpr (FORK) {
            if (r.bad != 2) p.kv_lens[r.slot] = st ? 0 : p.kv_lens[p.a[i]];
        } else {
            if (!st) p.kv_lens[r.slot] += p.b[i];
        }
    }
}

template <bool FORK>
void give_out(const PageArgs& p, hipStream_t stream) {
    if (p.n <= kScanThreads)
        hipLaunchKernelGGL((give_out_kernel<FORK, true>), dim3(1), dim3(kScanThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((give_out_kernel<FORK, false>), dim3(1), dim3(kScanThreads), 0, stream, p);
}

// Part `part` (of parts_of) of a page's copy.
__host__ __device__ inline int parts_of(const KvCache& c) {
    const int64_t bytes = 2 * (int64_t)c.num_heads * c.head_dim * kKvPage;
    return (int)((bytes + kCopyBytes - 1) / kCopyBytes);
}
// AWAY: pages not read again at once pass the caches by (8192 pages of 128 KiB half in use
// moved together in 104 us against 111).
template <bool AWAY>
__device__ __forceinline__ void copy_part(const KvCache& c, int64_t src, int64_t dst, int part) {
    typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
    const int64_t half = (int64_t)c.num_heads * c.head_dim * kKvPage;   // a multiple of 4096
    u32x4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t o = (int64_t)part * kCopyBytes + (k * kCopyThreads + (int)threadIdx.x) * 16;
        if (o >= 2 * half) break;
        const u32x4* from = reinterpret_cast<const u32x4*>(
            (o < half ? c.k_codes + o : c.v_codes + (o - half)) + src * c.page_stride);
        if constexpr (AWAY) v[k] = __builtin_nontemporal_load(from);
        else v[k] = *from;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t o = (int64_t)part * kCopyBytes + (k * kCopyThreads + (int)threadIdx.x) * 16;
        if (o >= 2 * half) break;
        u32x4* to = reinterpret_cast<u32x4*>((o < half ? c.k_codes + o : c.v_codes + (o - half)) +
                                             dst * c.page_stride);
        if constexpr (AWAY) __builtin_nontemporal_store(v[k], to);
        else *to = v[k];
    }
    if (part == 0)
        for (int h = (int)threadIdx.x; h < c.num_heads; h += kCopyThreads) {
            c.k_scales[dst * c.scale_stride + h] = c.k_scales[src * c.scale_stride + h];
            c.v_scales[dst * c.scale_stride + h] = c.v_scales[src * c.scale_stride + h];
        }
}

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const PageArgs p, int parts) {
    const int i = (int)(blockIdx.x / (uint32_t)parts), part = (int)(blockIdx.x % (uint32_t)parts);
    const int src = p.a[i], dst = p.b[i];
    if (src < 0 || src >= p.cache.num_pages || dst < 0 || dst >= p.cache.num_pages || src == dst)
        return;
    copy_part<true>(p.cache, src, dst, part);
}

// After give_out_kernel<true>: workgroup 0 of a fork shares the full pages, the others
// copy the parts of the last one.
__global__ void __launch_bounds__(kCopyThreads) fork_kernel(const PageArgs p, int parts) {
    const int i = (int)(blockIdx.x / (uint32_t)(parts + 1));
    const int part = (int)(blockIdx.x % (uint32_t)(parts + 1)) - 1;
    if (p.status[i] != 0) return;
    const int parent = p.a[i], child = p.b[i];     // both inside the table (status 0)
    const int len = p.kv_lens[child], full = len / kKvPage;
    const int32_t* from = p.table + parent * p.table_stride;
    int32_t* to = p.table + child * p.table_stride;
    if (part < 0) {
        for (int k = (int)threadIdx.x; k < full; k += kCopyThreads) {
            const int page = from[k];
            to[k] = page;
            if (page >= 0 && page < p.cache.num_pages) atomicAdd(p.refcounts + page, 1);
        }
    } else if (len % kKvPage != 0) {
        const int src = from[full], dst = to[full];
        if (src >= 0 && src < p.cache.num_pages && dst >= 0 && dst < p.cache.num_pages)
            copy_part<false>(p.cache, src, dst, part);
    }
}

__global__ void __launch_bounds__(kCopyThreads) pages_free_kernel(const PageArgs p) {
    __shared__ int held;
    const int slot = p.a[blockIdx.x];
    if (slot < 0 || slot >= p.num_seqs) return;
    // taken, not read: a slot named twice is freed once
    if (threadIdx.x == 0) held = atomicExch(p.kv_lens + slot, 0);
    __syncthreads();
    const int used = held < 0 ? 0 : min(pages_of(held), p.max_pages);
    for (int k = (int)threadIdx.x; k < used; k += kCopyThreads) {
        const int page = p.table[slot * p.table_stride + k];
        if (page >= 0 && page < p.cache.num_pages) atomicSub(p.refcounts + page, 1);
    }
}

// ------------------------------------------------------------ compaction

// The moves and the new counts, by one workgroup: count the pages in use
// (n), list those at n and above and the free ones below n, both in order
// (there are as many), and pair them.
__global__ void __launch_bounds__(kScanThreads) compact_plan_kernel(const CompactArgs p) {
    __shared__ int tmp[kScanWaves];
    const int tid = (int)threadIdx.x, N = p.cache.num_pages;
    // the first kKept steps' counts stay in registers
    constexpr int kKept = 4;
    int ref[kKept][4], mine = 0, live;
#pragma unroll
    for (int s = 0; s < kKept; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t i = (int64_t)s * 4 * kScanThreads + 4 * tid + k;
            ref[s][k] = i < N ? p.refs[i] : 0;
        }
#pragma unroll
    for (int s = 0; s < kKept; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) mine += ref[s][k] > 0;
    for (int64_t b = kKept * 4 * kScanThreads + 4 * tid; b < N; b += 4 * kScanThreads)
#pragma unroll
        for (int k = 0; k < 4; ++k) mine += b + k < N && p.refs[b + k] > 0;
    block_prefix(mine, tmp, live);
    int32_t* src = p.moves + 4;
    int32_t* dst = src + N / 2 + 1;
    int32_t* renumber = dst + N / 2 + 1;           // of pages n and above
    int n_src = 0, n_dst = 0;
    auto step = [&](int64_t b0, const int (&ref)[4]) {
        const int64_t b = b0 + 4 * tid;
        int s[4], d[4], vs = 0, vd = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t i = b + k;
            s[k] = i < N && i >= live && ref[k] > 0;
            d[k] = i < N && i < live && ref[k] <= 0;
            vs += s[k];
            vd += d[k];
            if (i < N && !s[k] && !d[k]) {
                p.refs_out[i] = i < live ? ref[k] : 0;
                if (i >= live) renumber[i] = (int32_t)i;
            }
        }
        // both counts in one sum: a step holds at most 4096 of either
        int total;
        const int both = block_prefix(vs | vd << 16, tmp, total);
        int rs = n_src + (both & 0xFFFF), rd = n_dst + (both >> 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (s[k]) src[rs++] = (int32_t)(b + k);
            if (d[k]) dst[rd++] = (int32_t)(b + k);
        }
        n_src += total & 0xFFFF;
        n_dst += total >> 16;
    };
#pragma unroll
    for (int s = 0; s < kKept; ++s)
        if ((int64_t)s * 4 * kScanThreads < N) step((int64_t)s * 4 * kScanThreads, ref[s]);
    for (int64_t b0 = kKept * 4 * kScanThreads; b0 < N; b0 += 4 * kScanThreads) {
        int more[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) more[k] = b0 + 4 * tid + k < N ? p.refs[b0 + 4 * tid + k] : 0;
        step(b0, more);
    }
    __syncthreads();
    for (int k = tid; k < n_src; k += kScanThreads) {
        const int from = src[k], to = dst[k], ref = p.refs[from];
        renumber[from] = to;
        p.refs_out[to] = ref;
        p.refs_out[from] = 0;
    }
    if (tid == 0) {
        p.moves[0] = n_src;
        p.moves[1] = live;
        *p.num_live = live;
    }
}

// Workgroups below table_blocks rewrite the table, the others move pages.
__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const CompactArgs p, int parts,
                                                                    int table_blocks) {
    const int N = p.cache.num_pages;
    const int32_t* src = p.moves + 4;
    const int32_t* dst = src + N / 2 + 1;
    const int32_t* renumber = dst + N / 2 + 1;
    const int64_t moves = p.moves[0], live = p.moves[1];
    if ((int)blockIdx.x < table_blocks) {
        const int64_t entries = (int64_t)p.num_seqs * p.max_pages;
        for (int64_t e = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; e < entries;
             e += (int64_t)table_blocks * kCopyThreads) {
            const int64_t s = e / p.max_pages, k = e - s * p.max_pages;
            int32_t page = p.table[s * p.table_stride + k];
            const int len = p.kv_lens[s];
            if (len > 0 && k < pages_of(len) && page >= live && page < N) page = renumber[page];
            p.table_out[s * p.table_out_stride + k] = page;
        }
        return;
    }
    for (int64_t w = blockIdx.x - table_blocks; w < moves * parts; w += gridDim.x - table_blocks)
        copy_part<true>(p.cache, src[w / parts], dst[w / parts], (int)(w % parts));
}

}  // namespace

hipError_t launch_pages_copy(const PageArgs& p, hipStream_t stream) {
    const int parts = parts_of(p.cache);
    hipLaunchKernelGGL(pages_copy_kernel, dim3((uint32_t)((int64_t)p.n * parts)),
                       dim3(kCopyThreads), 0, stream, p, parts);
    return hipGetLastError();
}

hipError_t launch_pages_reserve(const PageArgs& p, hipStream_t stream) {
    give_out<false>(p, stream);
    return hipGetLastError();
}

hipError_t launch_pages_fork(const PageArgs& p, hipStream_t stream) {
    give_out<true>(p, stream);
    const int parts = parts_of(p.cache);
    hipLaunchKernelGGL(fork_kernel, dim3((uint32_t)((int64_t)p.n * (parts + 1))),
                       dim3(kCopyThreads), 0, stream, p, parts);
    return hipGetLastError();
}

hipError_t launch_pages_free(const PageArgs& p, hipStream_t stream) {
    hipLaunchKernelGGL(pages_free_kernel, dim3((uint32_t)p.n), dim3(kCopyThreads), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_pages_compact(const CompactArgs& p, hipStream_t stream) {
    hipLaunchKernelGGL(compact_plan_kernel, dim3(1), dim3(kScanThreads), 0, stream, p);
    const int64_t entries = (int64_t)p.num_seqs * p.max_pages;
    const int64_t want = (entries + kCopyThreads - 1) / kCopyThreads;
    const int table_blocks = (int)(want > 256 ? 256 : want);
    // eight workgroups for each of the 256 CUs walk the moves, whose number only the device knows
    hipLaunchKernelGGL(compact_move_kernel, dim3((uint32_t)table_blocks + 2048), dim3(kCopyThreads),
                       0, stream, p, parts_of(p.cache), table_blocks);
    return hipGetLastError();
}

}  // namespace bsq
