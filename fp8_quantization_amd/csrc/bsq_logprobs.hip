// bsq_logprobs.hip -- gfx950 kernels of the log probabilities of tokens, with
// entropy and the likeliest tokens (include/bsq_decoder.h states the arithmetic).
//
// A workgroup takes a slice of a row, a chunk in registers after the other, so
// the sums and the slice's likeliest tokens come from one read.  The likeliest: the
// first chunk is cut into 64 parts, whose largest are compared; the top-th of
// those is at most the top-th of all, so few elements reach it.  They are
// collected in LDS (in whatever order) and ranked by counting.  A row of several
// slices is joined by a second kernel.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "bsq_serving_internal.h"
#include "bsq_wave.h"

namespace bsq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = 4;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kMostFound = 2048;     // elements that are ranked at most
constexpr int kFew = 256;            // and of a row's slices

// A number and a place in the order of the answer: the larger number, then the lower place.
// 0: nothing.
__device__ __forceinline__ uint64_t entry_of(float x, int place) {
    return (uint64_t)key_of(x) << 32 | (uint32_t)~place;
}

// exp(x - m); 1 where both are the same infinity, 0 for x = -inf.
__device__ __forceinline__ float share(float x, float m) {
    return x == m ? 1.0f : __builtin_amdgcn_exp2f((x - m) * kLog2e);
}

// The log probability of z: relative to the largest logit m, whose sum of shares is l.
__device__ __forceinline__ float logprob(float z, float m, float log_l) {
    if (!(z > -INFINITY)) return -INFINITY;
    return (z == m ? 0.0f : z - m) - log_l;
}

template <bool F32>
__device__ __forceinline__ float element(const LogprobArgs& a, int64_t row, int64_t i) {
    float x;
    if constexpr (F32) x = static_cast<const float*>(a.logits)[row * a.ldl + i];
    else x = __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[row * a.ldl + i] << 16);
    return x == x ? x : -INFINITY;
}

// A row's results from its sums; every thread of the workgroup.
template <bool F32>
__device__ __forceinline__ void finish(const LogprobArgs& a, int64_t row, float m, float l, float t) {
    const float log_l = __builtin_amdgcn_logf(l) * kLn2;
    if (a.entropy && threadIdx.x == 0) a.entropy[row] = m == -INFINITY ? 0.0f : fmaxf(log_l - t / l, 0.0f);
    for (int i = (int)threadIdx.x; i < a.num_tokens; i += (int)blockDim.x) {
        const int32_t id = a.tokens[row * a.num_tokens + i];
        const bool there = id >= 0 && id < a.vocab;
        a.logprobs[row * a.num_tokens + i] = there ? logprob(element<F32>(a, row, id), m, log_l) : -INFINITY;
    }
}
__device__ __forceinline__ void store_top(const LogprobArgs& a, int64_t row, int rank, uint64_t e, float m, float l) {
    a.top_ids[row * a.top + rank] = (int32_t)~(uint32_t)e;
    a.top_logprobs[row * a.top + rank] =
        logprob(value_of((uint32_t)(e >> 32)), m, __builtin_amdgcn_logf(l) * kLn2);
}

// Logits up to this size take the fast sums; others the careful ones.  Below -kFar all count as 0
// beside a largest one above -kNear.
constexpr float kFar = 16384.0f, kNear = 16000.0f;

// A thread's sums of the elements it has seen: of 2^y and y 2^y, y = z log2(e) - ref.
struct Sums {
    float m = -INFINITY;             // the largest
    float l = 0.0f, t = 0.0f;
    // y's reference for a largest logit m
    static __device__ __forceinline__ float ref(float m) { return m == -INFINITY ? 0.0f : m * kLog2e; }
    // The sums relative to a logit that is no smaller than m.
    __device__ __forceinline__ void move(float to) {
        const float d = m == -INFINITY ? 0.0f : ref(m) - ref(to), f = __builtin_amdgcn_exp2f(d);
        t = f * __builtin_fmaf(d, l, t);
        l *= f;
        m = to;
    }
    // What m log2(e) loses as a number of 32 bits: the sums are relative to it, not to m.
    static __device__ __forceinline__ float lost(float m) {
        return m == -INFINITY ? 0.0f : __builtin_fmaf(m, kLog2e, -ref(m));
    }
};

// Elements first .. end of a row that one workgroup takes, in ways that hold for any numbers: the
// sums, and the best of a slice with many equal ones.  x(i) is element i.
template <bool F32>
struct Careful {
    const LogprobArgs& a;
    int64_t row;
    int first, end;
    float* red;                      // [kWaves]
    __device__ __forceinline__ float x(int i) const { return element<F32>(a, row, i); }
    __device__ __forceinline__ float all_sum(float v) const {
        v = wave_sum(v);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        return (red[0] + red[1]) + (red[2] + red[3]);
    }
    // m, and l and t in units of e
    __device__ void sums(float& m, float& l, float& t) const {
        m = -INFINITY;
        for (int i = first + (int)threadIdx.x; i < end; i += kThreads) m = fmaxf(m, x(i));
        m = wave_max(m);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
        __syncthreads();
        m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        l = t = 0.0f;
        for (int i = first + (int)threadIdx.x; i < end; i += kThreads) {
            const float v = x(i);
            if (v == -INFINITY) continue;
            const float s = share(v, m);
            l += s;
            t += v == m || s == 0.0f ? 0.0f : s * (v - m);
        }
        l = all_sum(l);
        t = all_sum(t);
    }
    template <class F>
    __device__ __forceinline__ int count(F f) const {
        int n = 0;
        for (int i = first + (int)threadIdx.x; i < end; i += kThreads) n += f(i) ? 1 : 0;
        return (int)all_sum((float)n);   // at most 2^19: exact
    }
    // The lowest entry of the `top` best: its number by halving, then its place.
    __device__ uint64_t least(int top) const {
        uint32_t key = 0;
        for (int b = 31; b >= 0; --b) {
            const uint32_t with = key | 1u << b;
            if (count([&](int i) { return key_of(x(i)) >= with; }) >= top) key = with;
        }
        const int over = count([&](int i) { return key_of(x(i)) > key; });
        int lo = first, hi = end - 1;    // the lowest place by which there are enough
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            if (over + count([&](int i) { return i <= mid && key_of(x(i)) == key; }) >= top) hi = mid;
            else lo = mid + 1;
        }
        return (uint64_t)key << 32 | (uint32_t)~lo;
    }
};

// A slice is a.chunks chunks of kThreads * N elements of the row, counted from the 16-byte boundary
// at or before its first; each thread keeps sums of its own, relative to the largest it has
// seen, until the end.  Bound by the vector instructions beside the reads: an element takes some
// seven, among them an exponential.
template <bool F32, int N>
__global__ void __launch_bounds__(kThreads, F32 ? 6 : 8) logprob_slice_kernel(const LogprobArgs a) {
    constexpr int V = F32 ? 4 : 8, K = N / V;            // elements and number of a thread's loads
    constexpr int kChunk = kThreads * N, kSize = F32 ? 4 : 2;
    __shared__ float red[3][kWaves];
    __shared__ float part[kThreads];
    __shared__ uint64_t found[kMostFound];
    __shared__ float bar;
    __shared__ uint32_t count, odd, far;
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x / (uint32_t)a.slices;
    const int slice = (int)(blockIdx.x % (uint32_t)a.slices);
    const char* p = static_cast<const char*>(a.logits) + row * a.ldl * kSize;
    const int skew = (int)((reinterpret_cast<uintptr_t>(p) & 15) / kSize);
    const int begin = slice * a.chunks * kChunk - skew;  // may lie before the row
    const int first = max(begin, 0), end = min(begin + a.chunks * kChunk, a.vocab);
    if (tid == 0) count = odd = far = 0;
    __syncthreads();

    // a chunk's pieces of the thread, k * kThreads + tid; past the slice -inf
    auto fetch = [&](int chunk, u32x4 (&w)[K]) {
        const int at = begin + chunk * kChunk;
        if (at >= first && at + kChunk <= end) {
            const char* from = p + (int64_t)at * kSize;
#pragma unroll
            for (int k = 0; k < K; ++k)
                w[k] = *reinterpret_cast<const u32x4*>(from + (uint32_t)(k * kThreads + tid) * 16);
            return;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = at + (k * kThreads + tid) * V;
            if (i >= first && i + V <= end) {
                w[k] = *reinterpret_cast<const u32x4*>(p + (int64_t)i * kSize);
                continue;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (F32) {
                    w[k][e] = i + e >= first && i + e < end ? __float_as_uint(element<F32>(a, row, i + e)) : 0xFF800000u;
                } else {
                    const int j = i + 2 * e;
                    const uint32_t lo = j >= first && j < end ? __float_as_uint(element<F32>(a, row, j)) >> 16 : 0xFF80u;
                    const uint32_t hi = j + 1 >= first && j + 1 < end ? __float_as_uint(element<F32>(a, row, j + 1)) : 0xFF800000u;
                    w[k][e] = lo | (hi & 0xFFFF0000u);
                }
            }
        }
    };
    Sums sum;
    bool strange = false, low = false;   // NaN or large numbers; numbers below -kFar alone
    float least = INFINITY, highest = -INFINITY;
    u32x4 next[K];
    fetch(0, next);
    for (int chunk = 0; chunk < a.chunks; ++chunk) {
        if (begin + chunk * kChunk >= a.vocab) break;
        float x[N];
#pragma unroll
        for (int e = 0; e < N; ++e)
            x[e] = __uint_as_float(F32 ? next[e / V][e % 4]
                                       : e % 2 ? next[e / V][e % V / 2] & 0xFFFF0000u : next[e / V][e % V / 2] << 16);
        if (chunk + 1 < a.chunks) fetch(chunk + 1, next);
        float top = x[0];            // NaN if there is one
#pragma unroll
        for (int e = 1; e < N; ++e) top = __builtin_elementwise_maximum(top, x[e]);
        strange |= !(top <= kFar);
        low |= top < -kFar && top > -INFINITY;
        highest = __builtin_elementwise_maximum(highest, top);
        if (a.top > 0 && (chunk & (chunk - 1)) == 0) {
            // The largest number that at least `top` of 64 parts of what was read reach, to 16
            // bits: their best elements are that many that do.  Again after 1, 2, 4, ... chunks.
            part[tid] = highest;
            __syncthreads();
            if (wave == 0) {
                float v = part[lane];
#pragma unroll
                for (int i = 1; i < kWaves; ++i) v = __builtin_elementwise_maximum(v, part[lane + 64 * i]);
                const uint32_t key = key_of(v);
                uint32_t low = 0;
#pragma unroll
                for (int b = 31; b >= 16; --b) {
                    const uint32_t with = low | 1u << b;
                    if (__popcll(__ballot(key >= with)) >= a.top) low = with;
                }
                // too few parts with a number: every number
                if (lane == 0) bar = low < 0x00800000u ? -3.402823466e38f : value_of(low);
            }
            __syncthreads();
            least = bar;
        }
        if (top >= -kFar && top <= kFar) {
            if (top > sum.m) sum.move(top);
            const float ref = Sums::ref(sum.m), before = sum.t;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float y = __builtin_fmaf(x[e], kLog2e, -ref), s = __builtin_amdgcn_exp2f(y);
                sum.l += s;
                sum.t = __builtin_fmaf(s, y, sum.t);
            }
            if (sum.t != sum.t) {    // 0 times -inf: some logits are
                sum.t = before;
                float again = ref;   // hidden, or the ys of all elements wait here in registers
                asm volatile("" : "+v"(again));
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float y = fmaxf(__builtin_fmaf(x[e], kLog2e, -again), -200.0f);
                    sum.t = __builtin_fmaf(__builtin_amdgcn_exp2f(y), y, sum.t);
                }
            }
        }
        if (a.top > 0 && __any(top >= least)) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if (!__any(x[e] >= least)) continue;
                if (x[e] >= least) {
                    const uint32_t n = atomicAdd(&count, 1u);
                    if (n < (uint32_t)kMostFound)
                        found[n] = entry_of(x[e], begin + chunk * kChunk + (e / V * kThreads + tid) * V + e % V);
                }
            }
        }
    }
    const float wm = wave_max(sum.m);
    if (lane == 0) red[0][wave] = wm;
    if (strange) odd = 1;
    if (low) far = 1;
    __syncthreads();
    float m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    sum.move(m);
    const float wl = wave_sum(sum.l), wt = wave_sum(sum.t);
    if (lane == 0) {
        red[1][wave] = wl;
        red[2][wave] = wt;
    }
    __syncthreads();
    float l = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    float t = (red[2][0] + red[2][1]) + (red[2][2] + red[2][3]);
    const float lost = Sums::lost(m), f = __builtin_amdgcn_exp2f(-lost);
    t = f * __builtin_fmaf(-lost, l, t) * kLn2;
    l *= f;
    const Careful<F32> careful{a, row, first, end, red[0]};
    if (odd || (far && m < -kNear)) careful.sums(m, l, t);
    const int64_t unit = row * a.slices + slice;
    if (a.slices > 1) {
        if (tid == 0) {
            a.sums[3 * unit] = m;
            a.sums[3 * unit + 1] = l;
            a.sums[3 * unit + 2] = t;
        }
    } else {
        finish<F32>(a, row, m, l, t);
    }
    if (a.top == 0) return;

    const int wanted = min(a.top, end - first);          // of this slice; negative past the row
    int n = odd ? kMostFound + 1 : (int)count;
    if (n > kMostFound && wanted > 0) {
        // many equal numbers, or odd ones: exactly the best
        const uint64_t last = careful.least(wanted);
        if (tid == 0) count = 0;
        __syncthreads();
        for (int i = first + tid; i < end; i += kThreads) {
            const uint64_t e = entry_of(careful.x(i), i);
            if (e >= last) found[atomicAdd(&count, 1u)] = e;
        }
        __syncthreads();
        n = (int)count;
    } else if (n < wanted) {
        // all the numbers there are, and the first of the -inf: among the first n + wanted elements
        __syncthreads();
        for (int i = first + tid; i < min(first + n + wanted, end); i += kThreads)
            if (careful.x(i) == -INFINITY) found[atomicAdd(&count, 1u)] = entry_of(-INFINITY, i);
        __syncthreads();
        n = (int)count;
    }
    auto store = [&](int rank, uint64_t e) {
        if (a.slices > 1) a.best[unit * a.top + rank] = e;
        else store_top(a, row, rank, e, m, l);
    };
    for (int i = tid; i < n; i += kThreads) {
        const uint64_t e = found[i];
        int rank = 0;
        for (int o = 0; o < n; ++o) rank += found[o] > e ? 1 : 0;
        if (rank < a.top) store(rank, e);
    }
    // a slice with fewer elements than that
    for (int i = max(wanted, 0) + tid; i < a.top; i += kThreads) store(i, 0);
}

// A row's slices: a wave, each lane a slice, whose best wait in LDS.
template <bool F32>
__global__ void __launch_bounds__(64) logprob_join_kernel(const LogprobArgs a) {
    extern __shared__ uint64_t lists[];
    const int lane = (int)threadIdx.x;
    const int64_t row = blockIdx.x, unit = row * a.slices + lane;
    const bool on = lane < a.slices;
    for (int i = lane; i < a.slices * a.top; i += 64) lists[i] = a.best[row * a.slices * a.top + i];
    const float ms = on ? a.sums[3 * unit] : -INFINITY;
    float l = on ? a.sums[3 * unit + 1] : 0.0f, t = on ? a.sums[3 * unit + 2] : 0.0f;
    const float m = wave_max(ms);
    // sums relative to m: t of s (d + ms - m)
    const float f = ms > -INFINITY ? share(ms, m) : 0.0f;
    t = f > 0.0f ? f * (t + (ms == m ? 0.0f : (ms - m) * l)) : 0.0f;
    l = wave_sum(l * f);
    t = wave_sum(t);
    finish<F32>(a, row, m, l, t);
    if (a.top == 0) return;
    __syncthreads();
    const uint64_t* mine = lists + lane * a.top;
    uint64_t head = on ? mine[0] : 0;
    // As in a slice: the top-th of the lists' first entries (their numbers) is at most the top-th
    // of all.  The entries that reach it are ranked by counting (the 20 best of 63 lists:
    // 14.6 us a call, by the rounds below 17.4).
    __shared__ uint64_t found[kFew];
    __shared__ uint32_t count;
    uint32_t bar = 0;
#pragma unroll
    for (int b = 31; b >= 0; --b) {
        const uint32_t with = bar | 1u << b;
        if (__popcll(__ballot((uint32_t)(head >> 32) >= with)) >= a.top) bar = with;
    }
    if (bar > 0) {
        if (lane == 0) count = 0;
        __syncthreads();
        for (int i = 0; on && i < a.top; ++i) {
            const uint64_t e = mine[i];
            if ((uint32_t)(e >> 32) < bar) break;
            const uint32_t n = atomicAdd(&count, 1u);
            if (n >= (uint32_t)kFew) break;
            found[n] = e;
        }
        __syncthreads();
        const int n = (int)count;
        if (n <= kFew) {
            for (int i = lane; i < n; i += 64) {
                const uint64_t e = found[i];
                int rank = 0;
                for (int o = 0; o < n; ++o) rank += found[o] > e ? 1 : 0;
                if (rank < a.top) store_top(a, row, rank, e, m, l);
            }
            return;
        }
    }
    // fewer lists than that, or many equal numbers: the best of the next ones, again and again
    int next = 0;
    for (int r = 0; r < a.top; ++r) {
        const uint64_t e = wave_max(head);
        if (lane == 0) store_top(a, row, r, e, m, l);
        if (head == e) {             // one lane's: places differ
            ++next;
            head = next < a.top ? mine[next] : 0;
        }
    }
}

template <bool F32, int N>
void logprobs(const LogprobArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((logprob_slice_kernel<F32, N>), dim3((uint32_t)(a.rows * a.slices)), dim3(kThreads), 0,
                       stream, a);
    if (a.slices > 1)
        hipLaunchKernelGGL((logprob_join_kernel<F32>), dim3((uint32_t)a.rows), dim3(64),
                           (uint32_t)(a.slices * a.top * sizeof(uint64_t)), stream, a);
}

// Elements of a thread and chunk.  Short ones, one chunk a workgroup, where a row fits (2000 rows of
// 1000: 8.5 us, long 11.6) or where long ones would leave few workgroups; else long ones, several
// a workgroup as long as there are kWorkgroups (2048 rows of 128000: 105 us, with 4096 workgroups
// 119, 8192 140).  Chunks a workgroup are rounded down, so a row's last slice may be short: 2000 rows
// are slices of 31 chunks and of one, 167 us in a graph where 2048, a slice each, take 112.
constexpr int kLong = 16, kShort = 8;
constexpr int64_t kWorkgroups = 2048;

}  // namespace

void plan_logprobs(LogprobArgs& a) {
    // a row may begin inside 16 bytes: 7 elements more
    const int64_t span = (int64_t)a.vocab + 7;
    const int64_t fine = (span + kThreads * kShort - 1) / (kThreads * kShort);
    const int64_t chunks = (span + kThreads * kLong - 1) / (kThreads * kLong);
    if (fine == 1 || (fine <= 64 && a.rows * chunks < kWorkgroups / 4)) {
        a.slices = (int32_t)fine;
        a.per_thread = kShort;
        a.chunks = 1;
        return;
    }
    // as many chunks a workgroup as leave kWorkgroups of them, in 64 slices at most
    a.per_thread = kLong;
    const int64_t least = (chunks + 63) / 64;
    a.chunks = (int32_t)std::min(std::max(a.rows * chunks / kWorkgroups, least), chunks);
    a.slices = (int32_t)((chunks + a.chunks - 1) / a.chunks);
}

hipError_t launch_logprobs(const LogprobArgs& a, bool f32, hipStream_t stream) {
    if (a.per_thread == kLong) f32 ? logprobs<true, kLong>(a, stream) : logprobs<false, kLong>(a, stream);
    else f32 ? logprobs<true, kShort>(a, stream) : logprobs<false, kShort>(a, stream);
    return hipGetLastError();
}

}  // namespace bsq
