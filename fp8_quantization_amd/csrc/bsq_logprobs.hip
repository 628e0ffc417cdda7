// bsq_logprobs.hip -- gfx950 kernels of the log probabilities of tokens, with
// entropy and the likeliest tokens (include/bsq_decoder.h states the arithmetic).
//
// A workgroup takes a slice of a row, all of it in registers, so the largest
// logit, the sums relative to it and the slice's likeliest tokens come from one
// read.  The likeliest: the row's slice is cut into 64 parts, whose largest are
// compared first; the top-th of those is at most the top-th of all, so few
// elements reach it.  They are collected in LDS (in whatever order) and ranked by
// counting.  A row of several slices is joined by a second kernel.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "bsq_serving_internal.h"

namespace bsq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = 4;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kMostFound = 1024;     // elements that are ranked; more are taken one after the other

__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
// A number and a place in the order of the answer: the larger number, then the lower place.
// 0: nothing.
__device__ __forceinline__ uint64_t entry_of(float x, int place) {
    return (uint64_t)key_of(x) << 32 | (uint32_t)~place;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
    return v;
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, off);
        v = o > v ? o : v;
    }
    return v;
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

// V: elements of 16 bytes; N: of a thread.  A slice is kThreads * N elements of the row, counted from
// the 16-byte boundary at or before its first.
template <bool F32, int N>
__global__ void __launch_bounds__(kThreads) logprob_slice_kernel(const LogprobArgs a) {
    constexpr int V = F32 ? 4 : 8;
    __shared__ float red[3][kWaves];
    __shared__ float part[kThreads];
    __shared__ uint64_t found[kMostFound];
    __shared__ float bar;
    __shared__ uint32_t count;
    __shared__ uint64_t best[kWaves];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x / (uint32_t)a.slices;
    const int slice = (int)(blockIdx.x % (uint32_t)a.slices);
    constexpr int kSize = F32 ? 4 : 2;
    const char* p = static_cast<const char*>(a.logits) + row * a.ldl * kSize;
    const int skew = (int)((reinterpret_cast<uintptr_t>(p) & 15) / kSize);
    // element e of the thread's piece k is element at(k) + e of the row
    auto at = [&](int k) { return (slice * (N / V) + k) * (kThreads * V) + tid * V - skew; };
    if (tid == 0) count = 0;

    float x[N];
#pragma unroll
    for (int k = 0; k < N / V; ++k) {
        const int i = at(k);
        if (i >= 0 && i + V <= a.vocab) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(p + (int64_t)i * kSize);
#pragma unroll
            for (int e = 0; e < V; ++e)
                x[k * V + e] = __uint_as_float(F32 ? w[e % 4] : e % 2 ? w[e / 2 % 4] & 0xFFFF0000u : w[e / 2 % 4] << 16);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                x[k * V + e] = i + e >= 0 && i + e < a.vocab ? element<F32>(a, row, i + e) : -INFINITY;
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        x[e] = x[e] == x[e] ? x[e] : -INFINITY;
        top = fmaxf(top, x[e]);
    }
    part[tid] = top;
    const float wm = wave_max(top);
    if (lane == 0) red[0][wave] = wm;
    __syncthreads();
    const float m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    float l = 0.0f, t = 0.0f;
    if (m > -INFINITY && m < INFINITY) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float d = x[e] - m, s = __builtin_amdgcn_exp2f(d * kLog2e);
            l += s;
            t += d > -INFINITY ? s * d : 0.0f;
        }
    } else if (m == INFINITY) {      // its equals share the probability
#pragma unroll
        for (int e = 0; e < N; ++e) l += x[e] == m ? 1.0f : 0.0f;
    }
    l = wave_sum(l);
    t = wave_sum(t);
    if (lane == 0) {
        red[1][wave] = l;
        red[2][wave] = t;
    }
    if (a.top > 0 && wave == 0) {
        // the largest number that at least `top` of the 64 parts reach, to 16 bits: their best
        // elements are that many that do
        const uint32_t key = key_of(fmaxf(fmaxf(part[lane], part[lane + 64]), fmaxf(part[lane + 128], part[lane + 192])));
        uint32_t low = 0;
#pragma unroll
        for (int b = 31; b >= 16; --b) {
            const uint32_t with = low | 1u << b;
            if (__popcll(__ballot(key >= with)) >= a.top) low = with;
        }
        // up to the key of -inf all of them do
        if (lane == 0) bar = low < 0x00800000u ? -INFINITY : value_of(low);
    }
    __syncthreads();
    l = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    t = (red[2][0] + red[2][1]) + (red[2][2] + red[2][3]);
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

    const float least = bar;
    auto inside = [&](int e) { const int i = at(e / V) + e % V; return i >= 0 && i < a.vocab; };
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (x[e] >= least) {
            if (inside(e)) {
                const uint32_t n = atomicAdd(&count, 1u);
                if (n < (uint32_t)kMostFound) found[n] = entry_of(x[e], at(e / V) + e % V);
            }
        }
    }
    __syncthreads();
    const int n = (int)count;
    auto store = [&](int rank, uint64_t e) {
        if (a.slices > 1) a.best[unit * a.top + rank] = e;
        else store_top(a, row, rank, e, m, l);
    };
    if (n <= kMostFound) {
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t e = found[i];
            int rank = 0;
            for (int o = 0; o < n; ++o) rank += found[o] > e ? 1 : 0;
            if (rank < a.top) store(rank, e);
        }
        // a slice with fewer elements than that
        for (int i = n + tid; i < a.top; i += kThreads) store(i, 0);
        return;
    }
    // many equal numbers: the best below the last one, again and again
    uint64_t last = ~0ull;
    for (int r = 0; r < a.top; ++r) {
        uint64_t mine = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const uint64_t v = inside(e) ? entry_of(x[e], at(e / V) + e % V) : 0;
            if (v < last && v > mine) mine = v;
        }
        mine = wave_max(mine);
        if (lane == 0) best[wave] = mine;
        __syncthreads();
        last = max(max(best[0], best[1]), max(best[2], best[3]));
        if (tid == 0) store(r, last);
        __syncthreads();
    }
}

// A row's slices: a wave, each lane a slice.
template <bool F32>
__global__ void __launch_bounds__(64) logprob_join_kernel(const LogprobArgs a) {
    const int lane = (int)threadIdx.x;
    const int64_t row = blockIdx.x, unit = row * a.slices + lane;
    const bool on = lane < a.slices;
    const float ms = on ? a.sums[3 * unit] : -INFINITY;
    float l = on ? a.sums[3 * unit + 1] : 0.0f, t = on ? a.sums[3 * unit + 2] : 0.0f;
    const float m = wave_max(ms);
    // sums relative to m: t of s (d + ms - m)
    const float f = ms > -INFINITY ? share(ms, m) : 0.0f;
    t = f > 0.0f ? f * (t + (ms == m ? 0.0f : (ms - m) * l)) : 0.0f;
    l = wave_sum(l * f);
    t = wave_sum(t);
    finish<F32>(a, row, m, l, t);
    // the best of the slices' next ones, again and again
    const uint64_t* mine = a.best + unit * a.top;
    int next = 0;
    uint64_t head = on && a.top > 0 ? mine[0] : 0;
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
        hipLaunchKernelGGL((logprob_join_kernel<F32>), dim3((uint32_t)a.rows), dim3(64), 0, stream, a);
}

constexpr int kLong = 32, kShort = 8;                // elements of a thread

}  // namespace

// Slices of 8192 elements, or of 2048 where a row's are 64 at most and the rows are few.  A row
// may begin inside 16 bytes: 7 elements more.
void plan_logprobs(LogprobArgs& a) {
    const int64_t span = (int64_t)a.vocab + 7;
    a.slices = (int32_t)((span + kThreads * kLong - 1) / (kThreads * kLong));
    a.per_thread = kLong;
    const int64_t fine = (span + kThreads * kShort - 1) / (kThreads * kShort);
    if (fine <= 64 && a.rows * a.slices < 512) {
        a.slices = (int32_t)fine;
        a.per_thread = kShort;
    }
}

hipError_t launch_logprobs(const LogprobArgs& a, bool f32, hipStream_t stream) {
    if (a.per_thread == kLong) f32 ? logprobs<true, kLong>(a, stream) : logprobs<false, kLong>(a, stream);
    else f32 ? logprobs<true, kShort>(a, stream) : logprobs<false, kShort>(a, stream);
    return hipGetLastError();
}

}  // namespace bsq
