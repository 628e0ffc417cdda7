// bsq_route.hip -- gfx950 kernels of the routing to experts and of the grouped
// rows that follow from it (include/bsq_decoder.h states the arithmetic).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "bsq_serving_internal.h"
#include "bsq_wave.h"

namespace bsq {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr float kLog2e = 1.44269504088896340736f;

// ------------------------------------------------------------ routing
//
// A wave a token, expert e in lane e % 64 of register e / 64.  The topk largest
// are taken one after the other by the wave's largest key, a number's bits in
// an order of unsigned integers (0: not to be chosen).  Few tokens are bound by
// latency: 64 of 256 experts, 8 chosen, take 3.8 us in a graph by logits alone
// (1 chosen 2.6, an empty kernel 1.6), 5.6 with a bias, 7.0 with a bias and 8
// groups by sums of two (1 chosen 4.8).  Many are bound by the instructions: 16384
// tokens with bias and groups take 28 us (with every score in 64 bits 33).  Where
// logits alone choose, four tokens may share a wave.

// A logit; NaN counts as -inf.
template <bool F32>
__device__ __forceinline__ float logit(const RouteArgs& a, int64_t token, int e) {
    float x;
    if constexpr (F32) x = static_cast<const float*>(a.logits)[token * a.ldl + e];
    else x = __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[token * a.ldl + e] << 16);
    return x == x ? x : -INFINITY;
}
// A bias; NaN counts as -inf.
__device__ __forceinline__ float bias_of(const RouteArgs& a, int e) {
    if (!a.bias) return 0.0f;
    const float b = a.bias[e];
    return b == b ? b : -INFINITY;
}

// exp(x - top), and 1 where both are the same infinity.
__device__ __forceinline__ float share(float x, float top) {
    if (!(x > -INFINITY)) return 0.0f;
    return x == top ? 1.0f : __builtin_amdgcn_exp2f((x - top) * kLog2e);
}

// Whether what 32 bits put in this order is in it: a before b, which are off by `off` at most
// between them, and by a rounding each.
__device__ __forceinline__ bool surely(float a, float b, float off) {
    if (b == -INFINITY) return a > -INFINITY;
    return a - b > off + (__builtin_fabsf(a) + __builtin_fabsf(b)) * 0x1p-21f;
}

// A lane's choice: an expert and its logit, -inf where it has no weight.
struct Choice {
    int id = 0;
    float z = -INFINITY;
};
__device__ __forceinline__ float of_lane(float v, int lane) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ double of_lane(double v, int lane) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

// The topk largest keys, the lowest expert among equals: lane j gets the j-th.  x: the logits.
// CHECK: ok becomes false where the order of those and the next is not sure.
template <int REGS, bool CHECK, class K>
__device__ __forceinline__ Choice choose(K (&key)[REGS], const float (&x)[REGS],
                                         const float (&bias)[REGS], int topk, float off, bool& ok) {
    const int lane = (int)threadIdx.x & 63;
    Choice c;
    float last = INFINITY;
    for (int j = 0; j < topk + (CHECK ? 1 : 0); ++j) {
        K best = key[0];
#pragma unroll
        for (int k = 1; k < REGS; ++k) best = max(best, key[k]);
        best = wave_max(best);
        if constexpr (CHECK) {
            if (best == 0) break;    // no more to be chosen
            const float v = value_of(best);
            if (j > 0) ok = ok && surely(last, v, off);
            last = v;
            if (j == topk) break;
        }
        bool taken = false;
#pragma unroll
        for (int k = 0; k < REGS; ++k) {
            const uint64_t at = __ballot(key[k] == best);
            if (!taken && at) {
                taken = true;
                const int l = __ffsll((unsigned long long)at) - 1;
                const float z = of_lane(bias[k] > -INFINITY ? x[k] : -INFINITY, l);
                if (lane == j) {
                    c.id = 64 * k + l;
                    c.z = z;
                }
                if (lane == l) key[k] = 0;
            }
        }
    }
    return c;
}

// Closes the groups that are not kept: their experts' keys become 0.  Lane g * P + i looks at
// every P-th expert of group g; `all`: the wave's numbers in LDS.  CHECK as above.
template <int REGS, bool CHECK, class K, class F>
__device__ __forceinline__ void close_groups(const RouteArgs& a, K (&key)[REGS], const F (&c)[REGS], F* all,
                                             float off, bool& ok) {
    const int lane = (int)threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < REGS; ++k)
        if (64 * k + lane < a.experts) all[64 * k + lane] = c[k];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int P = a.group_lanes, g = lane / P, first = g * a.group_size;
    F one = -INFINITY, two = -INFINITY;
    if (g < a.groups)
        for (int e = lane % P; e < a.group_size; e += P) {
            const F v = all[first + e];
            two = v > one ? one : v > two ? v : two;
            one = v > one ? v : one;
        }
    for (int by = P / 2; by >= 1; by >>= 1) {
        const F o1 = __shfl_xor(one, by), o2 = __shfl_xor(two, by);
        two = o1 > one ? (one > o2 ? one : o2) : (two > o1 ? two : o1);
        one = o1 > one ? o1 : one;
    }
    F score = one;
    if (a.group_top == 2 && a.group_size > 1) score = one == -INFINITY || two == -INFINITY ? -INFINITY : one + two;
    // how many groups go before this one
    int before = 0;
    for (int o = 0; o < a.groups; ++o) {
        const F v = of_lane(score, o * P);
        before += v > score || (v == score && o < g) ? 1 : 0;
    }
    const bool group = g < a.groups && lane % P == 0, keep = group && before < a.keep;
    const uint64_t kept = __ballot(keep);
    if constexpr (CHECK) {           // the lowest kept, the highest not
        const float in = -wave_max(keep ? -score : -INFINITY);
        const float out = wave_max(group && !keep ? score : -INFINITY);
        ok = a.keep == a.groups || surely(in, out, 2.0f * off);
    }
#pragma unroll
    for (int k = 0; k < REGS; ++k) {
        const int e = 64 * k + lane;
        const int group = (int)(((uint32_t)e * a.group_magic) >> 20);
        if (e < a.experts && !((kept >> (group * P)) & 1)) key[k] = 0;
    }
    __builtin_amdgcn_wave_barrier();
}

// The weights of a token's experts, lane j's having the logit z (past topk -inf).
template <int REGS>
__device__ __forceinline__ float weight_of(const RouteArgs& a, float z, const float (&x)[REGS]) {
    float s, sum;
    if (a.sigmoid) {
        // where every chosen logit is negative their scores are taken relative to the largest's
        const float top = wave_max(z), m = a.renormalize && top < 0.0f && top > -INFINITY ? top : 0.0f;
        const float t = __builtin_amdgcn_exp2f(-__builtin_fabsf(z) * kLog2e);        // exp(-|z|)
        s = (z > 0.0f ? 1.0f : share(z, m)) / (1.0f + t);
        if (!(z > -INFINITY)) s = 0.0f;
        sum = a.renormalize ? wave_sum(s) : 1.0f;
    } else {
        float top = z;
        if (!a.renormalize) {
            top = x[0];
#pragma unroll
            for (int k = 1; k < REGS; ++k) top = fmaxf(top, x[k]);
        }
        top = wave_max(top);
        s = sum = share(z, top);
        if (!a.renormalize) {
            sum = 0.0f;
#pragma unroll
            for (int k = 0; k < REGS; ++k) sum += share(x[k], top);
        } else {                     // an infinite one that is not chosen leaves the chosen nothing
            bool infinite = false;
#pragma unroll
            for (int k = 0; k < REGS; ++k) infinite |= x[k] == INFINITY;
            if (top < INFINITY && __any(infinite)) sum = 0.0f;
        }
        sum = wave_sum(sum);
    }
    return sum > 0.0f ? s / sum * a.factor : 0.0f;
}

// The choice by c in 64 bits (of experts by the logits where there is no bias).
template <int REGS>
__device__ __forceinline__ Choice choose_exactly(const RouteArgs& a, const float (&x)[REGS],
                                                 const float (&bias)[REGS], double* all) {
    const int lane = (int)threadIdx.x & 63;
    double s[REGS], sum = 0.0;
    float top = x[0];
    if (!a.sigmoid) {
#pragma unroll
        for (int k = 1; k < REGS; ++k) top = fmaxf(top, x[k]);
        top = wave_max(top);
    }
#pragma unroll
    for (int k = 0; k < REGS; ++k) {
        if (a.sigmoid) s[k] = 1.0 / (1.0 + exp(-(double)x[k]));
        else s[k] = !(x[k] > -INFINITY) ? 0.0 : x[k] == top ? 1.0 : exp((double)x[k] - (double)top);
        sum += s[k];
    }
    if (!a.sigmoid) {
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
    }
    uint64_t key[REGS];
#pragma unroll
    for (int k = 0; k < REGS; ++k) {
        const int e = 64 * k + lane;
        const float b = bias[k];
        s[k] = !(x[k] > -INFINITY) || b == -INFINITY ? -INFINITY : (a.sigmoid ? s[k] : s[k] / sum) + b;
        key[k] = e < a.experts ? key_of(a.bias ? s[k] : (double)x[k]) : 0;
    }
    bool ok;
    if (a.groups > 1) close_groups<REGS, false>(a, key, s, all, 0.0f, ok);
    return choose<REGS, false>(key, x, bias, a.topk, 0.0f, ok);
}

// The choice by c in 32 bits; ok: it is that of 64.
//   sigmoid: the exponential of x is off by 1.5 |x| + 2 in units of 2^-24 of it, 1 + t and the
//     reciprocal by 3: with s (1 - s) |x| < 0.23 and s (1 - s) <= 1/4, s by less than 4.  Two of
//     them: 2^-21; four times that is taken.
//   softmax: a share e^-d of the largest is off by (2.5 d + 2) of it, the sum by the shares' mean of
//     that (at most 2.5 log 1024 + 2) and 22 for its additions, the quotient by 2: s by less than
//     50 in units of 2^-24 of the largest s.  Two of them: 2^-17 of it; twice that is taken.
template <int REGS>
__device__ __forceinline__ Choice choose_nearly(const RouteArgs& a, const float (&x)[REGS],
                                                const float (&bias)[REGS], float* all, bool& ok) {
    const int lane = (int)threadIdx.x & 63;
    float s[REGS], off = 0x1p-19f, scale = 1.0f;
    if (!a.sigmoid) {
        float top = x[0], sum = 0.0f;
#pragma unroll
        for (int k = 1; k < REGS; ++k) top = fmaxf(top, x[k]);
        top = wave_max(top);
#pragma unroll
        for (int k = 0; k < REGS; ++k) {
            s[k] = share(x[k], top);
            sum += s[k];
        }
        scale = __builtin_amdgcn_rcpf(wave_sum(sum));
        off = scale * 0x1p-16f;
    }
    uint32_t key[REGS];
#pragma unroll
    for (int k = 0; k < REGS; ++k) {
        const int e = 64 * k + lane;
        const float b = bias[k];
        if (a.sigmoid) s[k] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[k] * -kLog2e));
        s[k] = !(x[k] > -INFINITY) || b == -INFINITY ? -INFINITY : s[k] * scale + b;
        key[k] = e < a.experts ? key_of(a.bias ? s[k] : x[k]) : 0u;
    }
    ok = true;
    if (a.groups > 1) close_groups<REGS, true>(a, key, s, all, off, ok);
    if (a.bias) return choose<REGS, true>(key, x, bias, a.topk, off, ok);
    return choose<REGS, false>(key, x, bias, a.topk, off, ok);
}

// Without a bias, and with groups by their best, c goes by the logit.
template <int REGS>
__device__ __forceinline__ Choice choose_logits(const RouteArgs& a, const float (&x)[REGS],
                                                const float (&bias)[REGS], float* all) {
    const int lane = (int)threadIdx.x & 63;
    uint32_t key[REGS];
    bool ok;
#pragma unroll
    for (int k = 0; k < REGS; ++k) key[k] = 64 * k + lane < a.experts ? key_of(x[k]) : 0u;
    if (a.groups > 1) close_groups<REGS, false>(a, key, x, all, 0.0f, ok);
    return choose<REGS, false>(key, x, bias, a.topk, 0.0f, ok);
}

template <int REGS, bool F32>
__global__ void __launch_bounds__(kThreads) moe_route_kernel(const RouteArgs a) {
    __shared__ double all[kWaves][REGS * 64];
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t token = (int64_t)blockIdx.x * kWaves + wave;
    if (token >= a.tokens) return;
    float x[REGS], bias[REGS];
#pragma unroll
    for (int k = 0; k < REGS; ++k) {
        const int e = 64 * k + lane;
        x[k] = e < a.experts ? logit<F32>(a, token, e) : -INFINITY;
        bias[k] = e < a.experts ? bias_of(a, e) : -INFINITY;
    }
    Choice c;
    if (!a.bias && (a.groups == 1 || a.group_top == 1 || a.group_size == 1)) {
        c = choose_logits(a, x, bias, reinterpret_cast<float*>(all[wave]));
    } else {
        bool ok;
        c = choose_nearly(a, x, bias, reinterpret_cast<float*>(all[wave]), ok);
        if (!ok) c = choose_exactly(a, x, bias, all[wave]);
    }
    const float w = weight_of(a, c.z, x);
    if (lane < a.topk) {
        a.ids[token * a.topk + lane] = c.id;
        a.weights[token * a.topk + lane] = w;
    }
}

// Four tokens a wave, for the choice by logits among all experts: expert 16 k + l is register k
// of lane l of the token's 16.  A round's instructions serve four tokens, but look at four times the
// registers one after the other.  In a graph, a wave a token against this:
//   64 experts:   1 token 2.4 us, 2.4;     1024 tokens 2.9, 2.7;    16384 tokens 7.7, 3.9
//   128 experts:  2048 tokens 3.4, 3.8;    4096 tokens 4.2, 3.8;    16384 tokens 9.0, 6.0
//   256 experts:  4096 tokens 5.1, 5.7;    16384 tokens 11.3, 9.5
template <int REGS, bool F32>
__global__ void __launch_bounds__(kThreads) moe_route_many_kernel(const RouteArgs a) {
    const int lane = (int)threadIdx.x & 63, l = lane & 15;
    const int64_t token = ((int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6)) * 4 + (lane >> 4);
    const bool on = token < a.tokens;
    const auto largest = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
    const auto lowest = [](uint32_t x, uint32_t y) { return x < y ? x : y; };
    const auto sum_of = [](uint32_t x, uint32_t y) { return __float_as_uint(__uint_as_float(x) + __uint_as_float(y)); };
    float x[REGS];
    uint32_t key[REGS];
#pragma unroll
    for (int k = 0; k < REGS; ++k) {
        const bool there = on && 16 * k + l < a.experts;
        x[k] = there ? logit<F32>(a, token, 16 * k + l) : -INFINITY;
        key[k] = there ? key_of(x[k]) : 0u;
    }
    uint32_t id = 0, mine = 0, top = 0;
    for (int j = 0; j < a.topk; ++j) {
        uint32_t best = key[0], at = 0;
#pragma unroll
        for (int k = 1; k < REGS; ++k) {
            at = key[k] > best ? k : at;
            best = max(best, key[k]);
        }
        const uint32_t most = row_all(best, largest);
        const uint32_t e = row_all(best == most ? 16 * at + l : 0xFFFFu, lowest);
        if (j == 0) top = most;
        if (l == j) {
            id = e;
            mine = most;
        }
#pragma unroll
        for (int k = 0; k < REGS; ++k) key[k] = e == 16u * k + l ? 0u : key[k];
    }
    // as weight_of
    const float z = l < a.topk ? value_of(mine) : -INFINITY, t = value_of(top);
    float s, sum;
    if (a.sigmoid) {
        const float m = a.renormalize && t < 0.0f && t > -INFINITY ? t : 0.0f;
        s = (z > 0.0f ? 1.0f : share(z, m)) / (1.0f + __builtin_amdgcn_exp2f(-__builtin_fabsf(z) * kLog2e));
        if (!(z > -INFINITY)) s = 0.0f;
        sum = s;
    } else {
        s = sum = share(z, t);
        if (!a.renormalize) {
            sum = 0.0f;
#pragma unroll
            for (int k = 0; k < REGS; ++k) sum += share(x[k], t);
        }
    }
    sum = __uint_as_float(row_all(__float_as_uint(sum), sum_of));
    if (a.sigmoid && !a.renormalize) sum = 1.0f;
    if (on && l < a.topk) {
        a.ids[token * a.topk + l] = (int32_t)id;
        a.weights[token * a.topk + l] = sum > 0.0f ? s / sum * a.factor : 0.0f;
    }
}

// Whether four tokens share a wave: where that is not the slower one above.
bool four_a_wave(const RouteArgs& a) {
    if (a.bias || a.groups > 1 || a.experts > 256) return false;
    return a.experts <= 64 || a.tokens >= (a.experts <= 128 ? 4096 : 8192);
}

template <int REGS>
void route_many(const RouteArgs& a, bool f32, hipStream_t stream) {
    const dim3 grid((uint32_t)((a.tokens + 4 * kWaves - 1) / (4 * kWaves)));
    if (f32) hipLaunchKernelGGL((moe_route_many_kernel<REGS, true>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((moe_route_many_kernel<REGS, false>), grid, dim3(kThreads), 0, stream, a);
}

template <int REGS>
void route(const RouteArgs& a, bool f32, hipStream_t stream) {
    const dim3 grid((uint32_t)((a.tokens + kWaves - 1) / kWaves));
    if (f32) hipLaunchKernelGGL((moe_route_kernel<REGS, true>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((moe_route_kernel<REGS, false>), grid, dim3(kThreads), 0, stream, a);
}

// ------------------------------------------------------------ grouped rows
//
// A stable counting sort.  A workgroup has a tile of consecutive entries, each of
// its waves a part of it; a wave goes through its part 64 entries at a time.
// Which of the 64 name the same expert is found by a ballot for each bit of the
// number, so an entry's rank among them is a count of lanes, and no order of
// atomics takes part.  Few entries are one workgroup's; of more, a first kernel
// finds the ranks within the tiles and the tiles' counts, and a second adds up the
// counts for each tile and places the entries.  Bound by the latency of these
// steps: 131072 entries of 256 experts take 13.4 us a call (with counts, then ranks
// and places in one kernel 20.7), 512 take 7.0.

constexpr int kSortThreads = 512, kSortWaves = kSortThreads / 64;
constexpr int kKept = 8;             // steps of a wave whose entries stay in registers

// The lanes whose number is the same.
__device__ __forceinline__ uint64_t same_lanes(int v, int bits) {
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const bool set = (v >> b) & 1;
        const uint64_t at = __ballot(set);
        m &= set ? at : ~at;
    }
    return m;
}
__device__ __forceinline__ int expert_of(const GroupArgs& a, int64_t i, int64_t end) {
    const int id = i < end ? a.ids[i] : -1;
    return id >= 0 && id < a.experts ? id : a.experts;      // experts: no expert
}

// Sums over the experts before, of n and padded: thread t has experts 2 t and 2 t + 1.
struct Offsets {
    uint32_t rows[2], scales[2], all_rows;
};
__device__ __forceinline__ Offsets offsets_of(const GroupArgs& a, const uint32_t (&n)[2],
                                              uint32_t (*sums)[kSortWaves], bool store) {
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t padded[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) padded[k] = (n[k] + a.pad - 1) / a.pad * a.pad;
    uint32_t r = n[0] + n[1], s = padded[0] + padded[1];
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t ro = __shfl_up(r, off), so = __shfl_up(s, off);
        if (lane >= off) {
            r += ro;
            s += so;
        }
    }
    if (lane == 63) {
        sums[0][wave] = r;
        sums[1][wave] = s;
    }
    __syncthreads();
    Offsets o;
    o.all_rows = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        if (w < wave) {
            r += sums[0][w];
            s += sums[1][w];
        }
        o.all_rows += sums[0][w];
    }
    r -= n[0] + n[1];
    s -= padded[0] + padded[1];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        o.rows[k] = r;
        o.scales[k] = s;
        if (store && 2 * tid + k <= a.experts) {
            a.row_offsets[2 * tid + k] = r;
            a.scales_offsets[2 * tid + k] = s;
        }
        r += n[k];
        s += padded[k];
    }
    // 1024 experts: the last offset is no thread's expert
    if (store && tid == kSortThreads - 1 && a.experts == 2 * kSortThreads) {
        a.row_offsets[a.experts] = r;
        a.scales_offsets[a.experts] = s;
    }
    return o;
}

// ALONE: all of the work.  Else the tile's ranks and counts.  KEEP: a wave has at most kKept steps.
template <bool ALONE, bool KEEP>
__global__ void __launch_bounds__(kSortThreads) group_rank_kernel(const GroupArgs a) {
    // per wave and expert: its entries, then where its next one goes
    __shared__ volatile int32_t place[kSortWaves][kMoeMaxExperts + 1];
    __shared__ uint32_t sums[2][kSortWaves];
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t first = (int64_t)blockIdx.x * a.tile, tile_end = min(first + a.tile, a.entries);
    const int64_t part = a.tile / kSortWaves;
    const int64_t from = first + wave * part, to = min(from + part, tile_end);
    const uint64_t below = (1ull << lane) - 1;

    int e[kKept], rank[kKept];
    if constexpr (KEEP) {
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            e[k] = from + 64 * k < to ? expert_of(a, from + 64 * k + lane, to) : a.experts;
    }
    for (int x = lane; x <= a.experts; x += 64) place[wave][x] = 0;
    __builtin_amdgcn_wave_barrier();
    // one step: the entry's rank among the wave's of its expert so far
    const auto step = [&](int x) {
        const uint64_t m = same_lanes(x, a.bits);
        const int r = place[wave][x] + __popcll(m & below);
        __builtin_amdgcn_wave_barrier();
        if (!(m & below)) place[wave][x] = r + __popcll(m);
        __builtin_amdgcn_wave_barrier();
        return r;
    };
    if constexpr (KEEP) {
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            if (from + 64 * k < to) rank[k] = step(e[k]);
    } else {
        for (int64_t i = from; i < to; i += 64) step(expert_of(a, i + lane, to));
    }
    __syncthreads();
    // thread t: experts 2 t and 2 t + 1; their counts, the waves' places within the tile
    uint32_t n[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int x = 2 * tid + k;
        if (x >= a.experts) continue;
        int32_t run = 0;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const int32_t c = place[w][x];
            place[w][x] = run;
            run += c;
        }
        n[k] = (uint32_t)run;
        if (!ALONE) a.counts[(int64_t)blockIdx.x * a.experts + x] = run;
    }
    uint32_t rows = 0;
    if constexpr (ALONE) {
        const Offsets o = offsets_of(a, n, sums, true);
        rows = o.all_rows;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (2 * tid + k < a.experts) {
#pragma unroll
                for (int w = 0; w < kSortWaves; ++w)
                    place[w][2 * tid + k] = place[w][2 * tid + k] + (int32_t)o.rows[k];
            }
    }
    __syncthreads();
    const auto put = [&](int64_t at, int x, int row) {
        if (at >= to) return;
        if constexpr (ALONE) {
            if (x < a.experts) a.row_indices[row] = (int32_t)((uint32_t)at / (uint32_t)a.topk);
            if (a.entry_rows) a.entry_rows[at] = x < a.experts ? row : -1;
        } else {
            a.ranks[at] = row;
        }
    };
    if constexpr (KEEP) {
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            if (from + 64 * k < to) put(from + 64 * k + lane, e[k], place[wave][e[k]] + rank[k]);
    } else {
        for (int64_t i = from; i < to; i += 64) {
            const int x = expert_of(a, i + lane, to);
            put(i + lane, x, step(x));
        }
    }
    if (ALONE)
        for (int64_t i = (int64_t)rows + tid; i < tile_end; i += kSortThreads) a.row_indices[i] = -1;
}

// The tiles' entries to their rows.
__global__ void __launch_bounds__(kSortThreads) group_place_kernel(const GroupArgs a) {
    __shared__ int32_t total[kMoeMaxExperts], base[kMoeMaxExperts];
    __shared__ uint32_t sums[2][kSortWaves];
    const int tid = (int)threadIdx.x;
    for (int x = tid; x < a.experts; x += kSortThreads) total[x] = base[x] = 0;
    __syncthreads();
    // the counts of all tiles, and of those before this one; threads share an expert's tiles
    const int lanes = a.count_lanes, per = kSortThreads / lanes;
    for (int x = tid % lanes; x < a.experts; x += lanes) {
        int32_t all = 0, mine = 0;
        for (int t0 = tid / lanes; t0 < a.tiles; t0 += 16 * per) {
            int32_t c[16];
#pragma unroll
            for (int k = 0; k < 16; ++k)
                c[k] = t0 + k * per < a.tiles ? a.counts[(int64_t)(t0 + k * per) * a.experts + x] : 0;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                all += c[k];
                mine += t0 + k * per < (int)blockIdx.x ? c[k] : 0;
            }
        }
        atomicAdd(&total[x], all);   // whole numbers: in any order
        atomicAdd(&base[x], mine);
    }
    __syncthreads();
    uint32_t n[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) n[k] = 2 * tid + k < a.experts ? (uint32_t)total[2 * tid + k] : 0u;
    const Offsets o = offsets_of(a, n, sums, blockIdx.x == 0);
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (2 * tid + k < a.experts) base[2 * tid + k] += (int32_t)o.rows[k];
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * a.tile, end = min(first + a.tile, a.entries);
    for (int64_t i = first + tid; i < end; i += kSortThreads) {
        const int x = expert_of(a, i, end);
        const int32_t row = x < a.experts ? base[x] + a.ranks[i] : -1;
        if (row >= 0) a.row_indices[row] = (int32_t)((uint32_t)i / (uint32_t)a.topk);
        if (a.entry_rows) a.entry_rows[i] = row;
    }
    for (int64_t i = max(first, (int64_t)o.all_rows) + tid; i < end; i += kSortThreads) a.row_indices[i] = -1;
}

// One workgroup takes so many entries (2048: 8.1 us; 4000 in one 11.4, in tiles 10.7).
constexpr int64_t kAlone = 2048;
// Else tiles of this many at least, and at most that many tiles (32000 entries: 10.8 us, in tiles
// of 2048 12.0, of 4096 16.4; 1048576 of 128 experts, in a graph: 22.8, in 128 tiles 36, in 512
// 26.9).  Every workgroup reads the counts of all tiles and experts, so many experts take fewer:
// tiles * experts counts are kCounts times a tile's entries at most (131072 entries of 1024
// experts: 64 tiles 20.9, 128 26.9, 32 22.0).
constexpr int64_t kTile = 1024, kTiles = 256;
constexpr double kCounts = 32.0;

}  // namespace

void plan_route(RouteArgs& a) {
    a.group_size = a.experts / a.groups;
    a.group_magic = ((1u << 20) + a.group_size - 1) / a.group_size;
    a.group_lanes = 1;
    while (a.group_lanes * 2 * a.groups <= 64) a.group_lanes *= 2;
}

hipError_t launch_route(const RouteArgs& a, bool f32, hipStream_t stream) {
    if (four_a_wave(a)) {
        if (a.experts <= 64) route_many<4>(a, f32, stream);
        else if (a.experts <= 128) route_many<8>(a, f32, stream);
        else route_many<16>(a, f32, stream);
        return hipGetLastError();
    }
    if (a.experts <= 128) route<2>(a, f32, stream);
    else if (a.experts <= 256) route<4>(a, f32, stream);
    else route<kMoeMaxExperts / 64>(a, f32, stream);
    return hipGetLastError();
}

void plan_group(GroupArgs& a) {
    a.bits = 0;
    while ((1 << a.bits) <= a.experts) ++a.bits;
    a.tiles = 1;
    if (a.entries > kAlone)
        a.tiles = (int32_t)std::min({kTiles, (a.entries + kTile - 1) / kTile,
                                     (int64_t)sqrt(kCounts * (double)a.entries / a.experts)});
    const int64_t per = (a.entries + a.tiles - 1) / a.tiles;
    a.tile = (per + kSortThreads - 1) / kSortThreads * kSortThreads;
    a.tiles = a.tile > 0 ? (int32_t)((a.entries + a.tile - 1) / a.tile) : 1;
    a.tiles = std::max(a.tiles, 1);
    a.count_lanes = 64;
    while (a.count_lanes < a.experts && a.count_lanes < kSortThreads) a.count_lanes *= 2;
}

hipError_t launch_group(const GroupArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)a.tiles), block(kSortThreads);
    const bool keep = a.tile <= kKept * kSortThreads;
    if (a.tiles == 1) {
        hipLaunchKernelGGL((group_rank_kernel<true, true>), grid, block, 0, stream, a);
        return hipGetLastError();
    }
    if (keep) hipLaunchKernelGGL((group_rank_kernel<false, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((group_rank_kernel<false, false>), grid, block, 0, stream, a);
    hipLaunchKernelGGL(group_place_kernel, grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace bsq
