// bsq_route.hip -- gfx950 kernels of the routing to experts and of the grouped
// rows that follow from it (include/bsq_decoder.h states the arithmetic).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "bsq_serving_internal.h"

namespace bsq {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr float kLog2e = 1.44269504088896340736f;

// ------------------------------------------------------------ routing
//
// A wave a token, expert e in lane e % 64 of register e / 64.  The topk largest
// are taken one after the other by the wave's largest key, a number's bits in
// an order of unsigned integers (0: not to be chosen).

__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | 1ull << 63;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
// The largest of the wave's numbers, in every lane: rotations within the rows of 16 lanes, then
// across them.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = dpp_max<0x128>(v);
    v = dpp_max<0x124>(v);
    v = dpp_max<0x122>(v);
    v = dpp_max<0x121>(v);
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return __builtin_amdgcn_readfirstlane(max(b[0], b[1]));
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
    const uint32_t hi = wave_max((uint32_t)(v >> 32));
    const uint32_t lo = wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
    return v;
}

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

// The topk largest keys, the lowest expert among equals: lane j gets the j-th's expert.
template <int REGS, class K>
__device__ __forceinline__ int choose(K (&key)[REGS], int topk) {
    const int lane = (int)threadIdx.x & 63;
    int id = 0;
    for (int j = 0; j < topk; ++j) {
        K best = key[0];
#pragma unroll
        for (int k = 1; k < REGS; ++k) best = max(best, key[k]);
        best = wave_max(best);
        bool taken = false;
#pragma unroll
        for (int k = 0; k < REGS; ++k) {
            const uint64_t at = __ballot(key[k] == best);
            if (!taken && at) {
                taken = true;
                const int l = __ffsll((unsigned long long)at) - 1;
                if (lane == j) id = 64 * k + l;
                if (lane == l) key[k] = 0;
            }
        }
    }
    return id;
}

// Closes the groups that are not kept: their experts' keys become 0.  Lane g * P + i looks at
// every P-th expert of group g; `all`: the wave's numbers in LDS.
template <int REGS, class K, class F>
__device__ __forceinline__ void close_groups(const RouteArgs& a, K (&key)[REGS], const F (&c)[REGS], F* all) {
    const int lane = (int)threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < REGS; ++k)
        if (64 * k + lane < a.experts) all[64 * k + lane] = c[k];
    __builtin_amdgcn_wave_barrier();
    const int P = a.group_lanes, g = lane / P, first = g * a.group_size;
    F one = -INFINITY, two = -INFINITY;
    if (g < a.groups)
        for (int e = lane % P; e < a.group_size; e += P) {
            const F v = all[first + e];
            two = v > one ? one : v > two ? v : two;
            one = v > one ? v : one;
        }
    for (int off = P / 2; off >= 1; off >>= 1) {
        const F o1 = __shfl_xor(one, off), o2 = __shfl_xor(two, off);
        two = o1 > one ? (one > o2 ? one : o2) : (two > o1 ? two : o1);
        one = o1 > one ? o1 : one;
    }
    F score = one;
    if (a.group_top == 2 && a.group_size > 1) score = one == -INFINITY || two == -INFINITY ? -INFINITY : one + two;
    // how many groups go before this one
    int before = 0;
    for (int o = 0; o < a.groups; ++o) {
        const F v = __shfl(score, o * P);
        before += v > score || (v == score && o < g) ? 1 : 0;
    }
    const uint64_t kept = __ballot(g < a.groups && lane % P == 0 && before < a.keep);
#pragma unroll
    for (int k = 0; k < REGS; ++k) {
        const int e = 64 * k + lane;
        const int group = (int)(((uint32_t)e * a.group_magic) >> 20);
        if (e < a.experts && !((kept >> (group * P)) & 1)) key[k] = 0;
    }
    __builtin_amdgcn_wave_barrier();
}

// The weights of a token's experts, lane j's being `id`.
template <bool F32, int REGS>
__device__ __forceinline__ float weight_of(const RouteArgs& a, int64_t token, int id, const float (&x)[REGS]) {
    const int lane = (int)threadIdx.x & 63;
    const bool mine = lane < a.topk;
    float z = -INFINITY;
    if (mine && bias_of(a, id) > -INFINITY) z = logit<F32>(a, token, id);
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
        s = share(z, top);
        sum = s;
        if (!a.renormalize) {
            sum = 0.0f;
#pragma unroll
            for (int k = 0; k < REGS; ++k) sum += share(x[k], top);
        }
        sum = wave_sum(sum);
    }
    return sum > 0.0f ? s / sum * a.factor : 0.0f;
}

// The choice by c in 64 bits (of experts by the logits where there is no bias).
template <int REGS>
__device__ __forceinline__ int choose_exactly(const RouteArgs& a, const float (&x)[REGS], double* all) {
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
        const float b = e < a.experts ? bias_of(a, e) : -INFINITY;
        s[k] = !(x[k] > -INFINITY) || b == -INFINITY ? -INFINITY : (a.sigmoid ? s[k] : s[k] / sum) + b;
        key[k] = e < a.experts ? key_of(a.bias ? s[k] : (double)x[k]) : 0;
    }
    if (a.groups > 1) close_groups(a, key, s, all);
    return choose(key, a.topk);
}

// Without a bias, and with groups by their best, c goes by the logit.
template <int REGS>
__device__ __forceinline__ int choose_logits(const RouteArgs& a, const float (&x)[REGS], float* all) {
    const int lane = (int)threadIdx.x & 63;
    uint32_t key[REGS];
#pragma unroll
    for (int k = 0; k < REGS; ++k) key[k] = 64 * k + lane < a.experts ? key_of(x[k]) : 0u;
    if (a.groups > 1) close_groups(a, key, x, all);
    return choose(key, a.topk);
}

template <int REGS, bool F32>
__global__ void __launch_bounds__(kThreads) moe_route_kernel(const RouteArgs a) {
    __shared__ double all[kWaves][REGS * 64];
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t token = (int64_t)blockIdx.x * kWaves + wave;
    if (token >= a.tokens) return;
    float x[REGS];
#pragma unroll
    for (int k = 0; k < REGS; ++k)
        x[k] = 64 * k + lane < a.experts ? logit<F32>(a, token, 64 * k + lane) : -INFINITY;
    const int id = !a.bias && (a.groups == 1 || a.group_top == 1 || a.group_size == 1)
                       ? choose_logits(a, x, reinterpret_cast<float*>(all[wave]))
                       : choose_exactly(a, x, all[wave]);
    const float w = weight_of<F32>(a, token, id, x);
    if (lane < a.topk) {
        a.ids[token * a.topk + lane] = id;
        a.weights[token * a.topk + lane] = w;
    }
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
// atomics takes part.  Few entries are one workgroup's; more are counted by a
// kernel before, a tile a workgroup, whose counts every workgroup then adds up
// for its own place.

constexpr int kSortThreads = 512, kSortWaves = kSortThreads / 64;

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

__global__ void __launch_bounds__(kSortThreads) group_count_kernel(const GroupArgs a) {
    __shared__ int32_t count[kMoeMaxExperts + 1];
    for (int e = (int)threadIdx.x; e <= a.experts; e += kSortThreads) count[e] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * a.tile, end = min(first + a.tile, a.entries);
    for (int64_t i = first + threadIdx.x; i < end; i += kSortThreads)
        atomicAdd(&count[expert_of(a, i, end)], 1);
    __syncthreads();
    for (int e = (int)threadIdx.x; e < a.experts; e += kSortThreads)
        a.counts[(int64_t)blockIdx.x * a.experts + e] = count[e];
}

template <bool ALONE>
__global__ void __launch_bounds__(kSortThreads) group_rows_kernel(const GroupArgs a) {
    // per wave and expert: its entries, then where its next one goes
    __shared__ volatile int32_t place[kSortWaves][kMoeMaxExperts + 1];
    __shared__ int32_t total[kMoeMaxExperts], before[kMoeMaxExperts];
    __shared__ uint32_t sums[2][kSortWaves];
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t first = (int64_t)blockIdx.x * a.tile, tile_end = min(first + a.tile, a.entries);
    const int64_t part = a.tile / kSortWaves;
    const int64_t from = first + wave * part, to = min(from + part, tile_end);
    const uint64_t below = (1ull << lane) - 1;

    for (int e = lane; e <= a.experts; e += 64) place[wave][e] = 0;
    __builtin_amdgcn_wave_barrier();
    for (int64_t i = from; i < to; i += 64) {
        const int e = expert_of(a, i + lane, to);
        const uint64_t m = same_lanes(e, a.bits);
        if (!(m & below)) place[wave][e] = place[wave][e] + __popcll(m);
        __builtin_amdgcn_wave_barrier();
    }
    if (!ALONE) {
        // the counts of all tiles, and of those before this one; threads share an expert's tiles
        for (int e = tid; e < a.experts; e += kSortThreads) total[e] = before[e] = 0;
        __syncthreads();
        const int lanes = a.count_lanes, per = kSortThreads / lanes;
        for (int e = tid % lanes; e < a.experts; e += lanes) {
            int32_t all = 0, mine = 0;
            for (int t = tid / lanes; t < a.tiles; t += per) {
                const int32_t n = a.counts[(int64_t)t * a.experts + e];
                all += n;
                if (t < (int)blockIdx.x) mine += n;
            }
            atomicAdd(&total[e], all);
            atomicAdd(&before[e], mine);
        }
    }
    __syncthreads();
    // thread t: experts 2 t and 2 t + 1; their totals, the waves' places within the group
    uint32_t n[2] = {0, 0}, padded[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int e = 2 * tid + k;
        if (e >= a.experts) continue;
        int32_t run = ALONE ? 0 : before[e];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const int32_t c = place[w][e];
            place[w][e] = run;
            run += c;
        }
        n[k] = (uint32_t)(ALONE ? run : total[e]);
        padded[k] = (n[k] + a.pad - 1) / a.pad * a.pad;
    }
    // exclusive sums over the experts
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
    uint32_t rows = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        if (w < wave) {
            r += sums[0][w];
            s += sums[1][w];
        }
        rows += sums[0][w];
    }
    r -= n[0] + n[1];
    s -= padded[0] + padded[1];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int e = 2 * tid + k;
        if (e < a.experts) {
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) place[w][e] = place[w][e] + (int32_t)r;
        }
        if (e <= a.experts && blockIdx.x == 0) {
            a.row_offsets[e] = r;
            a.scales_offsets[e] = s;
        }
        r += n[k];
        s += padded[k];
    }
    // 1024 experts: the last offset is no thread's expert
    if (blockIdx.x == 0 && tid == kSortThreads - 1 && a.experts == 2 * kSortThreads) {
        a.row_offsets[a.experts] = r;
        a.scales_offsets[a.experts] = s;
    }
    __syncthreads();
    for (int64_t i = from; i < to; i += 64) {
        const int64_t at = i + lane;
        const int e = expert_of(a, at, to);
        const uint64_t m = same_lanes(e, a.bits);
        const int32_t row = place[wave][e] + __popcll(m & below);
        __builtin_amdgcn_wave_barrier();
        if (!(m & below)) place[wave][e] = place[wave][e] + __popcll(m);
        __builtin_amdgcn_wave_barrier();
        if (at < to) {
            if (e < a.experts) a.row_indices[row] = (int32_t)((uint32_t)at / (uint32_t)a.topk);
            if (a.entry_rows) a.entry_rows[at] = e < a.experts ? row : -1;
        }
    }
    for (int64_t i = max(first, (int64_t)rows) + tid; i < tile_end; i += kSortThreads) a.row_indices[i] = -1;
}

// One workgroup takes so many entries.
constexpr int64_t kAlone = 4096;
// Else tiles of this many at least, and at most that many tiles.
constexpr int64_t kTile = 2048, kTiles = 128;

}  // namespace

void plan_route(RouteArgs& a) {
    a.group_size = a.experts / a.groups;
    a.group_magic = ((1u << 20) + a.group_size - 1) / a.group_size;
    a.group_lanes = 1;
    while (a.group_lanes * 2 * a.groups <= 64) a.group_lanes *= 2;
}

hipError_t launch_route(const RouteArgs& a, bool f32, hipStream_t stream) {
    if (a.experts <= 128) route<2>(a, f32, stream);
    else if (a.experts <= 256) route<4>(a, f32, stream);
    else route<kMoeMaxExperts / 64>(a, f32, stream);
    return hipGetLastError();
}

void plan_group(GroupArgs& a) {
    a.bits = 0;
    while ((1 << a.bits) <= a.experts) ++a.bits;
    a.tiles = 1;
    if (a.entries > kAlone) a.tiles = (int32_t)std::min(kTiles, (a.entries + kTile - 1) / kTile);
    const int64_t per = (a.entries + a.tiles - 1) / a.tiles;
    a.tile = (per + kSortThreads - 1) / kSortThreads * kSortThreads;
    a.tiles = a.tile > 0 ? (int32_t)((a.entries + a.tile - 1) / a.tile) : 1;
    a.tiles = std::max(a.tiles, 1);
    a.count_lanes = 64;
    while (a.count_lanes < a.experts && a.count_lanes < kSortThreads) a.count_lanes *= 2;
}

hipError_t launch_group(const GroupArgs& a, hipStream_t stream) {
    if (a.tiles == 1) {
        hipLaunchKernelGGL((group_rows_kernel<true>), dim3(1), dim3(kSortThreads), 0, stream, a);
    } else {
        hipLaunchKernelGGL(group_count_kernel, dim3((uint32_t)a.tiles), dim3(kSortThreads), 0, stream, a);
        hipLaunchKernelGGL((group_rows_kernel<false>), dim3((uint32_t)a.tiles), dim3(kSortThreads), 0,
                           stream, a);
    }
    return hipGetLastError();
}

}  // namespace bsq
