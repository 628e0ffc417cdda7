// bsq_rope.hip -- gfx950 kernel of the norms and the rotation of queries and
// keys (include/bsq_decoder.h states the arithmetic).
//
// A lane holds 8 consecutive elements of a head, L lanes a head, so every load
// and store is whole 16-byte pieces and a wave's are consecutive.  The angles of
// a row are the same for all of its heads: a wave finds their cosines and sines
// once, a lane each, and takes several heads with them, one step (64 / L heads)
// after the other, the next step's elements being on their way.  The norm is a
// sum over the L lanes; with halves a pair's other element is 8 elements of
// another lane (rotary_dim being a multiple of 16), with neighbours it is the
// lane's own.  Bound by the bytes: 16384 rows of 32 + 8 heads of 128 in BF16, 336
// MB read and written, take 75 us a call (4.5 TB/s; a copy reaches 5.2).  With
// the angles found by every lane for its own elements and lanes exchanged
// through LDS it took 85.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "bsq_serving_internal.h"

namespace bsq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = 4;

// Sine and cosine of t turns (t in 64 bits, any size).  t less its nearest quarter
// is exact; the rest, at most an eighth of a turn, goes through the Taylor series
// in 32 bits: x^11 / 11! and x^12 / 12! at pi / 4 are below 2^-28.
__device__ __forceinline__ void sincos_turns(double t, float& s, float& c) {
    const double f = t - __builtin_rint(t);              // [-1/2, 1/2]
    const double n = __builtin_rint(4.0 * f);
    const float x = (float)((f - 0.25 * n) * 6.283185307179586476925);
    const float z = x * x;
    float p = __builtin_fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
    p = __builtin_fmaf(z, p, 8.3333333e-3f);
    p = __builtin_fmaf(z, p, -1.6666667e-1f);
    const float sx = __builtin_fmaf(x * z, p, x);
    float q = __builtin_fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
    q = __builtin_fmaf(z, q, -1.3888889e-3f);
    q = __builtin_fmaf(z, q, 4.1666667e-2f);
    q = __builtin_fmaf(z, q, -0.5f);
    const float cx = __builtin_fmaf(z, q, 1.0f);
    const int k = (int)n & 3;                            // a NaN's is of no account
    const float a = k & 1 ? cx : sx, b = k & 1 ? sx : cx;
    s = k & 2 ? -a : a;
    c = k == 1 || k == 2 ? -b : b;
}

// The instruction takes no subnormal numbers.
__device__ __forceinline__ float inv_sqrt(float v) {
    const bool tiny = v < 0x1p-100f;
    return __builtin_amdgcn_rsqf(tiny ? v * 0x1p60f : v) * (tiny ? 0x1p30f : 1.0f);
}

template <int CTRL>
__device__ __forceinline__ float moved(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
// The number of lane ^ 16.
__device__ __forceinline__ float across_rows(float v) {
    const uint32_t b = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    return __uint_as_float(threadIdx.x & 16 ? a[0] : a[1]);
}
// The sum over the L lanes of a head, in each of them: lanes ^ 1, ^ 2, mirrors of 8 and of 16.
template <int L>
__device__ __forceinline__ float head_sum(float v) {
    v += moved<0xB1>(v);
    v += moved<0x4E>(v);
    v += moved<0x141>(v);
    if constexpr (L >= 16) v += moved<0x140>(v);
    if constexpr (L == 32) v += across_rows(v);
    return v;
}
// The number of lane ^ L / 2.
template <int L>
__device__ __forceinline__ float of_other_half(float v) {
    if constexpr (L == 8) return moved<0x1B>(moved<0x141>(v));
    else if constexpr (L == 16) return moved<0x128>(v);
    else return across_rows(v);
}

template <bool F32>
struct Piece {
    u32x4 w[F32 ? 2 : 1];            // 8 elements
};
template <bool F32, bool ONCE>
__device__ __forceinline__ Piece<F32> load_piece(const void* x, int64_t at) {
    Piece<F32> p;
    const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const char*>(x) + at * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) p.w[i] = ONCE ? __builtin_nontemporal_load(s + i) : s[i];
    return p;
}
template <bool F32>
__device__ __forceinline__ void unpack(const Piece<F32>& p, float (&y)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (F32) y[e] = __uint_as_float(p.w[e / 4][e % 4]);
        else y[e] = __uint_as_float(e % 2 ? p.w[0][e / 2] & 0xFFFF0000u : p.w[0][e / 2] << 16);
    }
}

// How pairs lie: anywhere in two halves, in the two halves of all L lanes, or beside each other.
enum Pairs { kHalves, kWhole, kNeighbours };

template <int L, bool F32, Pairs PAIRS, bool ONCE>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int H = 64 / L;                            // heads of a step
    const int lane = (int)threadIdx.x & 63, l = lane % L, sub = lane / L;
    const int64_t wave = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t row = wave / a.parts;
    if (row >= a.num_rows) return;
    const int first = (int)(wave % a.parts) * a.steps, end = min(first + a.steps, a.all_steps);
    const int d = 8 * l;
    const bool on = d < a.head_dim;

    // step -> segment (q, k or v) and its first head
    auto place = [&](int step, int& seg, int& head) {
        seg = step < a.seg_steps[0] ? 0 : step < a.seg_steps[0] + a.seg_steps[1] ? 1 : 2;
        if (seg > 0) step -= a.seg_steps[0];
        if (seg > 1) step -= a.seg_steps[1];
        head = step * H + sub;
    };
    auto fetch = [&](int step) {
        int seg, head;
        place(step, seg, head);
        Piece<F32> p{};
        if (on && head < a.heads[seg])
            p = load_piece<F32, ONCE>(a.x[seg], row * a.ldx[seg] + (int64_t)head * a.head_dim + d);
        return p;
    };
    // Each lane finds one angle of the row (or two), and takes those of its elements from the
    // others; the first of a pair takes the sine off.
    constexpr int N = PAIRS == kNeighbours ? 4 : 8;
    __shared__ f32x4 turns[kWaves][2][32];
    float cs[N], sn[N];
    const bool turned = d < a.rotary_dim;
    const int half = a.rotary_dim / 2;
    const bool low = d < half;
    const Piece<F32> early = fetch(first);
    if (half > 0) {
        const double pos = (double)a.positions[row] * 0.15915494309189533576888;   // 1 / (2 pi)
        float* all = reinterpret_cast<float*>(turns[threadIdx.x >> 6]);
        for (int i = lane; i < half; i += 64) sincos_turns(pos * a.inv_freq[i], all[i], all[128 + i]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (turned) {
            const int i = PAIRS == kNeighbours ? d / 2 : low ? d : d - half;   // a multiple of 4
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float s = turns[threadIdx.x >> 6][0][i / 4 + e / 4][e % 4];
                sn[e] = PAIRS != kNeighbours && low ? -s : s;
                cs[e] = turns[threadIdx.x >> 6][1][i / 4 + e / 4][e % 4];
            }
        }
    }
    const int other = PAIRS != kHalves || !turned ? lane : low ? lane + half / 8 : lane - half / 8;

    float w[8];
    int weights_of = -1;
    Piece<F32> next = early;
    for (int step = first; step < end; ++step) {
        int seg, head;
        place(step, seg, head);
        const Piece<F32> now = next;
        if (step + 1 < end) next = fetch(step + 1);
        float y[8];
        unpack<F32>(now, y);
        const float* weight = seg < 2 ? a.weight[seg] : nullptr;
        if (weight) {
            if (seg != weights_of) {
                weights_of = seg;
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = on ? weight[d + e] : 0.0f;
            }
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(y[e], y[e], sum);
            const float inv = inv_sqrt(__builtin_fmaf(head_sum<L>(sum), a.inv_dim, a.eps));
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = y[e] * inv * w[e];
        }
        if (seg < 2 && a.rotary_dim > 0) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (PAIRS == kWhole) {
                    o[e] = __builtin_fmaf(y[e], cs[e], of_other_half<L>(y[e]) * sn[e]);
                } else if constexpr (PAIRS == kNeighbours) {
                    const float t = e % 2 ? sn[e / 2] : -sn[e / 2];
                    o[e] = __builtin_fmaf(y[e], cs[e / 2], y[e ^ 1] * t);
                } else {
                    o[e] = __builtin_fmaf(y[e], cs[e], __shfl(y[e], other) * sn[e]);
                }
            }
            if (turned) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = o[e];
            }
        }
        if (on && head < a.heads[seg]) {
            u32x4 r;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bf16x2 b = {(__bf16)y[2 * e], (__bf16)y[2 * e + 1]};
                r[e] = __builtin_bit_cast(uint32_t, b);
            }
            *reinterpret_cast<u32x4*>(a.out[seg] + row * a.ldo[seg] + (int64_t)head * a.head_dim + d) = r;
        }
    }
}

// Steps of a wave: all of a row's where that gives waves enough for the CUs, else fewer, down to one
// (16384 rows of 40 heads: 76 us with 10 steps a wave, 79 with five).
constexpr int64_t kWavesWanted = 4096;
// Calls whose inputs and outputs together are larger than the memory-side cache read the inputs past
// the caches.  Rows just written, past the caches and through them: BF16, 130 MB of input 56 us and
// 55, 160 MB 66 and 68, 220 MB 88 and 105; FP32, whose outputs are half as large, 60 MB 27 and 22,
// 200 MB 77 and 57, 260 MB 89 and 90, 300 MB 98 and 117.  Rows that no longer lie there are read past
// them the faster at any size (BF16, 160 MB: 74 and 95; FP32, 200 MB: 69 and 98), so the rule of one
// size for both types loses in FP32 from 180 to 260 MB what it gains for such rows.
constexpr int64_t kCached = 256 << 20;

template <int L, bool F32, Pairs PAIRS>
void rope(const RopeArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)((a.num_rows * a.parts + kWaves - 1) / kWaves));
    if (a.once)
        hipLaunchKernelGGL((qk_norm_rope_kernel<L, F32, PAIRS, true>), grid, dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((qk_norm_rope_kernel<L, F32, PAIRS, false>), grid, dim3(kThreads), 0, stream, a);
}
template <int L, bool F32>
void rope_of(const RopeArgs& a, bool pairs, hipStream_t stream) {
    if (pairs) rope<L, F32, kNeighbours>(a, stream);
    else if (a.rotary_dim == 8 * L) rope<L, F32, kWhole>(a, stream);
    else rope<L, F32, kHalves>(a, stream);
}
template <int L>
void rope_of(const RopeArgs& a, bool f32, bool pairs, hipStream_t stream) {
    f32 ? rope_of<L, true>(a, pairs, stream) : rope_of<L, false>(a, pairs, stream);
}

int lanes_of(int head_dim) { return head_dim <= 64 ? 8 : head_dim <= 128 ? 16 : 32; }

}  // namespace

void plan_rope(RopeArgs& a, bool f32) {
    const int heads = 64 / lanes_of(a.head_dim);
    a.all_steps = 0;
    for (int s = 0; s < 3; ++s) {
        a.seg_steps[s] = (a.heads[s] + heads - 1) / heads;
        a.all_steps += a.seg_steps[s];
    }
    const int64_t all = a.num_rows * a.all_steps;
    a.steps = (int32_t)std::min<int64_t>(std::max<int64_t>(all / kWavesWanted, 1), a.all_steps);
    a.parts = (a.all_steps + a.steps - 1) / a.steps;
    const int64_t width = (int64_t)(a.heads[0] + a.heads[1] + a.heads[2]) * a.head_dim;
    a.once = (double)a.num_rows * width * (f32 ? 6 : 4) > (double)kCached;
}

hipError_t launch_rope(const RopeArgs& a, bool f32, bool pairs, hipStream_t stream) {
    switch (lanes_of(a.head_dim)) {
        case 8: rope_of<8>(a, f32, pairs, stream); break;
        case 16: rope_of<16>(a, f32, pairs, stream); break;
        default: rope_of<32>(a, f32, pairs, stream); break;
    }
    return hipGetLastError();
}

}  // namespace bsq
