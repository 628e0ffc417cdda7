// bsq_kv.hip -- gfx950 kernels of the paged 8-bit key/value cache: writing
// tokens into it, attention over it.  include/bsq_serving.h states the
// layouts and the arithmetic.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "bsq_serving_internal.h"

namespace bsq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256, kWaves = 4;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// Sequence s of a call: rows [lo, lo + n), L tokens in all.  n = 0 when its
// offsets or its length make no sense.
struct Seq {
    int64_t lo;
    int32_t n, L;
};
__device__ __forceinline__ Seq load_seq(const KvSeqs& q, int s) {
    const int64_t lo = q.row_offsets[s], hi = q.row_offsets[s + 1];
    const int32_t L = q.kv_lens[s];
    Seq r{lo, 0, L};
    if (lo < hi && hi <= q.num_rows && hi - lo <= 0x7FFFFFFF && L >= 0) r.n = (int32_t)(hi - lo);
    return r;
}

// The i-th longest of up to 64 sequences, the lower number among equals.
__device__ __forceinline__ int longest(const KvSeqs& q, int i) {
    const int lane = (int)threadIdx.x & 63;
    const int32_t L = lane < q.num_seqs ? q.kv_lens[lane] : 0;
    int before = 0;
    for (int o = 0; o < q.num_seqs; ++o) {
        const int32_t other = __builtin_amdgcn_readlane(L, o);
        before += other > L || (other == L && o < lane) ? 1 : 0;
    }
    const uint64_t at = __ballot(before == i && lane < q.num_seqs);
    return __ffsll((unsigned long long)at) - 1;
}

// ------------------------------------------------------------ append
//
// One workgroup per (page touched, head, K or V).  It reads its new tokens
// once, held in registers, takes their largest magnitude, and writes their
// codes; the codes already in the page are read only when the scale grew.
// Work items are 4 tokens x 4 elements: the four tokens 4 m .. 4 m + 3 of one
// element are one dword of V, and four elements of one token one dword of K,
// so the same item serves both layouts and every store but those of a partial
// group of tokens is a dword.  A page that is filled whole goes through LDS and
// leaves in 16-byte stores (from the items' dwords, V's each in a line of its
// own, 16384 tokens of 8 heads of 128 took 19.7 us, this way 15.9: 4.2 TB/s).  A
// few tokens a sequence (decode) take one wave and no barrier.

// Four E4M3 codes times a power of two, rounded to E4M3 again.
__device__ __forceinline__ uint32_t rescale_codes(uint32_t v, float f) {
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(v, 1.0f, false);
    const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(v, 1.0f, true);
    i16x2 r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a[0] * f, a[1] * f, 1.0f, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, b[0] * f, b[1] * f, 1.0f, true);
    return __builtin_bit_cast(uint32_t, r);
}

// QUADS: groups of 4 tokens that a page's new tokens touch, at most
template <int D, int THREADS, int QUADS>
__global__ void __launch_bounds__(THREADS) kv_append_kernel(const AppendArgs a) {
    constexpr int kPieces = D / 4;                 // 4-element pieces of a token
    constexpr int kItems = (QUADS * kPieces + THREADS - 1) / THREADS;
    const int s = (int)(blockIdx.x / (uint32_t)a.pages_per_seq);
    const int pi = (int)(blockIdx.x % (uint32_t)a.pages_per_seq);
    const int head = (int)blockIdx.y, is_v = (int)blockIdx.z, tid = (int)threadIdx.x;
    const Seq sq = load_seq(a.seqs, s);
    const int64_t old = (int64_t)sq.L - sq.n;      // tokens held before
    if (sq.n == 0 || old < 0) return;
    const int64_t page_i = old / kKvPage + pi;
    const int64_t base = page_i * kKvPage;
    const int64_t end = min((int64_t)sq.L, old + a.max_new);   // of the rows that are written
    if (base >= end || page_i >= a.seqs.max_pages) return;
    const int t0 = (int)(base < old ? old - base : 0);                   // first new token
    const int t1 = (int)(end - base < kKvPage ? end - base : kKvPage);   // end of them
    const int32_t page = a.seqs.table[(int64_t)s * a.seqs.table_stride + page_i];
    const int64_t ldx = a.ldx[is_v];
    const uint16_t* x = a.x[is_v] + (sq.lo + (base - old)) * ldx + (int64_t)head * D;

    // item w: tokens 4 (t0 / 4 + w / kPieces) .., elements 4 (w % kPieces) ..
    const int q0 = t0 / 4;
    u32x2 v[kItems][4];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int w = tid + k * THREADS;
        const int tq = 4 * (q0 + w / kPieces), d = 4 * (w % kPieces);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = tq + e;
            v[k][e] = (u32x2){0u, 0u};
            if (t >= t0 && t < t1) v[k][e] = *reinterpret_cast<const u32x2*>(x + t * ldx + d);
        }
    }
    if (page < 0 || page >= a.cache.num_pages) return;
    uint8_t* codes = (is_v ? a.cache.v_codes : a.cache.k_codes) +
                     (int64_t)page * a.cache.page_stride + (int64_t)head * D * kKvPage;
    uint8_t* scale = (is_v ? a.cache.v_scales : a.cache.k_scales) +
                     (int64_t)page * a.cache.scale_stride + head;
    const uint32_t was = t0 > 0 ? *scale : 0u;
    uint32_t amax = 0;
#pragma unroll
    for (int k = 0; k < kItems; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint32_t m = v[k][e][c] & 0x7FFF7FFFu;
                amax = max(amax, max(m & 0xFFFFu, m >> 16));
            }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, off));
    if constexpr (THREADS > 64) {
        __shared__ uint32_t red[THREADS / 64];
        if ((tid & 63) == 0) red[tid >> 6] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) amax = max(amax, red[w]);
    }

    const bool nan = amax >= 0x7F80u || was == 255u;
    uint32_t byte = (uint32_t)max((int)(amax >> 7) - 8, 0);
    byte = nan ? 255u : max(byte, was);
    // 2^X for the conversion: the instruction reads the exponent field alone
    const float sc = __uint_as_float((nan ? 127u : byte) << 23);
    // 448 * 2^X as a BF16 pattern: larger magnitudes saturate to it
    const uint32_t cap = (byte << 7) + 0x460u;
    const u16x2 cap2 = __builtin_bit_cast(u16x2, cap | (cap << 16));
    // The page's codes in LDS.  K's 16-byte piece of chunk c and token t at token t ^ (c % 8),
    // V's rows 17 dwords apart: the items of a wave then write to different banks.
    constexpr bool kWhole = QUADS == kKvPage / 4;
    __shared__ __attribute__((aligned(16))) uint32_t image[kWhole ? D * 17 : 1];
    const bool whole = kWhole && t0 == 0 && t1 == kKvPage;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int w = tid + k * THREADS;
        const int tq = 4 * (q0 + w / kPieces), d = 4 * (w % kPieces);
        if (tq >= t1) break;
        uint32_t c[4];                             // 4 codes of token tq + e
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bf16x2 p[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t word = v[k][e][h];
                const u16x2 m = __builtin_elementwise_min(
                    __builtin_bit_cast(u16x2, word & 0x7FFF7FFFu), cap2);
                p[h] = __builtin_bit_cast(bf16x2, __builtin_bit_cast(uint32_t, m) |
                                                      (word & 0x80008000u));
            }
            i16x2 r = {0, 0};
            r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, p[0], sc, false);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, p[1], sc, true);
            c[e] = nan ? 0u : __builtin_bit_cast(uint32_t, r);
        }
        if (!is_v) {
            if (whole) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    image[(d / 16 * kKvPage + ((tq + e) ^ (d / 16 % 8))) * 4 + d % 16 / 4] = c[e];
                continue;
            }
            uint8_t* o = codes + (d / 16) * (16 * kKvPage) + d % 16;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (tq + e >= t0 && tq + e < t1)
                    *reinterpret_cast<uint32_t*>(o + (tq + e) * 16) = c[e];
        } else {
            // tokens 16 j + 4 g + e at 16 g + 4 j + e
            uint8_t* o = codes + d * kKvPage + 16 * (tq / 4 % 4) + 4 * (tq / 16);
#pragma unroll
            for (int b = 0; b < 4; ++b) {          // element d + b, tokens tq .. tq + 3
                const uint32_t word = ((c[0] >> (8 * b)) & 0xFFu) |
                                      (((c[1] >> (8 * b)) & 0xFFu) << 8) |
                                      (((c[2] >> (8 * b)) & 0xFFu) << 16) |
                                      (((c[3] >> (8 * b)) & 0xFFu) << 24);
                if (whole) {
                    image[(d + b) * 17 + 4 * (tq / 4 % 4) + tq / 16] = word;
                } else if (tq >= t0 && tq + 4 <= t1) {
                    *reinterpret_cast<uint32_t*>(o + b * kKvPage) = word;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (tq + e >= t0 && tq + e < t1)
                            o[b * kKvPage + e] = (uint8_t)(word >> (8 * e));
                }
            }
        }
    }
    if (whole) {
        __syncthreads();
        for (int y = tid; y < D * kKvPage / 16; y += THREADS) {
            u32x4 o;
            if (!is_v) {
                const int c = y / kKvPage, t = y % kKvPage;
                o = *reinterpret_cast<const u32x4*>(&image[(c * kKvPage + (t ^ (c % 8))) * 4]);
            } else {
                const uint32_t* r = &image[y / 4 * 17 + y % 4 * 4];
                o = (u32x4){r[0], r[1], r[2], r[3]};
            }
            *reinterpret_cast<u32x4*>(codes + 16 * y) = o;
        }
    }
    // The tokens that were there, on the grown scale, a dword at a time: four elements of a
    // token of K, four tokens of an element of V.  Of V's group that the new tokens share,
    // only the old tokens' bytes are written.
    if (t0 > 0 && byte != was) {
        const float f = nan ? 0.0f : __builtin_ldexpf(1.0f, (int)was - (int)byte);
        if (!is_v) {
#pragma unroll 4
            for (int w = tid; w < t0 * kPieces; w += THREADS) {
                const int t = w / kPieces, d = 4 * (w % kPieces);
                uint32_t* o = reinterpret_cast<uint32_t*>(codes + (d / 16) * (16 * kKvPage) + t * 16 +
                                                          d % 16);
                *o = nan ? 0u : rescale_codes(*o, f);
            }
        } else {
#pragma unroll 4
            for (int w = tid; w < t0 / 4 * D; w += THREADS) {
                const int q = w / D, d = w % D;
                uint32_t* o = reinterpret_cast<uint32_t*>(codes + d * kKvPage + 16 * (q % 4) + 4 * (q / 4));
                *o = nan ? 0u : rescale_codes(*o, f);
            }
            const int left = t0 % 4, q = t0 / 4;
            for (int w = tid; w < left * D; w += THREADS) {
                const int e = w / D, d = w % D;
                uint8_t* o = codes + d * kKvPage + 16 * (q % 4) + 4 * (q / 4) + e;
                *o = nan ? 0 : (uint8_t)rescale_codes(*o, f);
            }
        }
    }
    // `was` was read by every thread before the barrier above
    if (tid == 0) *scale = (uint8_t)byte;
}

// ------------------------------------------------------------ attention
//
// The products run transposed, so that nothing moves between lanes:
//   S^T (tokens x columns) = K Q^T    mfma_f32_16x16x32_bf16, four 16-token tiles a page
//   O^T (head_dim x columns) += V^T P^T   mfma_f32_16x16x32_f16
// A column is a (query row, head of the group) pair.  Lane l serves column
// l % 16 and group g = l / 16; its scores are the tokens 16 j + 4 g + e
// (j the tile, e the register), which are the 16 bytes of V that the lane
// loads for an element: its weights are the B operand of the second product
// as they stand.  K's 16-byte pieces hold 16 elements of a token: two steps
// of the contraction, whose order q shares.

// 8 E4M3 codes as BF16, and times a power of two as FP16.
__device__ __forceinline__ bf16x8 to_bf16(uint32_t a, uint32_t b) {
    const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    return (bf16x8){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}
__device__ __forceinline__ f16x8 to_f16(uint32_t a, uint32_t b, float scale) {
    const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, scale, false);
    const f16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, scale, true);
    const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, scale, false);
    const f16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, scale, true);
    return (f16x8){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// The largest, and the sum, over the four lanes that share a column.
__device__ __forceinline__ float group_max(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

__device__ __forceinline__ float group_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// The running state of 16 CB columns.  Scores are in units of log 2; m is a
// column's reference score, weights are 2^(score - m + kShift) and l and acc
// (the lane's part of O^T, in units of 2^unit) their sums.  m follows the
// largest score only when that passes it by kSlack: most pages then neither
// rescale acc nor exchange their maxima between lanes.  Weights stay below
// 2^(kShift + kSlack) = 2^15 and are normal FP16 numbers down to 2^-25 of m's.
constexpr float kShift = 11.0f, kSlack = 4.0f;
template <int D, int CB>
struct AttState {
    f32x4 acc[CB][D / 16];
    float m[CB], l[CB];              // l: the lane's share
    int unit;                        // the unit of acc
};

template <int D, int CB>
__device__ __forceinline__ void init_state(AttState<D, CB>& st) {
#pragma unroll
    for (int c = 0; c < CB; ++c) {
        st.m[c] = -INFINITY;
        st.l[c] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.acc[c][i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    }
    st.unit = -1000;
}

// What a wave needs of its columns to mask: each lane's column sees tokens
// [first, last].  MASKED (kv_cache_attention_masked): the tokens [0, sinks) too, and of the
// tokens from `base` on (a tree's rows) those whose bits are set.
template <int CB, bool MASKED>
struct Columns {
    int first[CB], last[CB];         // per lane
    int all_from, all_to;            // tokens that every column of the wave sees
};
template <int CB>
struct Columns<CB, true> {
    int first[CB], last[CB];
    int all_from, all_to;
    const uint64_t* mask[CB];        // per lane; null: no tree
    int words, base, end, sinks;     // end: the sequence's length

    // The lowest k bits.
    static __device__ __forceinline__ uint64_t low(int k) {
        return k <= 0 ? 0 : k >= 64 ? ~0ull : (1ull << k) - 1;
    }
    // Which tokens of the page that starts at token t column cb sees.
    __device__ __forceinline__ uint64_t page(int cb, int t) const {
        const uint64_t near = ~low(first[cb] - t) | low(min(sinks, end) - t);
        if (!mask[cb]) return near & low(last[cb] + 1 - t);
        uint64_t seen = near & low(base - t);
        if (t + kKvPage > base) {
            const int x = t - base, i = x >> 6, s = x & 63;   // x < 0: i is -1
            uint64_t bits = 0;
            if (i >= 0 && i < words) bits = mask[cb][i] >> s;
            if (s && i + 1 < words) bits |= mask[cb][i + 1] << (64 - s);
            seen |= bits & low(end - t) & ~low(base - t);
        }
        return seen;
    }
};
// The lane's 16 of a page's tokens: bit k is token 16 (k / 4) + 4 g + k % 4.
__device__ __forceinline__ uint32_t lane_bits(uint64_t page, int g) {
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) r |= ((uint32_t)(page >> (16 * j + 4 * g)) & 15u) << (4 * j);
    return r;
}

// 2^n for the n of units and scales; below the normal numbers 0.
__device__ __forceinline__ float power_of_two(int n) {
    return n < -126 ? 0.0f : __uint_as_float((uint32_t)(min(n, 127) + 127) << 23);
}
// V's scale goes into its conversion to FP16, relative to acc's unit: exact
// within [-15, 7] of it.  Past that the unit moves, but stays within 2^60 of the
// largest scale so far: acc, at most 2^9 2^15 2^60 a token, then cannot overflow.
// A page with the NaN scale leaves the unit and enters in it, beside weights that
// are NaN where a row sees it and 0 where none does.
struct Unit {
    int unit = -1000, top = -1000;   // of acc; the largest scale so far (never below the unit)
    // The factor of V's conversion.
    __device__ __forceinline__ float follow(uint32_t vs) {
        const int e = vs == 255u ? unit : (int)vs - 127;
        top = max(top, e);
        if (e > unit + 7 || e < unit - 15) unit = max(e, top - 60);
        return power_of_two(e - unit);
    }
};
// Of the dword of V that holds tokens t .. t + 3, the bytes before the
// sequence's end: those past it may hold anything.
__device__ __forceinline__ uint32_t before_end(int t, int L) {
    const int left = L - t;
    return left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
}

template <int D, int CB>
__device__ __forceinline__ void move_unit(AttState<D, CB>& st, int unit) {
    const float step = power_of_two(st.unit - unit);
    st.unit = unit;
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.acc[cb][i] *= step;
}

// One page.  kf(j, k): the lane's 8 elements of K of token tile j and step k of
// the contraction; vf(i, u): its 8 tokens of V of 16-element tile i and step u,
// in units of 2^st.unit.
template <int D, int CB, bool MASKED, bool LDS, class KF, class VF>
__device__ __forceinline__ void attend_page(AttState<D, CB>& st, const Columns<CB, MASKED>& cols,
                                            const bf16x8 (&q)[CB][D / 32], KF kf, VF vf, uint32_t ks,
                                            uint32_t vs, int base, float c0) {
    constexpr int VI = D / 16;
    const int g = (int)(threadIdx.x & 63) >> 4;
    f32x4 s[CB][4];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[cb][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < D / 32; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf16x8 a = kf(j, k);
#pragma unroll
            for (int cb = 0; cb < CB; ++cb)
                s[cb][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, q[cb][k], s[cb][j], 0, 0, 0);
        }
    if constexpr (CB > 1 && LDS) {
        // K comes from LDS: six reads ahead of the products, not two (2% of a prompt)
        __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
        for (int x = 0; x < D / 8 - 6; ++x) {
            __builtin_amdgcn_sched_group_barrier(0x008, CB, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, CB * 6, 0);
    }
    // to units of log 2; a NaN scale of K or V makes NaN of every weight it meets
    float c = c0 * __builtin_ldexpf(1.0f, (int)ks - 127);
    if (ks == 255u || vs == 255u) c = NAN;
    const bool masked = base < cols.all_from || base + kKvPage - 1 > cols.all_to;
    // bit k: the column sees the lane's token k (16 (k / 4) + 4 g + k % 4)
    uint32_t seen[CB];
    float top[CB];
    if (masked) {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
            seen[cb] = 0;
            top[cb] = -INFINITY;
            if constexpr (MASKED) seen[cb] = lane_bits(cols.page(cb, base), g);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                bool in;
                if constexpr (MASKED) {
                    in = (seen[cb] >> k) & 1u;
                } else {
                    const int t = base + 16 * (k / 4) + 4 * g + k % 4;
                    in = t >= cols.first[cb] && t <= cols.last[cb];
                    seen[cb] |= in ? 1u << k : 0u;
                }
                top[cb] = fmaxf(top[cb], in ? s[cb][k / 4][k % 4] : -INFINITY);
            }
        }
    } else {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
            top[cb] = s[cb][0][0];
#pragma unroll
            for (int k = 1; k < 16; ++k) top[cb] = fmaxf(top[cb], s[cb][k / 4][k % 4]);
        }
    }
    bool passed = false;
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) passed |= top[cb] * c > st.m[cb] + kSlack;
    if (__any(passed)) {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
            // no score seen so far: alpha is 0 or, with none in this page either, 1
            const float m = fmaxf(st.m[cb], group_max(top[cb]) * c);
            const float alpha = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m[cb] - m);
            st.m[cb] = m;
            st.l[cb] *= alpha;
#pragma unroll
            for (int i = 0; i < VI; ++i) st.acc[cb][i] *= alpha;
        }
    }
    f16x8 p[CB][2];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        const float off = kShift - (st.m[cb] == -INFINITY ? 0.0f : st.m[cb]);
        float w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
            w[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[cb][k / 4][k % 4], c, off));
        if (masked) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (!((seen[cb] >> k) & 1u)) w[k] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) p[cb][k / 8][k % 8] = (_Float16)w[k];
#pragma unroll
        for (int n = 8; n >= 1; n /= 2)
#pragma unroll
            for (int k = 0; k < n; ++k) w[k] += w[k + n];
        st.l[cb] += w[0];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < VI; ++i) {
            const f16x8 a = vf(i, u);
#pragma unroll
            for (int cb = 0; cb < CB; ++cb)
                st.acc[cb][i] =
                    __builtin_amdgcn_mfma_f32_16x16x32_f16(a, p[cb][u], st.acc[cb][i], 0, 0, 0);
        }
}

// Columns of a sequence (its rows past max_q have none); with a block's more they fit an int.
__device__ __forceinline__ int columns(const AttendArgs& a, const Seq& sq) {
    return min(sq.n, a.max_q) * a.group;
}
// Column c of a sequence: its row (i), head of the group and the tokens it sees.
struct Column {
    int i, head, first, last;
};
__device__ __forceinline__ Column column(const AttendArgs& a, const Seq& sq, int c) {
    Column r;
    r.i = c / a.group;
    r.head = c - r.i * a.group;
    r.last = sq.L - sq.n + r.i;
    r.first = a.window > 0 && r.last - a.window + 1 > 0 ? (int)(r.last - a.window + 1) : 0;
    return r;
}

// The rows of its sequence that a tree's row sees.
__device__ __forceinline__ int rows_seen(const AttendArgs& a, const Seq& sq, const uint64_t* mask) {
    int c = 0;
    for (int i = 0; i < a.mask_words && 64 * i < sq.n; ++i) {
        const int left = sq.n - 64 * i;
        c += __popcll(mask[i] & (left >= 64 ? ~0ull : (1ull << left) - 1));
    }
    return c;
}

template <int D, int CB, bool MASKED>
__device__ __forceinline__ void load_q(const AttendArgs& a, const Seq& sq, int kvh, int c0, int cols,
                                       bf16x8 (&q)[CB][D / 32], Columns<CB, MASKED>& v) {
    const int lane = (int)threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const uint32_t sign = a.scale < 0.0f ? 0x80008000u : 0u;   // scores take |scale|
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        const int c = c0 + 16 * cb + r;
        const Column k = column(a, sq, c < cols ? c : cols - 1);
        v.first[cb] = k.first;
        v.last[cb] = k.last;
        if constexpr (MASKED) {
            v.mask[cb] = a.masks ? a.masks + (sq.lo + k.i) * a.mask_words : nullptr;
            if (a.masks)
                v.first[cb] = a.window > 0
                    ? (int)max((int64_t)0, (int64_t)sq.L - sq.n - a.window + rows_seen(a, sq, v.mask[cb])) : 0;
        }
        const uint16_t* src = a.q + (sq.lo + k.i) * a.ldq + (int64_t)(kvh * a.group + k.head) * D;
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                q[cb][2 * i + h] = __builtin_bit_cast(
                    bf16x8, *reinterpret_cast<const u32x4*>(src + 64 * i + 16 * g + 8 * h) ^ sign);
    }
    const int ce = min(c0 + 16 * CB, cols) - 1;
    v.all_to = column(a, sq, c0).last;
    v.all_from = column(a, sq, ce).first;
    if constexpr (MASKED) {
        v.words = a.mask_words;
        v.base = sq.L - sq.n;
        v.end = sq.L;
        v.sinks = a.sinks;
        if (a.masks) {               // a row sees at most n rows
            v.all_to = v.base - 1;
            v.all_from = a.window > 0 ? (int)max((int64_t)0, (int64_t)sq.L - a.window) : 0;
        }
    }
}

// Pages are walked by places: with sinks, a run of the first pages and then, past a gap, those
// of the window.  Without, a place is a page's number.
template <bool MASKED>
struct Places {
    static constexpr int sinks = 0;
    __device__ __forceinline__ int page(int p) const { return p; }
};
template <>
struct Places<true> {
    int sinks = 0, gap = 0;          // pages before the gap, and in it
    __device__ __forceinline__ int page(int p) const { return p < sinks ? p : p + gap; }
};

// The tokens' pages [p0, p1) that columns [c0, ce] see, beside the sinks.
template <bool MASKED>
__device__ __forceinline__ void page_range(const AttendArgs& a, const Seq& sq, int c0, int ce,
                                           int& p0, int& p1) {
    int first = column(a, sq, c0).first, last = column(a, sq, ce).last;
    if constexpr (MASKED) {
        if (a.masks) {               // a row that sees no row of its own looks back the furthest
            first = a.window > 0 ? (int)max((int64_t)0, (int64_t)sq.L - sq.n - a.window) : 0;
            last = sq.L - 1;
        }
    }
    p0 = first / kKvPage;
    p1 = last < 0 ? 0 : min(last / kKvPage + 1, a.seqs.max_pages);
    if (p1 < p0) p1 = p0;
}

// The places [p0, p1) of them, from 0 on where there are sinks.
template <bool MASKED>
__device__ __forceinline__ Places<MASKED> place_range(const AttendArgs& a, const Seq& sq, int c0,
                                                      int ce, int& p0, int& p1) {
    Places<MASKED> r;
    page_range<MASKED>(a, sq, c0, ce, p0, p1);
    if constexpr (MASKED) {          // the window may lie past the table, the sinks before its end
        const int head = (int)(((int64_t)a.sinks + kKvPage - 1) / kKvPage);
        r.sinks = min(min(head, p0), a.seqs.max_pages);
        r.gap = p0 - r.sinks;
        p1 -= r.gap;
        p0 = 0;
    }
    return r;
}

// A split's part of them: runs of split_pages pages; the last split takes what is left,
// however many.
__device__ __forceinline__ void split_range(const AttendArgs& a, int split, int& p0, int& p1) {
    const int64_t run = p0 + (int64_t)split * a.split_pages;
    if (split + 1 < a.splits) p1 = (int)min((int64_t)p1, run + a.split_pages);
    p0 = (int)min((int64_t)p1, run);
}

// The result of a column: O = acc 2^unit / l, or the partial sums of a split.
template <int D>
__device__ __forceinline__ void store_column(const AttendArgs& a, const Seq& sq, int kvh, int c,
                                             int cols, int split, const f32x4 (&o)[D / 16], float m,
                                             float l) {
    const int g = (int)(threadIdx.x & 63) >> 4;
    if (c >= cols) return;
    const Column k = column(a, sq, c);
    const int64_t row = sq.lo + k.i;
    const int head = kvh * a.group + k.head;
    if (a.splits > 1) {
        const int64_t at = ((int64_t)split * a.seqs.num_rows + row) * a.num_q_heads + head;
        float* dst = a.part_o + at * D;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) *reinterpret_cast<f32x4*>(dst + 16 * i + 4 * g) = o[i];
        if (g == 0) {
            a.part_ml[2 * at] = m;
            a.part_ml[2 * at + 1] = l;
        }
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t* dst = a.out + row * a.ldo + (int64_t)head * D;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        const bf16x2 x = {(__bf16)(o[i][0] * inv), (__bf16)(o[i][1] * inv)};
        const bf16x2 y = {(__bf16)(o[i][2] * inv), (__bf16)(o[i][3] * inv)};
        *reinterpret_cast<u32x2*>(dst + 16 * i + 4 * g) =
            (u32x2){__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y)};
    }
    if (a.lse && g == 0)
        a.lse[row * a.num_q_heads + head] =
            l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// Few columns (decode): a workgroup takes 16 CB columns of one (sequence, head)
// and a run of their pages, its W waves every W-th page; their states meet
// in LDS at the end.  ONCE: no other workgroup of the sequence reads these pages
// (one block of columns), so they are loaded past the caches' retention.  Bound by
// the pages' bytes: 64 sequences of 8192 tokens, 32 heads on 8 of 128, take 112 us
// (6.0 TB/s; a call 115, without ONCE 131).  Sequences that share their pages pay
// for it, as the host does not know of them: 64 forks of one such prompt take 78 us
// a call and would take 61, 8 of 100000 tokens 246 and 222 (apart 183 and 205).
//
// More columns than that but too few workgroups for the form below (trees of drafted tokens):
// bound by the vector instructions, the conversion of a page's 16384 codes to 16 bits above
// all, which two blocks of columns share (CB = 2).  16 trees of 48 tokens over 1500 .. 6000,
// 32 heads on 8 of 128, then take 89 us a call, with one block 97.  The longest sequences go
// first, as their workgroups come in more than one round (80 us, in the table's order 89).
// The next page's K loaded when this one's has been multiplied, V's behind it, gave nothing (81).
template <int D, int CB, int W, bool ONCE, bool MASKED>
__global__ void __launch_bounds__(64 * W, D == 256 ? 1 : W == 4 && CB == 1 ? 3 : 2)
attend_split_kernel(const AttendArgs a) {
    __shared__ float sm[W][16 * CB], sl[W][16 * CB];
    __shared__ f32x4 so[W / 2][D / 16][64];
    // heads fastest: workgroups that run at the same time read the parts of a page
    uint32_t b = blockIdx.x;
    const int kvh = (int)(b % (uint32_t)a.cache.num_heads);
    b /= (uint32_t)a.cache.num_heads;
    const int blk = (int)(b % (uint32_t)a.col_blocks);
    b /= (uint32_t)a.col_blocks;
    const int split = (int)(b % (uint32_t)a.splits);
    int s = (int)(b / (uint32_t)a.splits);
    if constexpr (CB > 1)
        if (a.seqs.num_seqs <= 64) s = longest(a.seqs, s);
    const Seq sq = load_seq(a.seqs, s);
    const int cols = columns(a, sq), c0 = 16 * CB * blk;
    if (c0 >= cols) return;
    const int lane = (int)threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    int p0, p1;
    const Places<MASKED> places = place_range<MASKED>(a, sq, c0, min(c0 + 16 * CB, cols) - 1, p0, p1);
    int from = p0, to = p1;
    split_range(a, split, from, to);
    if (split > 0 && from >= to) return;           // nor does the join look at it
    const int32_t* row = a.seqs.table + (int64_t)s * a.seqs.table_stride;
    int32_t next = from + wave < to ? row[places.page(from + wave)] : 0;
    bf16x8 q[CB][D / 32];
    Columns<CB, MASKED> v;
    load_q<D, CB>(a, sq, kvh, c0, cols, q, v);

    AttState<D, CB> st;
    init_state(st);
    Unit unit;
    const float cc = __builtin_fabsf(a.scale) * kLog2e;
    const int64_t head_off = (int64_t)kvh * D * kKvPage;
    for (int at_ = from + wave; at_ < to; at_ += W) {
        const int p = places.page(at_);
        const int32_t page = next;
        next = at_ + W < to ? row[places.page(at_ + W)] : 0;   // ahead of this page's loads
        if (page < 0 || page >= a.cache.num_pages) continue;
        const int64_t at = (int64_t)page * a.cache.page_stride + head_off;
        const uint8_t* kb = a.cache.k_codes + at + g * 1024 + r * 16;
        const uint8_t* vb = a.cache.v_codes + at + r * 64 + g * 16;
        const int64_t so_ = (int64_t)page * a.cache.scale_stride + kvh;
        auto load = [](const uint8_t* x) {
            if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x));
            else return *reinterpret_cast<const u32x4*>(x);
        };
        // all of the page's loads first
        u32x4 kr[4][D / 64], vr[D / 16];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < D / 64; ++i) kr[j][i] = load(kb + i * 4096 + j * 256);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) vr[i] = load(vb + i * 1024);
        const uint32_t ks = a.cache.k_scales[so_], vs = a.cache.v_scales[so_];
        const float vf = unit.follow(vs);
        if (unit.unit != st.unit) move_unit(st, unit.unit);
        if (p * kKvPage + kKvPage > sq.L) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    vr[i][j] &= before_end(p * kKvPage + 16 * j + 4 * g, sq.L);
        }
        attend_page<D, CB, MASKED, false>(
            st, v, q,
            [&](int j, int k) {
                const u32x4& x = kr[j][k / 2];
                return to_bf16(x[2 * (k % 2)], x[2 * (k % 2) + 1]);
            },
            [&](int i, int u) { return to_f16(vr[i][2 * u], vr[i][2 * u + 1], vf); }, ks, vs,
            p * kKvPage, cc);
    }
    // one state from the waves': their largest m, sums scaled to it
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        const float l = group_sum(st.l[cb]);
        if (g == 0) {
            sm[wave][16 * cb + r] = st.m[cb];
            sl[wave][16 * cb + r] = l;
        }
    }
    __syncthreads();
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        const int x = 16 * cb + r;
        float m = sm[0][x];
#pragma unroll
        for (int w = 1; w < W; ++w) m = fmaxf(m, sm[w][x]);
        const float ms = m == -INFINITY ? 0.0f : m;
        const float f = __builtin_ldexpf(__builtin_amdgcn_exp2f(st.m[cb] - ms - kShift),
                                         max(st.unit, -200));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.acc[cb][i] *= f;
#pragma unroll
        for (int h = W / 2; h >= 1; h /= 2) {
            if (wave >= h && wave < 2 * h) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) so[wave - h][i][lane] = st.acc[cb][i];
            }
            __syncthreads();
            if (wave < h) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) st.acc[cb][i] += so[wave][i][lane];
            }
            __syncthreads();
        }
        if (wave != 0) continue;
        float total = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w)
            total += sl[w][x] * __builtin_amdgcn_exp2f(sm[w][x] - ms - kShift);
        store_column<D>(a, sq, kvh, c0 + x, cols, split, st.acc[cb], m, total);
    }
}

// Many columns (a prompt): the waves of a workgroup take 16 CB columns each
// and read the same pages.  The workgroup converts a page once, K to BF16 and
// V to FP16, into one of two LDS buffers while the other is used (the codes of
// the page after it are on their way in registers): converted by every wave for
// itself, the conversions were half of the vector instructions.  In LDS K is
// [element / 8][token][8] and V [place / 8][element][8], the matrix
// instruction's 16-byte operands: 16 lanes read 256 consecutive bytes, and
// write as many (each wave's 1 KiB of V is dealt to its lanes by columns).  Bound
// by the vector instructions of the softmax beside the matrix cores: 2 x 2048
// rows in 8192 tokens, 32 heads of 128, reach 1.06 PFLOP/s (339 us).
template <int D, int CB, int W, bool MASKED>
__global__ void __launch_bounds__(64 * W, 2) attend_rows_kernel(const AttendArgs a) {
    constexpr int kHalf = D * kKvPage, kT = 64 * W, kLoads = kHalf / (kT * 16);
    __shared__ bf16x8 k0[kHalf / 8], k1[kHalf / 8];
    __shared__ f16x8 v0[kHalf / 8], v1[kHalf / 8];
    uint32_t b = blockIdx.x;
    const int kvh = (int)(b % (uint32_t)a.cache.num_heads);
    b /= (uint32_t)a.cache.num_heads;
    // the last rows, which see the most tokens, first
    const int blk = a.col_blocks - 1 - (int)(b % (uint32_t)a.col_blocks);
    b /= (uint32_t)a.col_blocks;
    const int split = (int)(b % (uint32_t)a.splits), s = (int)(b / (uint32_t)a.splits);
    const Seq sq = load_seq(a.seqs, s);
    const int cols = columns(a, sq);
    const int tid = (int)threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int w0 = 16 * CB * W * blk;              // the workgroup's first column
    if (w0 >= cols) return;
    const int c0 = w0 + 16 * CB * wave;
    const bool mine = c0 < cols;
    bf16x8 q[CB][D / 32];
    Columns<CB, MASKED> v;
    load_q<D, CB>(a, sq, kvh, mine ? c0 : w0, cols, q, v);
    int p0, p1, q0 = 0, q1 = 0;                    // the workgroup's places, the wave's pages
    const Places<MASKED> places =
        place_range<MASKED>(a, sq, w0, min(w0 + 16 * CB * W, cols) - 1, p0, p1);
    if (mine) page_range<MASKED>(a, sq, c0, min(c0 + 16 * CB, cols) - 1, q0, q1);
    if (a.splits > 1) {
        split_range(a, split, p0, p1);
        if (split > 0 && p0 >= p1) return;         // nor does the join look at it
    }
    AttState<D, CB> st;
    init_state(st);
    const float cc = __builtin_fabsf(a.scale) * kLog2e;
    const int32_t* row = a.seqs.table + (int64_t)s * a.seqs.table_stride;
    const int64_t head_off = (int64_t)kvh * D * kKvPage;

    // Pages on their way, in registers: 16 pieces of 16 bytes a wave and load, and the scale
    // bytes.  Page numbers are loaded one page ahead of that.  Both stay in vector
    // registers until they are used (`lane0` hides that they are the same in all lanes):
    // moved to scalar ones at the load, they made every page wait for its memory.
    u32x4 kr[kLoads], vr[kLoads];
    uint32_t ks_v = 0, vs_v = 0;
    int32_t page_v = -1;
    int page_in = -1;                              // the page fetched last; -1: none
    int lane0 = 0;
    asm volatile("" : "+v"(lane0));
    auto look_up = [&](int p) { page_v = row[places.page(min(p, p1 - 1)) + lane0]; };
    auto fetch = [&](int p) {
        const int page = __builtin_amdgcn_readfirstlane(page_v);
        page_in = p < p1 && page >= 0 && page < a.cache.num_pages ? page : -1;
        if (p + 1 < p1) look_up(p + 1);
        if (page_in < 0) return;
        const int64_t at = (int64_t)page_in * a.cache.page_stride + head_off;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            kr[k] = *reinterpret_cast<const u32x4*>(a.cache.k_codes + at + (k * kT + tid) * 16);
            vr[k] = *reinterpret_cast<const u32x4*>(a.cache.v_codes + at + (k * kT + (tid & ~63) + 4 * r + g) * 16);
        }
        const int64_t so_ = (int64_t)page_in * a.cache.scale_stride + kvh + lane0;
        ks_v = a.cache.k_scales[so_];
        vs_v = a.cache.v_scales[so_];
    };
    // scale bytes and unit of the page converted last (ks 256: it was none)
    uint32_t ks = 256, vs = 0;
    Unit unit;
    auto convert = [&](int p, bf16x8* kb, f16x8* vb) {
        ks = 256;
        if (page_in < 0) return;
        ks = __builtin_amdgcn_readfirstlane(ks_v);
        vs = __builtin_amdgcn_readfirstlane(vs_v);
        const float vf = unit.follow(vs);
        const int page = places.page(p);
        if (page * kKvPage + kKvPage > sq.L) {
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    vr[k][j] &= before_end(page * kKvPage + 16 * j + 4 * g, sq.L);
        }
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const int x = k * kT + tid;
            bf16x8* ko = kb + (x >> 6) * 128 + (x & 63);      // 16-element chunk, token
            ko[0] = to_bf16(kr[k][0], kr[k][1]);
            ko[64] = to_bf16(kr[k][2], kr[k][3]);
            f16x8* vo = vb + 2 * g * D + (x >> 6) * 16 + r;
            vo[0] = to_f16(vr[k][0], vr[k][1], vf);
            vo[D] = to_f16(vr[k][2], vr[k][3], vf);
        }
    };
    if (p0 < p1) look_up(p0);
    fetch(p0);
    convert(p0, k0, v0);
    fetch(p0 + 1);
    auto page_step = [&](int p, const bf16x8* kb, const f16x8* vb, bf16x8* ko, f16x8* vo) {
        // page p is in LDS, and no wave reads the other buffer any more
        __syncthreads();
        const uint32_t ks_now = ks, vs_now = vs;
        const int unit_now = unit.unit;
        convert(p + 1, ko, vo);
        fetch(p + 2);
        if (unit_now != st.unit) move_unit(st, unit_now);
        const int page = places.page(p);
        bool skip = page < q0 || page >= q1;
        if constexpr (MASKED)        // the workgroup's first columns look back further
            if (mine && page < q1 && (int64_t)page * kKvPage < a.sinks) skip = false;
        if (skip || ks_now == 256u) return;
        attend_page<D, CB, MASKED, true>(
            st, v, q, [&](int j, int k) { return kb[(8 * (k >> 1) + 2 * g + (k & 1)) * 64 + 16 * j + r]; },
            [&](int i, int u) { return vb[(2 * g + u) * D + (16 * i + r)]; }, ks_now,
            vs_now, page * kKvPage, cc);
    };
    for (int p = p0; p < p1; p += 2) {
        page_step(p, k0, v0, k1, v1);
        if (p + 1 < p1) page_step(p + 1, k1, v1, k0, v0);
    }
    if (!mine) return;
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        const float l = group_sum(st.l[cb]) * __builtin_ldexpf(1.0f, -(int)kShift);
        const float f = __builtin_ldexpf(1.0f, max(st.unit - (int)kShift, -200));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.acc[cb][i] *= f;
        store_column<D>(a, sq, kvh, c0 + 16 * cb + r, cols, split, st.acc[cb], st.m[cb], l);
    }
}

// Joins the splits' partial results: W waves per (row, head), a lane D / 64 consecutive
// elements.  Wave w takes the splits w, w + W, ..., and the waves' sums are added in their
// order.  The weights of 64 splits are found at once, a lane each, while the first sums are on
// their way.  Both sides of kJoinAlone: 64 rows of 32 heads of 128, few splits each, take 4.7 us
// with a wave for a pair and 8.6 with four; 4 rows of 32 heads over 32 splits 12.0 and 6.3.
template <int D, int W, bool MASKED>
__global__ void __launch_bounds__(kThreads) attend_join_kernel(const AttendArgs a) {
    constexpr int E = D / 64, kAhead = 8;
    __shared__ float so[kWaves][D], sl[kWaves];
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const uint32_t pair = W == 1 ? blockIdx.x * kWaves + wave : blockIdx.x;
    const int first = W == 1 ? 0 : wave;
    const int head = (int)(pair % (uint32_t)a.num_q_heads);
    const uint32_t si = pair / (uint32_t)a.num_q_heads;
    const int i = (int)(si % (uint32_t)a.max_q), s = (int)(si / (uint32_t)a.max_q);
    if (s >= a.seqs.num_seqs) return;              // the last workgroup of W == 1
    const Seq sq = load_seq(a.seqs, s);
    if (i >= sq.n) return;
    // splits past the sequence's pages hold nothing and are not read
    const int c0 = (i * a.group + head % a.group) / a.block_cols * a.block_cols;
    int p0, p1;
    place_range<MASKED>(a, sq, c0, min(c0 + a.block_cols, columns(a, sq)) - 1, p0, p1);
    const int used = (int)min((int64_t)a.splits,
                              ((int64_t)p1 - p0 + a.split_pages - 1) / a.split_pages);
    const int64_t row = sq.lo + i, at = row * a.num_q_heads + head;
    const int64_t stride = a.seqs.num_rows * a.num_q_heads;
    const float* part = a.part_o + at * D + lane * E;
    const float* ml = a.part_ml + 2 * at;
    float next[kAhead][E];
    const auto load = [&](int k0) {
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int k = k0 + x * W;
#pragma unroll
            for (int e = 0; e < E; ++e) next[x][e] = k < used ? part[k * stride * D + e] : 0.0f;
        }
    };
    load(first);
    float m = -INFINITY, mk = -INFINITY, lk = 0.0f;    // mk, lk: of split `lane`
    if (lane < used) {
        m = mk = ml[2 * lane * stride];
        lk = ml[2 * lane * stride + 1];
    }
    for (int k = lane + 64; k < used; k += 64) m = fmaxf(m, ml[2 * k * stride]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    const float ms = m == -INFINITY ? 0.0f : m;
    float l = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    float f = __builtin_amdgcn_exp2f(mk - ms);         // 0 past the last split
    lk *= f;
    for (int k0 = first;;) {
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int k = (k0 + x * W) & 63;
            l += __shfl(lk, k);
            const float w = __shfl(f, k);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += next[x][e] * w;
        }
        k0 += kAhead * W;                              // divides 64
        if (k0 - first >= used) break;
        load(k0);
        if (k0 == first + (k0 & ~63)) {                // the next 64 splits' weights
            const int k = k0 - first + lane;
            f = k < used ? __builtin_amdgcn_exp2f(ml[2 * k * stride] - ms) : 0.0f;
            lk = k < used ? ml[2 * k * stride + 1] * f : 0.0f;
        }
    }
    __bf16* dst = reinterpret_cast<__bf16*>(a.out) + row * a.ldo + (int64_t)head * D;
    if constexpr (W == 1) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int e = 0; e < E; ++e) dst[lane * E + e] = (__bf16)(o[e] * inv);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) so[wave][lane * E + e] = o[e];
        if (lane == 0) sl[wave] = l;
        __syncthreads();
        l = (sl[0] + sl[1]) + (sl[2] + sl[3]);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        for (int d = (int)threadIdx.x; d < D; d += kThreads)
            dst[d] = (__bf16)(((so[0][d] + so[1][d]) + (so[2][d] + so[3][d])) * inv);
    }
    if (a.lse && (W == 1 ? lane : (int)threadIdx.x) == 0)
        a.lse[at] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// 16-column blocks of a wave of the rows form (D = 256: one block's sums fill the registers
// that two do at 128), and columns of its workgroup, narrow and wide.  A wide one's eight
// waves share the conversion of a page, half the work of two narrow ones, but end together:
// with 32 heads of 128, 2 sequences of 2048 rows in 8192 tokens (512 wide workgroups) take
// 339 us wide and 361 narrow, 2 of 1024 in 4000 (256) 157 and 112.  Between them wide is the
// faster already: 1792 rows (448) 333 and 348, 1500 (384) 327 and 338, 1280 (320) 289 and 320.
// head_dim 64 is narrow (its page is too small for 512 threads), 256 has eight waves at 128
// columns.
template <int D>
constexpr int kRowBlocks = D == 256 ? 1 : 2;
constexpr int kRowColumns = 128, kWideColumns = 256;

constexpr int64_t kJoinAlone = 1024;

template <int D, int W, bool MASKED>
void attend_rows(const AttendArgs& a, dim3 grid, hipStream_t stream) {
    hipLaunchKernelGGL((attend_rows_kernel<D, kRowBlocks<D>, W, MASKED>), grid, dim3(64 * W), 0, stream, a);
}

template <int D, bool MASKED>
hipError_t attend(const AttendArgs& a, const AttendPlan& p, hipStream_t stream) {
    const int64_t per = (int64_t)a.seqs.num_seqs * a.cache.num_heads * a.col_blocks;
    const dim3 grid((uint32_t)(per * a.splits));
    if (p.rows_form) {
        if constexpr (D == 256) attend_rows<D, 8, MASKED>(a, grid, stream);
        else if constexpr (D == 64) attend_rows<D, 4, MASKED>(a, grid, stream);
        else if (p.wide) attend_rows<D, 8, MASKED>(a, grid, stream);
        else attend_rows<D, 4, MASKED>(a, grid, stream);
    } else if (p.block_cols == 32) {
        if constexpr (MASKED && D != 256) {
            hipLaunchKernelGGL((attend_split_kernel<D, 2, 4, false, true>), grid, dim3(256), 0, stream, a);
        } else {
            return hipErrorInvalidConfiguration;   // no plan of these kernels
        }
    } else if (p.wide) {
        hipLaunchKernelGGL((attend_split_kernel<D, 1, 8, false, MASKED>), grid, dim3(512), 0, stream, a);
    } else if (a.col_blocks == 1) {
        hipLaunchKernelGGL((attend_split_kernel<D, 1, 4, true, MASKED>), grid, dim3(256), 0, stream, a);
    } else {
        hipLaunchKernelGGL((attend_split_kernel<D, 1, 4, false, MASKED>), grid, dim3(256), 0, stream, a);
    }
    if (a.splits > 1) {
        const int64_t pairs = (int64_t)a.seqs.num_seqs * a.max_q * a.num_q_heads;
        if (pairs >= kJoinAlone)
            hipLaunchKernelGGL((attend_join_kernel<D, 1, MASKED>),
                               dim3((uint32_t)((pairs + kWaves - 1) / kWaves)), dim3(kThreads), 0,
                               stream, a);
        else
            hipLaunchKernelGGL((attend_join_kernel<D, kWaves, MASKED>), dim3((uint32_t)pairs),
                               dim3(kThreads), 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace

namespace {
template <int D>
void append(const AppendArgs& a, hipStream_t stream) {
    const dim3 grid((uint32_t)((int64_t)a.seqs.num_seqs * a.pages_per_seq),
                    (uint32_t)a.cache.num_heads, 2);
    if (append_threads(a.max_new) == 64)
        hipLaunchKernelGGL((kv_append_kernel<D, 64, 2>), grid, dim3(64), 0, stream, a);
    else
        hipLaunchKernelGGL((kv_append_kernel<D, kThreads, 16>), grid, dim3(kThreads), 0, stream, a);
}
}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, hipStream_t stream) {
    switch (a.cache.head_dim) {
        case 64: append<64>(a, stream); break;
        case 128: append<128>(a, stream); break;
        default: append<256>(a, stream); break;
    }
    return hipGetLastError();
}

// How work is split, with 32 heads of 128 on 8.  Target: 64 sequences of 8192 tokens 115 us a
// call (1024: 128, 4096: 114).  Least: 4 of 6000 tokens 14.3 us (8: 18.1, 32: 16.8).  None:
// 16 sequences of 5 rows in a window of 1024, 8 heads of 64, 8.4 us (split 12.8).  kRowsLeast:
// 128 rows in 1024 tokens 18.8 us (8 pages at least: 23.8, 16: 29.8).
constexpr int64_t kSplitTarget = 2048, kSplitLeast = 16, kSplitNone = 40;
constexpr int64_t kRowsLeast = 4;

// Masked calls (sinks, trees) of more than 16 columns: a chunk of a prompt in a window, and some
// tens of drafted tokens.  The form of many rows pays from 512 full workgroups of 128 columns on
// (1024 rows of 16 heads on 4 of 128 in a window of 2048, of 2, 3, 4 and 8 sequences: 63, 87, 87
// and 160 us, in blocks of 32 columns 54, 81, 105 and 192; trees of 48 tokens over 1500 .. 6000,
// 32 heads on 8, of 4, 16 and 32: 43, 116 and 161, in blocks 38, 80 and 146).  Fewer take blocks
// of 16 columns, or of 32 where there are kTwoBlocks of 16 (512: 36 and 38 us, 1024 of which the
// second holds 4 columns: 124 and 102), with four waves: eight, which are the faster for few blocks of
// 16, are the slower here (in a graph, 64 trees of 8 tokens over 125 .. 500: 19.3 us, with eight waves
// 28.7; over 1000 .. 4000: 71 and 75; 16 of 32 over those: 39 and 46; 64 of 8 with heads of 64: 12.6
// and 20.7, 36 and 40).  A tree has many pairs to join, so the pages are split
// only until there are kMaskedGroups workgroups (25 tokens over 20000, 56 workgroups: unsplit 67
// us, in four 31, in twenty 31; 100 over 6000, 200 workgroups: 27, in two 37, in four 34).
// Few columns of many pages are the form of many rows' again, its pages split: up to 80
// workgroups of 128 columns from kManyPages on (48 tokens over 30000: 53 us, in blocks 76; 300
// rows in 16000, 80 workgroups: 110 and 139; 100 over 10000, 157 pages: 42 and 42; 4 x 100 over
// 10000, 128 workgroups: 104 and 82).  So are columns of head_dim 256, whose blocks are never two,
// from 64 such workgroups on (1024 rows of 16 heads on 4 in a window of 4000, 128: 104 and 155;
// 4 x 100 of 8 on 2, 32: 33 and 30).
constexpr int64_t kMaskedRows = 512, kTwoBlocks = 768, kMaskedGroups = 256;
constexpr int64_t kManyPages = 150;

// The pages that one of a call's rows sees, or a block of them.
int64_t pages_seen(int64_t max_kv, int64_t window, int64_t sinks, int64_t rows) {
    const int64_t pages = (max_kv + kKvPage - 1) / kKvPage;
    if (window == 0 || window >= max_kv) return pages;
    return std::min(pages, (window + rows) / kKvPage + 2 + (sinks + kKvPage - 1) / kKvPage);
}

bool masked_as_rows(double heads, int64_t head_dim, int64_t cols, int64_t pages) {
    const double groups = heads * (double)((cols + kRowColumns - 1) / kRowColumns);
    if (cols <= 64) return false;
    return head_dim == 256 ? groups >= 64 || pages >= kManyPages : groups <= 80 && pages >= kManyPages;
}

AttendPlan plan_masked(int64_t num_heads, int64_t head_dim, int64_t num_q_heads, int64_t num_seqs,
                       int64_t max_q, int64_t max_kv, int64_t window, int64_t sinks, bool tree) {
    const int64_t group = num_q_heads / num_heads, cols = max_q * group;
    const double heads = (double)num_seqs * (double)num_heads;
    AttendPlan p{};
    p.masked = true;
    p.rows_form = cols > 64 && heads * (double)cols >= (double)kMaskedRows * kRowColumns;
    p.block_cols = 16;
    if (p.rows_form) {
        p.wide = head_dim == 128 && heads * (double)(cols / kWideColumns) >= 512;
        p.block_cols = p.wide ? kWideColumns : kRowColumns;
    } else if (head_dim != 256 && heads * (double)((cols + 15) / 16) >= kTwoBlocks) {
        p.block_cols = 32;
    }
    p.col_blocks = (int32_t)((cols + p.block_cols - 1) / p.block_cols);
    const int64_t pages = pages_seen(max_kv, window, sinks,
                                     tree ? max_q : std::min(max_q, p.block_cols / group + 2));
    const double blocks = heads * p.col_blocks;
    int64_t run = std::max<int64_t>(pages, 1);
    if (!p.rows_form && pages > kSplitNone && blocks > 0) {
        const int64_t n = std::max<int64_t>((int64_t)(kMaskedGroups / blocks + 0.5), 1);
        run = ((pages + n - 1) / n + kWaves - 1) / kWaves * kWaves;
        run = std::max(run, kSplitLeast);
    }
    p.splits = (int32_t)std::max<int64_t>((pages + run - 1) / run, 1);
    if (!p.rows_form) p.wide = p.block_cols == 16 && blocks * p.splits <= 512;
    p.threads = p.wide || (p.rows_form && head_dim == 256) ? 512 : 256;
    p.split_pages = (int32_t)run;
    return p;
}

AttendPlan plan_attend(int64_t num_heads, int64_t head_dim, int64_t num_q_heads, int64_t num_seqs,
                       int64_t max_q, int64_t max_kv, int64_t window, int64_t sinks, bool tree) {
    const bool masked = tree || (sinks > 0 && window > 0);
    if (masked && max_q * (num_q_heads / num_heads) > 16 &&
        !masked_as_rows((double)num_seqs * (double)num_heads, head_dim,
                        max_q * (num_q_heads / num_heads), pages_seen(max_kv, window, sinks, 0)))
        return plan_masked(num_heads, head_dim, num_q_heads, num_seqs, max_q, max_kv, window, sinks,
                           tree);
    const int64_t cols = max_q * (num_q_heads / num_heads);
    AttendPlan p{};
    p.masked = masked;
    p.rows_form = cols > 64;
    int64_t pages = (max_kv + kKvPage - 1) / kKvPage;
    if (window > 0 && window < max_kv) {
        const int64_t seen = (window + max_q) / kKvPage + 2 + (sinks + kKvPage - 1) / kKvPage;
        pages = sinks > 0 ? std::min(pages, seen) : seen;
    }
    const double heads = (double)num_seqs * (double)num_heads;
    p.block_cols = p.rows_form ? kRowColumns : 16;
    if (p.rows_form) {
        p.wide = head_dim == 128 && heads * (double)(cols / kWideColumns) >= 512;
        if (p.wide) p.block_cols = kWideColumns;
    }
    p.col_blocks = (int32_t)((cols + p.block_cols - 1) / p.block_cols);
    // Joining costs a second kernel (4 us and more), as much as a workgroup of the split form
    // takes for 32 pages more: up to kSplitNone pages that form splits nothing.
    const double blocks = heads * p.col_blocks;
    int64_t run;
    if (!p.rows_form) {
        // runs that give kSplitTarget workgroups if every sequence were the longest
        run = (int64_t)std::ceil(std::min((double)pages, (double)pages * blocks / kSplitTarget));
        run = (std::max(run, kSplitLeast) + kWaves - 1) / kWaves * kWaves;
        if (pages <= kSplitNone) run = kSplitNone;
    } else {
        // The rows form splits until the CUs hold all the workgroups they can (3, 2 and 1 each by
        // head_dim), but not where half of those are there already, nor where the pages are too
        // few for the sums that are joined, which grow with the workgroups: 192 of 128 pages 153
        // us, unsplit 187; 128 of 24 pages 37 and 42, of 16 32 and 31; 128 of 10 pages of
        // head_dim 64 27 and 17; 8 of 94 pages 23 and 144.
        const double slots = head_dim == 64 ? 768 : head_dim == 128 ? 512 : 256;
        const bool many = blocks <= slots / 2 && blocks <= 256 && 16.0 * pages >= 3.0 * blocks;
        const int64_t n = many && blocks > 0 ? std::llround(slots / blocks) : 1;
        run = std::max((pages + n - 1) / n, kRowsLeast);
    }
    const int64_t splits = (pages + run - 1) / run;
    p.splits = splits < 1 ? 1 : (int32_t)splits;
    // little work: eight waves share a run, so each walks half as many pages (8 sequences of 777
    // tokens 8.8 us, with four 10.8; 64 of 8192 145 and 115)
    if (!p.rows_form) p.wide = blocks * p.splits <= 512;
    p.threads = p.wide || (p.rows_form && head_dim == 256) ? 512 : 256;
    p.split_pages = (int32_t)run;
    return p;
}

namespace {
template <bool MASKED>
hipError_t attend_of(const AttendArgs& a, const AttendPlan& p, hipStream_t stream) {
    switch (a.cache.head_dim) {
        case 64: return attend<64, MASKED>(a, p, stream);
        case 128: return attend<128, MASKED>(a, p, stream);
        default: return attend<256, MASKED>(a, p, stream);
    }
}
}  // namespace

hipError_t launch_kv_attend(const AttendArgs& a, const AttendPlan& p, hipStream_t stream) {
    return p.masked ? attend_of<true>(a, p, stream) : attend_of<false>(a, p, stream);
}

}  // namespace bsq
