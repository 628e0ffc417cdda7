// bsq_moe.hip -- gfx950 kernels of the mixture-of-experts layer for a few
// tokens over MX weights (include/bsq_serving.h).
//
// With a few tokens the weights of the chosen experts are nearly all of the
// bytes, each read once and used for a handful of columns, so both kernels
// stream weights from memory straight to registers and feed the matrix cores
// with them as the left operand (16 weight rows), the tokens being the 16
// columns:  mfma_f32_16x16x32_bf16, lane l holding weight row l % 16 and whole
// MX blocks of it, so that a lane's codes have one scale each, which their
// conversion to BF16 applies exactly.  (The contraction's order is free as long
// as the tokens' values follow it.)
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "bsq.h"
#include "bsq_serving_internal.h"

namespace bsq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// A wave takes weights in steps of whole cache lines of each row: CH 128-element
// chunks, 64 bytes of E2M1 codes or 128 of E4M3 each.  Of a chunk lane group g
// takes the 32 elements at 32 g, one MX block; its scales in the step's chunks
// are bytes of the dword that a BSQ_SCALES_MFMA16 record keeps for the lane.
template <int FMT>
constexpr int kLong = FMT == BSQ_MXFP8 ? 2 : 4;          // chunks in 256 bytes
template <int FMT>
constexpr int kShort = FMT == BSQ_MXFP8 ? 1 : 2;         // and in 128
template <int FMT>
constexpr int kLoads = FMT == BSQ_MXFP8 ? 2 : 1;         // 16-byte loads of a lane and chunk

template <int FMT, int NT, int CH>
struct Step {
    u32x4 w[NT][CH * kLoads<FMT>];
    uint32_t s[NT];                  // scale bytes, chunk by chunk
};

// Where a lane's weights of NT 16-row tiles lie: its codes of chunk 0 and its dword of
// record 0.
template <int NT>
struct Rows {
    const uint8_t* w[NT];
    const uint8_t* s[NT];
};

// Rows row .. row + 15 (row a multiple of 16) of codes and scale records of K elements a row.
template <int FMT, int NT>
__device__ __forceinline__ void set_rows(Rows<NT>& p, int t, const uint8_t* codes,
                                         const uint8_t* scales, int64_t row, int K) {
    const int lane = (int)threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    p.w[t] = FMT == BSQ_MXFP8 ? codes + (row + r) * K + 32 * g : codes + (row + r) * (K / 2) + 16 * g;
    p.s[t] = scales + row / 16 * ((int64_t)((K + 511) / 512) * 256) + 4 * lane;
}

// Step c; chunks past the row's end repeat its last one.  Through the caches: two loads share
// each line (past them 64 tokens of 4 of 64 experts took 172 us, this way 158).
template <int FMT, int CH, int NT>
__device__ __forceinline__ Step<FMT, NT, CH> load_step(const Rows<NT>& p, int c, int K) {
    constexpr int L = kLoads<FMT>;
    Step<FMT, NT, CH> r;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const u32x4* w = reinterpret_cast<const u32x4*>(
                p.w[t] + (int64_t)min(c * CH + i, K / 128 - 1) * (64 * L));
#pragma unroll
            for (int k = 0; k < L; ++k) r.w[t][L * i + k] = w[k];
        }
        const uint8_t* s = p.s[t] + (int64_t)(c * CH >> 2) * 256 + (c * CH & 3);
        if constexpr (CH == 4) r.s[t] = *reinterpret_cast<const uint32_t*>(s);
        else if constexpr (CH == 2) r.s[t] = *reinterpret_cast<const uint16_t*>(s);
        else r.s[t] = *s;
    }
    return r;
}

// 2^(b - 127); 255 is NaN
__device__ __forceinline__ float scale_of(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7FC00000u : b == 0u ? 0x00400000u : b << 23);
}

// The lane's 32 codes of tile t and chunk i, times their scale, as BF16: exact (a code's few
// bits times a power of two) wherever the product is a normal number.
template <int FMT, int NT, int CH>
__device__ __forceinline__ void convert(const Step<FMT, NT, CH>& st, int t, int i, bf16x8 (&o)[4]) {
    const float f = scale_of((st.s[t] >> (8 * i)) & 255u);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        bf16x2 p[4];
        if constexpr (FMT == BSQ_MXFP8) {
            const u32x4& w = st.w[t][2 * i + s / 2];
            const uint32_t a = w[2 * (s % 2)], b = w[2 * (s % 2) + 1];
            p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, f, false);
            p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, f, true);
            p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, f, false);
            p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, f, true);
        } else {
            const uint32_t a = st.w[t][i][s];
            p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, f, 0);
            p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, f, 1);
            p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, f, 2);
            p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, f, 3);
        }
        o[s] = (bf16x8){p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
    }
}

// ------------------------------------------------------------ routing

// The logits' order as unsigned integers: NaN counts as -inf, -0 as 0; 0 is below all.
__device__ __forceinline__ uint32_t logit_key(float x) {
    const uint32_t b = __float_as_uint((x == x ? x : -INFINITY) + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
// The largest of the wave's numbers, in every lane: rotations by 8, 4, 2, 1 within the
// rows of 16 lanes, then across them.
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
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
    return v;
}

// One wave: a token's topk experts and their weights, lane j getting the j-th.
// Each round takes the largest logit left, the lowest expert among equals.
// REGS: experts / 64, rounded up.
template <int REGS>
__device__ __forceinline__ void route(const MoeArgs& a, const float* logits, int& id, float& weight) {
    const int lane = (int)threadIdx.x & 63;
    uint32_t key[REGS];
    float x[REGS];
#pragma unroll
    for (int k = 0; k < REGS; ++k) x[k] = 64 * k + lane < a.experts ? logits[64 * k + lane] : 0.0f;
#pragma unroll
    for (int k = 0; k < REGS; ++k) key[k] = 64 * k + lane < a.experts ? logit_key(x[k]) : 0u;
    id = 0;
    uint32_t mine = 0, top = 0;
    for (int j = 0; j < a.topk; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int k = 1; k < REGS; ++k) best = max(best, key[k]);
        best = wave_max(best);
        if (j == 0) top = best;
        bool taken = false;
#pragma unroll
        for (int k = 0; k < REGS; ++k) {
            const uint64_t at = __ballot(key[k] == best);
            if (!taken && at) {
                taken = true;
                const int l = __ffsll((unsigned long long)at) - 1;
                if (lane == j) {
                    id = 64 * k + l;
                    mine = best;
                }
                if (lane == l) key[k] = 0;
            }
        }
    }
    // exp(x - top); +inf shares the whole weight among its equals
    const float t = key_logit(top);
    auto share = [&](float v) {
        if (!(v > -INFINITY)) return 0.0f;
        return v == t ? 1.0f : __builtin_amdgcn_exp2f((v - t) * 1.44269504088896340736f);
    };
    const float own = lane < a.topk ? share(key_logit(mine)) : 0.0f;
    float sum = own;
    if (!a.renormalize) {
        sum = 0.0f;
#pragma unroll
        for (int k = 0; k < REGS; ++k) sum += 64 * k + lane < a.experts ? share(x[k]) : 0.0f;
    }
    sum = wave_sum(sum);
    weight = sum > 0.0f ? own / sum : 0.0f;
}

__device__ __forceinline__ void route_token(const MoeArgs& a, int t, int& id, float& weight) {
    const float* logits = a.logits + (int64_t)t * a.experts;
    if (a.experts <= 128) route<2>(a, logits, id, weight);
    else if (a.experts <= 256) route<4>(a, logits, id, weight);
    else route<kMoeMaxExperts / 64>(a, logits, id, weight);
}

// More than a workgroup's waves of tokens: routed by a kernel of their own, a wave each.
__global__ void __launch_bounds__(64) moe_route_kernel(const MoeArgs a) {
    const int t = (int)blockIdx.x, lane = (int)threadIdx.x;
    int id;
    float w;
    route_token(a, t, id, w);
    if (lane < a.topk) {
        a.ids[t * a.topk + lane] = id;
        a.weights[t * a.topk + lane] = w;
    }
}

// An entry (token t, place j) is t * topk + j.  It counts if its expert
// exists, its weight is not 0 and no earlier such entry of the token names the
// same expert; the weights of those that do add up in the first.
//
// Up to kFewEntries entries a wave keeps them all in its lanes: no LDS, no barrier.
struct FewEntries {
    int id;                          // of entry `lane`; -1: no expert, no weight or no entry
    float w;                         // with the weights of equal entries of the token
    uint64_t counted;                // the entries that count
};
// distinct: no token names an expert twice (logits routed it)
__device__ __forceinline__ FewEntries few_entries(const MoeArgs& a, int id, float w, bool distinct) {
    const int lane = (int)threadIdx.x & 63;
    FewEntries r;
    const bool valid = lane < a.tokens * a.topk && id >= 0 && id < a.experts && w != 0.0f;
    r.id = valid ? id : -1;
    r.w = w;
    r.counted = __ballot(valid);
    if (distinct) return r;
    // equal entries of the token before and after this one
    const int t0 = lane - lane % a.topk;
    bool again = false;
    for (int j = 0; j < a.topk; ++j) {
        const int o = __shfl(r.id, t0 + j);
        const float ow = __shfl(w, t0 + j);
        if (o != r.id || t0 + j == lane) continue;
        if (t0 + j < lane) again = true;
        else r.w += ow;
    }
    r.counted = __ballot(valid && !again);
    return r;
}
// The entries of an expert.
__device__ __forceinline__ uint64_t entries_of(const FewEntries& e, int expert) {
    return __ballot(e.id == expert) & e.counted;
}
// Whether entry u is the first of all that name its expert, and that expert.
__device__ __forceinline__ int expert_at(const FewEntries& e, int u) {
    return __builtin_amdgcn_readlane(e.id, u);
}
// The entry of column 16 b + lane % 16 of those from b0 on: the place of that bit of m, or of
// the last one.
template <int NB>
__device__ __forceinline__ void columns_of(uint64_t m, int b0, int (&row)[NB]) {
    const int c = b0 + ((int)threadIdx.x & 15);
    for (int i = 0; m; ++i, m &= m - 1) {
        const int at = __ffsll((unsigned long long)m) - 1;
#pragma unroll
        for (int b = 0; b < NB; ++b)
            if (16 * b + c >= i) row[b] = at;
    }
}

// Whether entry r of a table in LDS counts (ids: -1 for entries without weight or expert).
__device__ __forceinline__ bool counts(const int16_t* ids, int r, int topk) {
    const int id = ids[r];
    if (id < 0) return false;
    for (int k = r - r % topk; k < r; ++k)
        if (ids[k] == id) return false;
    return true;
}

// How a workgroup knows its expert and the expert's entries:
//  kRoute  few entries, from logits, for at most kUpWaves tokens: every workgroup
//          routes them itself, a wave each (one token 17.3 us a call, with a
//          kernel to route it 19.6)
//  kFew    few entries, from topk_ids
//  kEntry  a workgroup per entry of topk_ids
//  kExpert a workgroup per expert (more entries than experts)
// Except in the last, a workgroup whose expert an earlier entry names has nothing to do.
enum RowsFrom { kRoute, kFew, kEntry, kExpert };

// kEntry and kExpert: the entries of workgroup `unit`'s expert in LDS.
struct ManyEntries {
    int16_t ids[kMoeMaxTokens * kMoeMaxTopk];
    uint16_t rows[kMoeMaxTokens];
    int n;
};
// Their number (0: nothing to do), and the expert.
template <RowsFrom FROM, int THREADS>
__device__ __forceinline__ int many_entries(const MoeArgs& a, ManyEntries& m, int unit, int& expert) {
    const int tid = (int)threadIdx.x, entries = a.tokens * a.topk;
    if (tid == 0) m.n = 0;
    for (int r = tid; r < entries; r += THREADS) {
        const int id = a.ids[r];
        m.ids[r] = (int16_t)(id < 0 || id >= a.experts || a.weights[r] == 0.0f ? -1 : id);
    }
    __syncthreads();
    expert = unit;
    if constexpr (FROM == kEntry) {
        expert = m.ids[unit];
        bool later = expert < 0;
        for (int r = tid; r < unit; r += THREADS) later |= m.ids[r] == expert;
        if (__syncthreads_or(later)) return 0;
    }
    for (int r = tid; r < entries; r += THREADS)
        if (m.ids[r] == expert && counts(m.ids, r, a.topk))
            m.rows[atomicAdd(&m.n, 1)] = (uint16_t)r;
    __syncthreads();
    return m.n;
}

// ------------------------------------------------------------ gate and up
//
// A workgroup computes 16 or 32 columns of h for one expert (G blocks of 16):
// the rows of W1 and those of W3 that belong to them, over all of `hidden`, its
// waves taking contiguous runs of the steps.  16 NB entries at a time are the
// matrix columns; columns past the last repeat it, and no result of theirs is
// stored.  Bound by the weights' bytes and by its workgroups' rounds: 394 MB in
// 86 us in FP4 (4.6 TB/s) and 553 MB in 100 us in E4M3 (5.5 TB/s) are some 1630
// and 2048 workgroups with work, 2.1 and 2.7 times the 768 that fit (three waves a
// SIMD), and the CUs hold work in 79% and 88% of that time (SQ_BUSY_CU_CYCLES over
// GRBM_GUI_ACTIVE): while they do, the weights come at 5.8 and 6.3 TB/s.  More waves
// with fewer registers, steps loaded ahead in each wave, or two or eight waves a
// workgroup were no faster.

constexpr int kUpWaves = 4, kUpThreads = 64 * kUpWaves;
constexpr float kBf16Max = 0x1.FEp127f;

template <int FMT, int NB, int G, RowsFrom FROM>
__global__ void __launch_bounds__(kUpThreads) moe_up_kernel(const MoeArgs a, int tiles) {
    __shared__ f32x4 part[kUpWaves][2 * G][64];
    const int tid = (int)threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int unit = (int)(blockIdx.x / (uint32_t)tiles), tile = (int)(blockIdx.x % (uint32_t)tiles);
    const int entries = a.tokens * a.topk;
    int expert, n;
    uint64_t few = 0;
    constexpr bool kMany = FROM == kEntry || FROM == kExpert;
    __shared__ typename std::conditional<kMany, ManyEntries, int>::type many;
    if constexpr (FROM == kRoute || FROM == kFew) {
        int id = -1;
        float w = 0.0f;
        if constexpr (FROM == kRoute) {
            __shared__ int sid[kFewEntries];
            __shared__ float sw[kFewEntries];
            if (wave < a.tokens) {
                route_token(a, wave, id, w);
                if (lane < a.topk) {
                    sid[wave * a.topk + lane] = id;
                    sw[wave * a.topk + lane] = w;
                    if (blockIdx.x == 0) {
                        a.ids[wave * a.topk + lane] = id;
                        a.weights[wave * a.topk + lane] = w;
                    }
                }
            }
            __syncthreads();
            if (lane < entries) {
                id = sid[lane];
                w = sw[lane];
            }
        } else if (lane < entries) {
            id = a.ids[lane];
            w = a.weights[lane];
        }
        const FewEntries e = few_entries(a, id, w, FROM == kRoute);
        if (!((e.counted >> unit) & 1u)) return;
        expert = expert_at(e, unit);
        few = entries_of(e, expert);
        if (few & ((1ull << unit) - 1)) return;
        n = __popcll(few);
    } else {
        n = many_entries<FROM, kUpThreads>(a, many, unit, expert);
        if (n == 0) return;
    }

    constexpr int CH = kLong<FMT>, S = 128 * CH;
    const int steps = (a.hidden + S - 1) / S;
    const int c_from = steps * wave / kUpWaves, c_to = steps * (wave + 1) / kUpWaves;
    Rows<2 * G> w;                                 // W1's tiles, then W3's
#pragma unroll
    for (int t = 0; t < 2 * G; ++t)
        set_rows<FMT>(w, t, a.w13, a.w13_scales,
                      (int64_t)expert * 2 * a.inter + (t < G ? 0 : a.inter) + 16 * (G * tile + t % G),
                      a.hidden);
    for (int b0 = 0; b0 < n; b0 += 16 * NB) {
        int row[NB];                               // the entry of column 16 b + r16
        if constexpr (FROM == kRoute || FROM == kFew) {
            columns_of<NB>(few, b0, row);
        } else {
#pragma unroll
            for (int b = 0; b < NB; ++b) row[b] = many.rows[min(b0 + 16 * b + r16, n - 1)];
        }
        const uint16_t* xr[NB];
        f32x4 acc[NB][2 * G];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            xr[b] = a.x + (row[b] / a.topk) * a.ldx + 32 * g;
#pragma unroll
            for (int t = 0; t < 2 * G; ++t) acc[b][t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        }
        for (int c = c_from; c < c_to; ++c) {
            const auto st = load_step<FMT, CH>(w, c, a.hidden);
            // with registers to spare, the tokens' values too
            constexpr bool kAhead = NB == 1 && G == 1;
            bf16x8 xa[kAhead ? CH : 1][4];
            if constexpr (kAhead) {
#pragma unroll
                for (int i = 0; i < CH; ++i)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        xa[i][s] = *reinterpret_cast<const bf16x8*>(
                            xr[0] + min(c * S + 128 * i, a.hidden - 128) + 8 * s);
            }
            // all of the step's loads before any use: the compiler sank them past the first
            // chunks' products (16 tokens over 256 experts, 7168 x 512: 153 us a call, 149 so)
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int at = c * S + 128 * i;
                if (at >= a.hidden) break;
                bf16x8 xs[NB][4];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        if constexpr (kAhead) xs[b][s] = xa[i][s];
                        else xs[b][s] = *reinterpret_cast<const bf16x8*>(xr[b] + at + 8 * s);
                    }
#pragma unroll
                for (int t = 0; t < 2 * G; ++t) {
                    bf16x8 ws[4];
                    convert<FMT>(st, t, i, ws);
#pragma unroll
                    for (int s = 0; s < 4; ++s)
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[s], xs[b][s],
                                                                                acc[b][t], 0, 0, 0);
                }
            }
        }
        // the waves' sums in their order; lane l holds columns 4 g .. 4 g + 3 of row l % 16
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (b0 + 16 * b >= n) break;
            if (b0 + b > 0) __syncthreads();
#pragma unroll
            for (int t = 0; t < 2 * G; ++t) part[wave][t][lane] = acc[b][t];
            __syncthreads();
            if (wave >= G || b0 + 16 * b + r16 >= n) continue;
            f32x4 gate = part[0][wave][lane], up = part[0][G + wave][lane];
#pragma unroll
            for (int k = 1; k < kUpWaves; ++k) {
                gate += part[k][wave][lane];
                up += part[k][G + wave][lane];
            }
            // h as the sum of two BF16 numbers, 16 bits in all: with one, its rounding
            // alone made y's error 1.4 to 1.5 times that of rounding y.  The first stays
            // finite, so that the second is never the difference of two infinities: it
            // holds what fp32 has past BF16's range, an infinity or a NaN.
            bf16x2 hi[2], lo[2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float h =
                    gate[e] / (1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * gate[e])) * up[e];
                hi[e / 2][e % 2] = (__bf16)fminf(fmaxf(h, -kBf16Max), kBf16Max);
                lo[e / 2][e % 2] = (__bf16)(h - (float)hi[e / 2][e % 2]);
            }
            uint16_t* dst = a.h + (int64_t)row[b] * 2 * a.inter + 16 * (G * tile + wave) + 4 * g;
            *reinterpret_cast<u32x2*>(dst) = (u32x2){__builtin_bit_cast(uint32_t, hi[0]),
                                                     __builtin_bit_cast(uint32_t, hi[1])};
            *reinterpret_cast<u32x2*>(dst + a.inter) = (u32x2){__builtin_bit_cast(uint32_t, lo[0]),
                                                               __builtin_bit_cast(uint32_t, lo[1])};
        }
    }
}

// ------------------------------------------------------------ down, few entries
//
// A workgroup owns 16 columns of y and walks every expert in use: no partial
// result leaves it.  The (expert, step) pairs, experts in the order of their
// first entries, are dealt to the waves in contiguous runs; a wave adds an
// expert's part, times the tokens' weights, to sums of its own in LDS, and the
// waves' sums are added in their order at the end.  At most 16 tokens.

constexpr int kDownWaves = 8, kDownThreads = 64 * kDownWaves;

template <int FMT>
__global__ void __launch_bounds__(kDownThreads) moe_down_few_kernel(const MoeArgs a) {
    constexpr int CH = kShort<FMT>, S = 128 * CH;
    // [token][4 columns]: as vectors, so that their 16-byte accesses are aligned
    __shared__ f32x4 sums[kDownWaves][16 * 4];
    const int tid = (int)threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int entries = a.tokens * a.topk;
    sums[wave][lane] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    const FewEntries few =
        few_entries(a, lane < entries ? a.ids[lane] : -1, lane < entries ? a.weights[lane] : 0.0f,
                    a.logits != nullptr);
    uint64_t firsts = 0;                           // the first entry of each expert
    for (uint64_t m = few.counted; m;) {
        const int at = __ffsll((unsigned long long)m) - 1;
        firsts |= 1ull << at;
        m &= ~entries_of(few, expert_at(few, at));
    }
    const int act = __popcll(firsts), steps = (a.inter + S - 1) / S;
    const int col0 = 16 * (int)blockIdx.x;
    const int items = act * steps;
    const int it_from = items * wave / kDownWaves, it_to = items * (wave + 1) / kDownWaves;
    auto expert_in_use = [&](int ai) {             // the ai-th
        uint64_t m = firsts;
        for (int i = 0; i < ai; ++i) m &= m - 1;
        return expert_at(few, __ffsll((unsigned long long)m) - 1);
    };
    // an item's weights and h, both one item ahead of their use: h comes from other CUs' stores
    struct Item {
        Step<FMT, 1, CH> w;
        bf16x8 hi[CH][4], lo[CH][4];
        int row, n;                                // the entry of column r16; entries of the expert
    };
    auto load = [&](int it) {
        const int ai = it / steps, c = it - ai * steps, expert = expert_in_use(ai);
        Item r;
        Rows<1> w;
        set_rows<FMT>(w, 0, a.w2, a.w2_scales, (int64_t)expert * a.hidden + col0, a.inter);
        r.w = load_step<FMT, CH>(w, c, a.inter);
        const uint64_t m = entries_of(few, expert);
        int row[1];
        columns_of<1>(m, 0, row);
        r.row = row[0];
        r.n = __popcll(m);
        const uint16_t* h = a.h + (int64_t)r.row * 2 * a.inter + 32 * g;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int at = min(c * S + 128 * i, a.inter - 128);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                r.hi[i][s] = *reinterpret_cast<const bf16x8*>(h + at + 8 * s);
                r.lo[i][s] = *reinterpret_cast<const bf16x8*>(h + a.inter + at + 8 * s);
            }
        }
        return r;
    };
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    auto use = [&](const Item& item, int it) {
        const int ai = it / steps, c = it - ai * steps;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (c * S + 128 * i >= a.inter) break;
            bf16x8 ws[4];
            convert<FMT>(item.w, 0, i, ws);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[s], item.hi[i][s], acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[s], item.lo[i][s], acc, 0, 0, 0);
            }
        }
        // the expert's (or the wave's) last step: its part goes to the tokens' sums
        if (it + 1 < it_to && it + 1 < (ai + 1) * steps) return;
        const float f = __shfl(few.w, item.row);
        if (r16 < item.n) {
            f32x4& s = sums[wave][item.row / a.topk * 4 + g];
            s = s + acc * f;
        }
        acc = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    };
    if (it_from < it_to) {
        Item s0 = load(it_from), s1;
        for (int it = it_from;; it += 2) {
            // past the wave's last item its loads repeat that item's
            s1 = load(min(it + 1, it_to - 1));
            __builtin_amdgcn_sched_barrier(0);
            use(s0, it);
            if (it + 1 >= it_to) break;
            s0 = load(min(it + 2, it_to - 1));
            __builtin_amdgcn_sched_barrier(0);
            use(s1, it + 1);
            if (it + 2 >= it_to) break;
        }
    }
    __syncthreads();
    for (int k = tid; k < a.tokens * 16; k += kDownThreads) {
        float y = reinterpret_cast<const float*>(sums[0])[k];
#pragma unroll
        for (int w = 1; w < kDownWaves; ++w) y += reinterpret_cast<const float*>(sums[w])[k];
        reinterpret_cast<__bf16*>(a.y)[k / 16 * a.ldy + col0 + k % 16] = (__bf16)y;
    }
}

// ------------------------------------------------------------ down, many entries
//
// A workgroup takes 256 columns, 32 a wave, and every splits-th expert in use.
// Its work is a sequence of stages: 512 elements of the contraction for 16
// entries of an expert, whose h the waves share in LDS (read from memory by each
// wave for its 32 columns it was four times the weights' loads).  While a stage
// is computed, the next one's h and the next steps' weights are on their way,
// over the ends of experts too: a workgroup for each expert spent its life
// waiting for its first loads (128 entries, 101 experts of 7168 x 512 in FP4:
// 92 us, this form 54, of which the weights at 6.2 TB/s are 32).  The parts,
// times the tokens' weights, go to memory in 32 bits, a row an entry, and a
// third kernel adds a token's rows in their order.

constexpr int kStage = 512;          // elements of h in LDS
// 16 bytes more than a multiple of the banks' 256: 16 rows' pieces fall in different banks
constexpr int kStageRow = kStage + 8;
constexpr int kPartCols = 32 * kDownWaves;

template <int FMT>
__global__ void __launch_bounds__(kDownThreads, 4) moe_down_part_kernel(const MoeArgs a, int tiles,
                                                                        int splits) {
    constexpr int CH = kShort<FMT>, S = 128 * CH, kSteps = kStage / S;
    constexpr int kEntries = kMoeMaxTokens * kMoeMaxTopk;
    constexpr int kPieces = 16 * 2 * kStage / 8 / kDownThreads;   // 16-byte pieces of h a thread
    __shared__ __attribute__((aligned(16))) uint16_t stage0[2 * 16 * kStageRow];
    __shared__ __attribute__((aligned(16))) uint16_t stage1[2 * 16 * kStageRow];
    __shared__ int16_t ids[kEntries];
    __shared__ uint16_t order[kEntries];           // entries that count, by expert
    __shared__ int count[kMoeMaxExperts];
    __shared__ uint16_t first[kMoeMaxExperts];     // an expert's first place in `order`
    __shared__ uint16_t active[kMoeMaxExperts + 1];// the experts in use, ascending
    __shared__ int n_active, n_entries;
    const int tid = (int)threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tile = (int)(blockIdx.x % (uint32_t)tiles), split = (int)(blockIdx.x / (uint32_t)tiles);
    const int entries = a.tokens * a.topk;
    for (int e = tid; e < a.experts; e += kDownThreads) count[e] = 0;
    for (int r = tid; r < entries; r += kDownThreads) {
        const int id = a.ids[r];
        ids[r] = (int16_t)(id < 0 || id >= a.experts || a.weights[r] == 0.0f ? -1 : id);
    }
    __syncthreads();
    for (int r = tid; r < entries; r += kDownThreads)
        if (counts(ids, r, a.topk)) atomicAdd(&count[ids[r]], 1);
    __syncthreads();
    // the experts in use and where their entries start, by the first wave
    if (wave == 0) {
        int base = 0, used_experts = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 64) {
            const int e = e0 + lane, c = e < a.experts ? count[e] : 0;
            int x = c;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int y = __shfl_up(x, off);
                if (lane >= off) x += y;
            }
            const uint64_t used = __ballot(c > 0);
            if (e < a.experts) first[e] = (uint16_t)(base + x - c);
            if (c > 0) active[used_experts + __popcll(used & ((1ull << lane) - 1))] = (uint16_t)e;
            used_experts += __popcll(used);
            base += __shfl(x, 63);
        }
        if (lane == 0) {
            n_active = used_experts;
            n_entries = base;
        }
    }
    __syncthreads();
    // an expert's entries in any order: each is a column of its own
    for (int r = tid; r < entries; r += kDownThreads)
        if (counts(ids, r, a.topk)) {
            const int id = ids[r];
            order[first[id] + atomicSub(&count[id], 1) - 1] = (uint16_t)r;
        }
    __syncthreads();
    const int act = n_active;
    if (split >= act) return;

    const int col0 = kPartCols * tile + 32 * wave;
    const bool mine = col0 < a.hidden;             // hidden is a multiple of 128
    const int steps = (a.inter + S - 1) / S;
    // a place in the sequence of stages (and, for the weights, a step of the stage)
    struct Place {
        int ai, expert, begin, n, b0, c;           // entries order[begin ..]; b0 the first of 16
    };
    auto enter = [&](Place& p, int ai) {
        p.ai = ai;
        p.b0 = p.c = 0;
        if (ai >= act) return;
        p.expert = __builtin_amdgcn_readfirstlane((int)active[ai]);
        p.begin = __builtin_amdgcn_readfirstlane((int)first[p.expert]);
        p.n = (ai + 1 < act ? __builtin_amdgcn_readfirstlane((int)first[active[ai + 1]]) : n_entries) -
              p.begin;
    };
    // to the step `by` further; past the last one ai >= act
    auto advance = [&](Place& p, int by) {
        p.c += by;
        if (p.c < steps) return;
        p.c = 0;
        p.b0 += 16;
        if (p.b0 >= p.n) enter(p, p.ai + splits);
    };
    auto load = [&](const Place& p) {
        Rows<2> w;
#pragma unroll
        for (int t = 0; t < 2; ++t)
            set_rows<FMT>(w, t, a.w2, a.w2_scales,
                          (int64_t)p.expert * a.hidden + (mine ? col0 : 0) + 16 * t, a.inter);
        return load_step<FMT, CH>(w, p.c, a.inter);
    };
    u32x4 hv[kPieces];
    auto fetch = [&](const Place& p) {
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int x = k * kDownThreads + tid;
            const int piece = x % (kStage / 8), half = x / (kStage / 8) & 1, row = x / (kStage / 4);
            const int at = p.c * S + 8 * piece;
            if (p.b0 + row < p.n && at < a.inter)
                hv[k] = *reinterpret_cast<const u32x4*>(
                    a.h + ((int64_t)order[p.begin + p.b0 + row] * 2 + half) * a.inter + at);
        }
    };
    auto keep = [&](const Place& p, uint16_t* stage) {
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int x = k * kDownThreads + tid;
            const int piece = x % (kStage / 8), half = x / (kStage / 8) & 1, row = x / (kStage / 4);
            if (p.b0 + row < p.n && p.c * S + 8 * piece < a.inter)
                *reinterpret_cast<u32x4*>(stage + (half * 16 + row) * kStageRow + 8 * piece) = hv[k];
        }
    };
    f32x4 acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    Place at, ahead, next;                         // this stage; the weights' step; the next stage
    enter(at, split);
    ahead = at;
    Step<FMT, 2, CH> s0 = load(ahead), s1;
    advance(ahead, 1);
    fetch(at);
    keep(at, stage0);
    auto step = [&](const Step<FMT, 2, CH>& st, const uint16_t* h0, int c) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (c * S + 128 * i >= a.inter) break;
            bf16x8 ws[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) convert<FMT>(st, t, i, ws[t]);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const bf16x8 hi = *reinterpret_cast<const bf16x8*>(h0 + 128 * i + 8 * s);
                const bf16x8 lo = *reinterpret_cast<const bf16x8*>(h0 + 16 * kStageRow + 128 * i + 8 * s);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[t][s], hi, acc[t], 0, 0, 0);
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[t][s], lo, acc[t], 0, 0, 0);
                }
            }
        }
    };
    auto one_stage = [&](const uint16_t* now, uint16_t* other) {
        // this stage's h is in LDS, and no wave reads the other buffer any more
        __syncthreads();
        next = at;
        advance(next, kSteps);
        if (next.ai < act) fetch(next);
        const int rows = min(16, at.n - at.b0), r = min(r16, rows - 1);
        const uint16_t* h0 = now + r * kStageRow + 32 * g;
        // s0 is the stage's first step, and the next stage's afterwards
#pragma unroll
        for (int k = 0; k < kSteps; k += 2) {
            if (at.c + k >= steps) break;
            if (ahead.ai < act) {
                s1 = load(ahead);
                advance(ahead, 1);
            }
            step(s0, h0 + k * S, at.c + k);
            if (at.c + k + 1 >= steps) {
                s0 = s1;
                break;
            }
            if (ahead.ai < act) {
                s0 = load(ahead);
                advance(ahead, 1);
            }
            step(s1, h0 + (k + 1) * S, at.c + k + 1);
        }
        if (at.c + kSteps >= steps) {              // the 16 entries' last stage
            const int e = order[at.begin + at.b0 + r];
            float f = 0.0f;                        // of the equal entries of the token
            for (int k = e / a.topk * a.topk; k < (e / a.topk + 1) * a.topk; ++k)
                if (ids[k] == at.expert) f += a.weights[k];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (mine && r16 < rows)
                    *reinterpret_cast<f32x4*>(a.part + (int64_t)e * a.hidden + col0 + 16 * t + 4 * g) =
                        acc[t] * f;
                acc[t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
            }
        }
        if (next.ai < act) keep(next, other);
        at = next;
    };
    while (true) {
        one_stage(stage0, stage1);
        if (at.ai >= act) break;
        one_stage(stage1, stage0);
        if (at.ai >= act) break;
    }
}

// y of one token and 1024 columns: the sum of its entries' parts.
__global__ void __launch_bounds__(256) moe_sum_kernel(const MoeArgs a) {
    const int t = (int)blockIdx.y, col = 4 * (256 * (int)blockIdx.x + (int)threadIdx.x);
    const int lane = (int)threadIdx.x & 63;
    // lane j: whether entry j of the token counts
    int id = -1;
    if (lane < a.topk) {
        id = a.ids[t * a.topk + lane];
        if (id >= a.experts || a.weights[t * a.topk + lane] == 0.0f) id = -1;
    }
    bool again = false;
    for (int j = 0; j < a.topk; ++j) {
        const int other = __shfl(id, j);           // by every lane
        again |= j < lane && other == id;
    }
    uint64_t m = __ballot(id >= 0 && !again);
    if (col >= a.hidden) return;
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    for (; m; m &= m - 1)
        y += *reinterpret_cast<const f32x4*>(
            a.part + (int64_t)(t * a.topk + __ffsll((unsigned long long)m) - 1) * a.hidden + col);
    const bf16x2 p = {(__bf16)y[0], (__bf16)y[1]}, q = {(__bf16)y[2], (__bf16)y[3]};
    *reinterpret_cast<u32x2*>(a.y + t * a.ldy + col) =
        (u32x2){__builtin_bit_cast(uint32_t, p), __builtin_bit_cast(uint32_t, q)};
}

template <int FMT, int NB, int G>
void launch_up(const MoeArgs& a, bool few, bool routed, hipStream_t stream) {
    const int tiles = a.inter / (16 * G), entries = a.tokens * a.topk;
    const dim3 by_entry((uint32_t)(entries * tiles)), by_expert((uint32_t)(a.experts * tiles));
    const dim3 block(kUpThreads);
    // two blocks of entries: more entries than experts by far
    if (NB == 2 || (!few && entries > a.experts)) {
        hipLaunchKernelGGL((moe_up_kernel<FMT, NB, G, kExpert>), by_expert, block, 0, stream, a, tiles);
    } else if constexpr (NB == 1) {
        if (few && !routed)
            hipLaunchKernelGGL((moe_up_kernel<FMT, 1, G, kRoute>), by_entry, block, 0, stream, a, tiles);
        else if (few)
            hipLaunchKernelGGL((moe_up_kernel<FMT, 1, G, kFew>), by_entry, block, 0, stream, a, tiles);
        else
            hipLaunchKernelGGL((moe_up_kernel<FMT, 1, G, kEntry>), by_entry, block, 0, stream, a, tiles);
    }
}

template <int FMT>
hipError_t launch(const MoeArgs& a, hipStream_t stream) {
    const int entries = a.tokens * a.topk, units = std::min(a.experts, entries);
    const bool few = moe_is_few(a.tokens, a.topk);
    bool routed = a.logits == nullptr;
    if (!routed && !(few && a.tokens <= kUpWaves)) {
        hipLaunchKernelGGL(moe_route_kernel, dim3((uint32_t)a.tokens), dim3(64), 0, stream, a);
        routed = true;
    }
    // One block of 16 entries, whose waves are more at a time, unless experts commonly have more:
    // they would read their weights again.  64 tokens, 4096 x 1024 in E4M3: 4 of 64 experts (4 an
    // expert) 158 us and 167 with two, 2 of 8 (16 an expert) 60 and 56.
    const bool narrow = a.tokens <= 16 || entries <= 10 * a.experts;
    // Wide tiles (x read once for twice the weights) where they give workgroups enough, 8 experts a
    // token: of 128 (2048 x 768) 16 tokens (3072 wide tiles) take 68.7 us and 76.1 narrow, 8 (1536)
    // 48.2 and 51.9, 4 (768) 33.6 and 35.0, 2 (384) 24.8 and 23.6; of 256 (7168 x 512) 16 tokens
    // (2048) 149 and 152, 8 (1024) 95.2 and 92.5, 4 (512) 59.1 and 60.4, 1 (128) 29.7 and 24.9.
    if (units * (a.inter / 32) >= 768) {
        if (narrow) launch_up<FMT, 1, 2>(a, few, routed, stream);
        else launch_up<FMT, 2, 2>(a, few, routed, stream);
    } else {
        if (narrow) launch_up<FMT, 1, 1>(a, few, routed, stream);
        else launch_up<FMT, 2, 1>(a, few, routed, stream);
    }
    if (few) {
        hipLaunchKernelGGL(moe_down_few_kernel<FMT>, dim3((uint32_t)(a.hidden / 16)),
                           dim3(kDownThreads), 0, stream, a);
        return hipGetLastError();
    }
    // two workgroups for each of the 256 CUs, or one for each expert
    const int tiles = (a.hidden + kPartCols - 1) / kPartCols;
    const int splits = std::max(1, std::min(units, 512 / tiles));
    hipLaunchKernelGGL(moe_down_part_kernel<FMT>, dim3((uint32_t)(tiles * splits)), dim3(kDownThreads),
                       0, stream, a, tiles, splits);
    hipLaunchKernelGGL(moe_sum_kernel, dim3((uint32_t)((a.hidden + 1023) / 1024), (uint32_t)a.tokens),
                       dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe(int fmt, const MoeArgs& a, hipStream_t stream) {
    return fmt == BSQ_MXFP8 ? launch<BSQ_MXFP8>(a, stream) : launch<BSQ_MXFP4>(a, stream);
}

}  // namespace bsq
