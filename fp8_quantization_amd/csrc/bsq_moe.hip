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

// A wave takes weights in steps of 128 bytes of each row, whole cache lines:
// 256 elements of E2M1, 128 of E4M3, lane group g the 32 bytes at 32 g (64 or
// 32 elements: two or one MX blocks).  A step is loaded while the one before it
// is used.  (Lanes that took 16 bytes of each half line streamed at 4.4 TB/s
// where these do at 6.)
template <int FMT>
constexpr int kStep = FMT == BSQ_MXFP8 ? 128 : 256;      // elements of a step
template <int FMT>
constexpr int kHalves = kStep<FMT> / 128;                // MX blocks of a lane in a step

template <int NT>
struct Step {
    u32x4 w[NT][2];
    uint32_t s[NT][2];               // scale byte of each block
};

// Where a lane's weights of NT 16-row tiles lie: its codes of step 0, and the scale of its
// first block (the second's is 64 bytes on).
template <int NT>
struct Rows {
    const uint8_t* w[NT];
    const uint8_t* s[NT];
};
__device__ __forceinline__ int64_t group_bytes(int K) { return (int64_t)((K + 511) / 512) * 256; }

// Rows row .. row + 15 (row a multiple of 16) of codes and scale records of K elements a row.
template <int FMT, int NT>
__device__ __forceinline__ void set_rows(Rows<NT>& p, int t, const uint8_t* codes,
                                         const uint8_t* scales, int64_t row, int K) {
    const int lane = (int)threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    p.w[t] = codes + (row + r) * (FMT == BSQ_MXFP8 ? K : K / 2) + 32 * g;
    // block kb of a row has byte kb / 4 of dword row + 16 (kb % 4) in a record of 16 blocks
    p.s[t] = scales + row / 16 * group_bytes(K) +
             (FMT == BSQ_MXFP8 ? 4 * lane : 4 * (r + 16 * (2 * g & 3)) + (g >> 1));
}

// Step c.  An odd number of 128-element chunks leaves the last E2M1 step half full: its
// lane groups 2 and 3 get zeros.
template <int FMT, int NT>
__device__ __forceinline__ Step<NT> load_step(const Rows<NT>& p, int c, int K) {
    const bool out = FMT != BSQ_MXFP8 && (c + 1) * 256 > K && ((int)threadIdx.x & 32);
    Step<NT> r;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const u32x4* w = reinterpret_cast<const u32x4*>(p.w[t] + (int64_t)c * 128 - (out ? 64 : 0));
        r.w[t][0] = __builtin_nontemporal_load(w);
        r.w[t][1] = __builtin_nontemporal_load(w + 1);
        if constexpr (FMT == BSQ_MXFP8) {
            r.s[t][0] = p.s[t][(c >> 2) * 256 + (c & 3)];
        } else {
            const uint8_t* s = p.s[t] + (c >> 1) * 256 + 2 * (c & 1);
            r.s[t][0] = s[0];
            r.s[t][1] = s[64];
        }
    }
    if constexpr (FMT != BSQ_MXFP8) {
        if ((c + 1) * 256 > K) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    r.w[t][h] = out ? (u32x4){0, 0, 0, 0} : r.w[t][h];
                    r.s[t][h] = out ? 127u : r.s[t][h];
                }
        }
    }
    return r;
}

// 2^(b - 127); 255 is NaN
__device__ __forceinline__ float scale_of(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7FC00000u : b == 0u ? 0x00400000u : b << 23);
}

// The lane's 32 codes of tile t and block h, times their scale, as BF16: exact (a code's few
// bits times a power of two) wherever the product is a normal number.
template <int FMT, int NT>
__device__ __forceinline__ void convert(const Step<NT>& st, int t, int h, bf16x8 (&o)[4]) {
    const float f = scale_of(st.s[t][h]);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        bf16x2 p[4];
        if constexpr (FMT == BSQ_MXFP8) {
            const uint32_t a = st.w[t][s / 2][2 * (s % 2)], b = st.w[t][s / 2][2 * (s % 2) + 1];
            p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, f, false);
            p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, f, true);
            p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, f, false);
            p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, f, true);
        } else {
            const uint32_t a = st.w[t][h][s];
            p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, f, 0);
            p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, f, 1);
            p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, f, 2);
            p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, f, 3);
        }
        o[s] = (bf16x8){p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
    }
}

// Steps [c_from, c_to) of a wave: use(step, c) with the next one's loads in flight.
template <int FMT, int NT, class F>
__device__ __forceinline__ void for_steps(const Rows<NT>& w, int c_from, int c_to, int K, F use) {
    if (c_from >= c_to) return;
    Step<NT> s0 = load_step<FMT>(w, c_from, K), s1;
    for (int c = c_from;; c += 2) {
        // past the last step its loads repeat it
        s1 = load_step<FMT>(w, min(c + 1, c_to - 1), K);
        use(s0, c);
        if (c + 1 >= c_to) break;
        s0 = load_step<FMT>(w, min(c + 2, c_to - 1), K);
        use(s1, c + 1);
        if (c + 2 >= c_to) break;
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
__device__ __forceinline__ FewEntries few_entries(const MoeArgs& a, int id, float w) {
    const int lane = (int)threadIdx.x & 63;
    FewEntries r;
    const bool valid = lane < a.tokens * a.topk && id >= 0 && id < a.experts && w != 0.0f;
    r.id = valid ? id : -1;
    r.w = w;
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
//          routes them itself, a wave each
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
// stored.

constexpr int kUpWaves = 4, kUpThreads = 64 * kUpWaves;

template <int FMT, int NB, int G, RowsFrom FROM>
__global__ void __launch_bounds__(kUpThreads, 2) moe_up_kernel(const MoeArgs a, int tiles) {
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
        const FewEntries e = few_entries(a, id, w);
        if (!((e.counted >> unit) & 1u)) return;
        expert = expert_at(e, unit);
        few = entries_of(e, expert);
        if (few & ((1ull << unit) - 1)) return;
        n = __popcll(few);
    } else {
        n = many_entries<FROM, kUpThreads>(a, many, unit, expert);
        if (n == 0) return;
    }

    constexpr int E = kStep<FMT> / 4;              // elements of a lane in a step
    const int steps = (a.hidden + kStep<FMT> - 1) / kStep<FMT>;
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
            xr[b] = a.x + (row[b] / a.topk) * a.ldx + E * g;
#pragma unroll
            for (int t = 0; t < 2 * G; ++t) acc[b][t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        }
        for_steps<FMT>(w, c_from, c_to, a.hidden, [&](const Step<2 * G>& st, int c) {
            // lanes past the end of a row (whose weights are 0) read what lies before it
            const bool out = c * kStep<FMT> + E * g >= a.hidden;
            const int at = c * kStep<FMT> - (out ? 128 : 0);
#pragma unroll
            for (int h = 0; h < kHalves<FMT>; ++h) {
                bf16x8 ws[2 * G][4];
#pragma unroll
                for (int t = 0; t < 2 * G; ++t) convert<FMT>(st, t, h, ws[t]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if (b > 0 && b0 + 16 * b >= n) break;
                    bf16x8 xs[4];
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        xs[s] = *reinterpret_cast<const bf16x8*>(xr[b] + at + 32 * h + 8 * s);
                        if constexpr (FMT != BSQ_MXFP8)
                            if ((c + 1) * 256 > a.hidden && out) xs[s] = (bf16x8){};
                    }
#pragma unroll
                    for (int s = 0; s < 4; ++s)
#pragma unroll
                        for (int t = 0; t < 2 * G; ++t)
                            acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[t][s], xs[s],
                                                                                acc[b][t], 0, 0, 0);
                }
            }
        });
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
            // alone made y's error 1.4 to 1.5 times that of rounding y
            bf16x2 hi[2], lo[2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float h =
                    gate[e] / (1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * gate[e])) * up[e];
                hi[e / 2][e % 2] = (__bf16)h;
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
    constexpr int E = kStep<FMT> / 4;
    __shared__ float sums[kDownWaves][16 * 16];    // [token][column]
    const int tid = (int)threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int entries = a.tokens * a.topk;
    for (int k = lane; k < 16 * 16; k += 64) sums[wave][k] = 0.0f;
    const FewEntries few =
        few_entries(a, lane < entries ? a.ids[lane] : -1, lane < entries ? a.weights[lane] : 0.0f);
    uint64_t firsts = 0;                           // the first entry of each expert
    for (uint64_t m = few.counted; m;) {
        const int at = __ffsll((unsigned long long)m) - 1;
        firsts |= 1ull << at;
        m &= ~entries_of(few, expert_at(few, at));
    }
    const int act = __popcll(firsts), steps = (a.inter + kStep<FMT> - 1) / kStep<FMT>;
    const int col0 = 16 * (int)blockIdx.x;
    const int items = act * steps;
    const int it_from = items * wave / kDownWaves, it_to = items * (wave + 1) / kDownWaves;
    auto expert_in_use = [&](int ai) {             // the ai-th
        uint64_t m = firsts;
        for (int i = 0; i < ai; ++i) m &= m - 1;
        return expert_at(few, __ffsll((unsigned long long)m) - 1);
    };
    auto load = [&](int it) {
        const int ai = it / steps;
        Rows<1> w;
        set_rows<FMT>(w, 0, a.w2, a.w2_scales, (int64_t)expert_in_use(ai) * a.hidden + col0, a.inter);
        return load_step<FMT>(w, it - ai * steps, a.inter);
    };
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    auto use = [&](const Step<1>& st, int it) {
        const int ai = it / steps, c = it - ai * steps;
        const uint64_t m = entries_of(few, expert_in_use(ai));
        int row[1];
        columns_of<1>(m, 0, row);
        const bool out = c * kStep<FMT> + E * g >= a.inter;
        const uint16_t* h0 = a.h + (int64_t)row[0] * 2 * a.inter + c * kStep<FMT> + E * g - (out ? 128 : 0);
#pragma unroll
        for (int h = 0; h < kHalves<FMT>; ++h) {
            bf16x8 ws[4], hi[4], lo[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                hi[s] = *reinterpret_cast<const bf16x8*>(h0 + 32 * h + 8 * s);
                lo[s] = *reinterpret_cast<const bf16x8*>(h0 + a.inter + 32 * h + 8 * s);
                if constexpr (FMT != BSQ_MXFP8)
                    if ((c + 1) * 256 > a.inter && out) hi[s] = lo[s] = (bf16x8){};
            }
            convert<FMT>(st, 0, h, ws);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[s], hi[s], acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[s], lo[s], acc, 0, 0, 0);
            }
        }
        // the expert's (or the wave's) last step: its part goes to the tokens' sums
        if (it + 1 < it_to && it + 1 < (ai + 1) * steps) return;
        const float f = __shfl(few.w, row[0]);
        if (r16 < __popcll(m)) {
            f32x4* s = reinterpret_cast<f32x4*>(&sums[wave][row[0] / a.topk * 16 + 4 * g]);
            *s = *s + acc * f;
        }
        acc = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    };
    if (it_from < it_to) {
        Step<1> s0 = load(it_from), s1;
        for (int it = it_from;; it += 2) {
            // past the wave's last item its loads repeat that item's
            s1 = load(min(it + 1, it_to - 1));
            use(s0, it);
            if (it + 1 >= it_to) break;
            s0 = load(min(it + 2, it_to - 1));
            use(s1, it + 1);
            if (it + 2 >= it_to) break;
        }
    }
    __syncthreads();
    for (int k = tid; k < a.tokens * 16; k += kDownThreads) {
        float y = sums[0][k];
#pragma unroll
        for (int w = 1; w < kDownWaves; ++w) y += sums[w][k];
        reinterpret_cast<__bf16*>(a.y)[k / 16 * a.ldy + col0 + k % 16] = (__bf16)y;
    }
}

// ------------------------------------------------------------ down, many entries
//
// A workgroup computes 256 columns of one expert's part, 32 a wave, for 16
// entries at a time, whose h the waves share: it lies in LDS, 512 elements at a
// time (read from memory by each wave for its 32 columns it was four times the
// weights' loads, and half of the kernel's time).  The parts, times the
// tokens' weights, go to memory in 32 bits, one row an entry, and a third
// kernel adds a token's rows in their order.

constexpr int kStage = 512;          // elements of h in LDS
// 16 bytes apart from a multiple of the banks' 256: 16 rows' pieces fall in different banks
constexpr int kStageRow = kStage + 8;
constexpr int kPartCols = 32 * kDownWaves;

template <int FMT, RowsFrom FROM>
__global__ void __launch_bounds__(kDownThreads, 2) moe_down_part_kernel(const MoeArgs a, int tiles) {
    constexpr int E = kStep<FMT> / 4, kSteps = kStage / kStep<FMT>;
    __shared__ ManyEntries many;
    __shared__ __attribute__((aligned(16))) uint16_t stage[2][16][kStageRow];
    const int tid = (int)threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int unit = (int)(blockIdx.x / (uint32_t)tiles), tile = (int)(blockIdx.x % (uint32_t)tiles);
    int expert;
    const int n = many_entries<FROM, kDownThreads>(a, many, unit, expert);
    if (n == 0) return;
    const int col0 = kPartCols * tile + 32 * wave;
    const bool mine = col0 < a.hidden;             // hidden is a multiple of 128
    const int steps = (a.inter + kStep<FMT> - 1) / kStep<FMT>;
    Rows<2> w;
#pragma unroll
    for (int t = 0; t < 2; ++t)
        set_rows<FMT>(w, t, a.w2, a.w2_scales,
                      (int64_t)expert * a.hidden + (mine ? col0 : 0) + 16 * t, a.inter);
    for (int b0 = 0; b0 < n; b0 += 16) {
        const int rows = min(16, n - b0), r = min(r16, rows - 1);
        f32x4 acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
        Step<2> s0 = load_step<FMT>(w, 0, a.inter), s1;
        auto use = [&](const Step<2>& st, int c) {
            const uint16_t* h0 = &stage[0][r][c % kSteps * kStep<FMT> + E * g];
#pragma unroll
            for (int h = 0; h < kHalves<FMT>; ++h) {
                bf16x8 ws[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t) convert<FMT>(st, t, h, ws[t]);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const bf16x8 hi = *reinterpret_cast<const bf16x8*>(h0 + 32 * h + 8 * s);
                    const bf16x8 lo =
                        *reinterpret_cast<const bf16x8*>(h0 + 16 * kStageRow + 32 * h + 8 * s);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[t][s], hi, acc[t], 0, 0, 0);
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[t][s], lo, acc[t], 0, 0, 0);
                    }
                }
            }
        };
        for (int c0 = 0; c0 < steps; c0 += kSteps) {
            // the entries' next 512 elements of both numbers of h, zeros past the end
            __syncthreads();
            for (int k = tid; k < rows * 2 * (kStage / 8); k += kDownThreads) {
                const int piece = k % (kStage / 8), half = k / (kStage / 8) & 1, row = k / (kStage / 4);
                const int at = c0 * kStep<FMT> + 8 * piece;
                u32x4 v = {0, 0, 0, 0};
                if (at < a.inter)
                    v = *reinterpret_cast<const u32x4*>(
                        a.h + ((int64_t)many.rows[b0 + row] * 2 + half) * a.inter + at);
                *reinterpret_cast<u32x4*>(&stage[half][row][8 * piece]) = v;
            }
            __syncthreads();
            // two steps at a time, the next one's loads in flight
#pragma unroll
            for (int k = 0; k < kSteps; k += 2) {
                const int c = c0 + k;
                if (c >= steps) break;
                s1 = load_step<FMT>(w, min(c + 1, steps - 1), a.inter);
                use(s0, c);
                if (c + 1 >= steps) break;
                s0 = load_step<FMT>(w, min(c + 2, steps - 1), a.inter);
                use(s1, c + 1);
            }
        }
        if (!mine || r16 >= rows) continue;
        const int e = many.rows[b0 + r16], t0 = e / a.topk * a.topk;
        float f = 0.0f;                            // of the equal entries of the token
        for (int k = t0; k < t0 + a.topk; ++k)
            if (many.ids[k] == expert) f += a.weights[k];
#pragma unroll
        for (int t = 0; t < 2; ++t)
            *reinterpret_cast<f32x4*>(a.part + (int64_t)e * a.hidden + col0 + 16 * t + 4 * g) = acc[t] * f;
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
    if (few && !routed)
        hipLaunchKernelGGL((moe_up_kernel<FMT, NB, G, kRoute>), by_entry, block, 0, stream, a, tiles);
    else if (few)
        hipLaunchKernelGGL((moe_up_kernel<FMT, NB, G, kFew>), by_entry, block, 0, stream, a, tiles);
    else if (entries <= a.experts)
        hipLaunchKernelGGL((moe_up_kernel<FMT, NB, G, kEntry>), by_entry, block, 0, stream, a, tiles);
    else
        hipLaunchKernelGGL((moe_up_kernel<FMT, NB, G, kExpert>), by_expert, block, 0, stream, a, tiles);
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
    // wide tiles where there are workgroups enough for every CU
    if (units * (a.inter / 32) >= 1024) {
        if (a.tokens <= 16) launch_up<FMT, 1, 2>(a, few, routed, stream);
        else launch_up<FMT, 2, 2>(a, few, routed, stream);
    } else {
        if (a.tokens <= 16) launch_up<FMT, 1, 1>(a, few, routed, stream);
        else launch_up<FMT, 2, 1>(a, few, routed, stream);
    }
    if (few) {
        hipLaunchKernelGGL(moe_down_few_kernel<FMT>, dim3((uint32_t)(a.hidden / 16)),
                           dim3(kDownThreads), 0, stream, a);
        return hipGetLastError();
    }
    const int tiles = (a.hidden + kPartCols - 1) / kPartCols;
    const dim3 grid((uint32_t)(units * tiles));
    if (entries <= a.experts)
        hipLaunchKernelGGL((moe_down_part_kernel<FMT, kEntry>), grid, dim3(kDownThreads), 0, stream, a,
                           tiles);
    else
        hipLaunchKernelGGL((moe_down_part_kernel<FMT, kExpert>), grid, dim3(kDownThreads), 0, stream, a,
                           tiles);
    hipLaunchKernelGGL(moe_sum_kernel, dim3((uint32_t)((a.hidden + 1023) / 1024), (uint32_t)a.tokens),
                       dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe(int fmt, const MoeArgs& a, hipStream_t stream) {
    return fmt == BSQ_MXFP8 ? launch<BSQ_MXFP8>(a, stream) : launch<BSQ_MXFP4>(a, stream);
}

}  // namespace bsq
