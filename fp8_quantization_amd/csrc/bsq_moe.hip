// bsq_moe.hip -- gfx950 kernels of the mixture-of-experts layer for a few
// tokens over MX weights (include/bsq_serving.h).
//
// With a few tokens the weights of the chosen experts are nearly all of the
// bytes, each read once and used for a handful of columns, so both kernels
// stream weights from memory straight to registers and feed the matrix cores
// with them as the left operand (16 weight rows), the tokens being the 16
// columns:  mfma_f32_16x16x32_bf16, lane l holding weight row l % 16 and,
// of each 128 elements of the contraction, the 32 elements 32 g .. of group
// g = l / 16.  Those are one MX block: the lane's scale is the byte that the
// BSQ_SCALES_MFMA16 record keeps for it (dword l, byte of the 128-element
// step), and the conversion to BF16 applies it exactly.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

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
// two 128-element chunks of E2M1 codes, one of E4M3.  A step is loaded while
// the one before it is used.
template <int FMT>
constexpr int kStepChunks = FMT == BSQ_MXFP8 ? 1 : 2;

template <int NT>
struct Step {
    u32x4 w[NT][2];                  // E2M1: a chunk each; E4M3: halves of the lane's 32 codes
    uint32_t s[NT];                  // scale bytes of the step's chunks
};

// Where a lane's weights of NT 16-row tiles lie: codes at 16 or 32 bytes times
// its group, scales at its dword.
template <int NT>
struct Rows {
    const uint8_t* w[NT];
    const uint8_t* s[NT];
};

// Step from chunk c (a multiple of kStepChunks; chunks from c to last exist).
template <int FMT, int NT>
__device__ __forceinline__ Step<NT> load_step(const Rows<NT>& p, int c, int last) {
    Step<NT> r;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if constexpr (FMT == BSQ_MXFP8) {
            r.w[t][0] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4*>(p.w[t] + (int64_t)c * 128));
            r.w[t][1] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4*>(p.w[t] + (int64_t)c * 128 + 16));
            r.s[t] = p.s[t][(c >> 2) * 256 + (c & 3)];
        } else {
            r.w[t][0] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4*>(p.w[t] + (int64_t)c * 64));
            r.w[t][1] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4*>(p.w[t] + (int64_t)min(c + 1, last) * 64));
            r.s[t] = *reinterpret_cast<const uint16_t*>(p.s[t] + (c >> 2) * 256 + (c & 3));
        }
    }
    return r;
}

// 2^(b - 127); 255 is NaN
__device__ __forceinline__ float scale_of(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7FC00000u : b == 0u ? 0x00400000u : b << 23);
}

// The lane's 32 codes of tile t and the step's chunk i, times their scale, as BF16: exact
// (a code's few bits times a power of two) wherever the product is a normal number.
template <int FMT, int NT>
__device__ __forceinline__ void convert(const Step<NT>& st, int t, int i, bf16x8 (&o)[4]) {
    const float f = scale_of((st.s[t] >> (8 * i)) & 255u);
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
            const uint32_t a = st.w[t][i][s];
            p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, f, 0);
            p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, f, 1);
            p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, f, 2);
            p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, f, 3);
        }
        o[s] = (bf16x8){p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
    }
}

// Bytes of a row of K codes, and of a 16-row group of scale records.
template <int FMT>
__device__ __forceinline__ int64_t row_bytes(int K) {
    return FMT == BSQ_MXFP8 ? K : K / 2;
}
__device__ __forceinline__ int64_t group_bytes(int K) { return (int64_t)((K + 511) / 512) * 256; }

// Rows row .. row + 15 of codes and scales (row a multiple of 16), for this lane.
template <int FMT>
__device__ __forceinline__ const uint8_t* lane_codes(const uint8_t* codes, int64_t row, int K) {
    const int lane = (int)threadIdx.x & 63;
    return codes + (row + (lane & 15)) * row_bytes<FMT>(K) + (lane >> 4) * (FMT == BSQ_MXFP8 ? 32 : 16);
}
__device__ __forceinline__ const uint8_t* lane_scales(const uint8_t* scales, int64_t row, int K) {
    return scales + row / 16 * group_bytes(K) + 4 * ((int)threadIdx.x & 63);
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
// Up to 64 entries a wave keeps them all in its lanes: no LDS, no barrier.
constexpr int kFewEntries = 64;
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
// Column 16 b + lane % 16's entry: the place of that bit of m, or of the last one.
template <int NB>
__device__ __forceinline__ void columns_of(uint64_t m, int (&row)[NB]) {
    const int c = (int)threadIdx.x & 15;
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

// ------------------------------------------------------------ gate and up
//
// A workgroup computes 16 or 32 columns of h for one expert (G blocks of 16):
// the rows of W1 and those of W3 that belong to them, over all of `hidden`, its
// waves taking contiguous runs of the steps.  Columns past the expert's rows
// repeat its last one; no result of theirs is stored.

constexpr int kUpWaves = 4, kUpThreads = 64 * kUpWaves;

// How a workgroup knows its expert and the expert's entries:
//  kRoute  few entries, from logits, for at most kUpWaves tokens: every workgroup
//          routes them itself, a wave each
//  kFew    few entries, from topk_ids
//  kEntry  a workgroup per entry of topk_ids
//  kExpert a workgroup per expert (more entries than experts)
// Except in the last, a workgroup whose expert an earlier entry names has nothing to do.
enum RowsFrom { kRoute, kFew, kEntry, kExpert };

template <int FMT, int NB, int G, RowsFrom FROM>
__global__ void __launch_bounds__(kUpThreads) moe_up_kernel(const MoeArgs a, int tiles) {
    __shared__ f32x4 part[kUpWaves][2 * G][64];
    const int tid = (int)threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int unit = (int)(blockIdx.x / (uint32_t)tiles), tile = (int)(blockIdx.x % (uint32_t)tiles);
    const int entries = a.tokens * a.topk;
    int expert, n, row[NB];                        // row: the entry of column 16 b + r16
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
        const uint64_t m = entries_of(e, expert);
        if (m & ((1ull << unit) - 1)) return;
        n = __popcll(m);
        columns_of<NB>(m, row);
    } else {
        __shared__ int16_t ids[kMoeMaxTokens * kMoeMaxTopk];
        __shared__ uint16_t rows[kMoeMaxTokens];
        __shared__ int n_rows;
        if (tid == 0) n_rows = 0;
        for (int r = tid; r < entries; r += kUpThreads) {
            const int id = a.ids[r];
            ids[r] = (int16_t)(id < 0 || id >= a.experts || a.weights[r] == 0.0f ? -1 : id);
        }
        __syncthreads();
        expert = unit;
        if constexpr (FROM == kEntry) {
            expert = ids[unit];
            bool later = expert < 0;
            for (int r = tid; r < unit; r += kUpThreads) later |= ids[r] == expert;
            if (__syncthreads_or(later)) return;
        }
        for (int r = tid; r < entries; r += kUpThreads)
            if (ids[r] == expert && counts(ids, r, a.topk))
                rows[atomicAdd(&n_rows, 1)] = (uint16_t)r;
        __syncthreads();
        n = n_rows;
        if (n == 0) return;
#pragma unroll
        for (int b = 0; b < NB; ++b) row[b] = rows[min(16 * b + r16, n - 1)];
    }

    constexpr int CS = kStepChunks<FMT>;
    const int chunks = a.hidden / 128, steps = (chunks + CS - 1) / CS;
    const int c_from = CS * (steps * wave / kUpWaves);
    const int c_to = min(chunks, CS * (steps * (wave + 1) / kUpWaves));
    Rows<2 * G> w;                                 // W1's tiles, then W3's
#pragma unroll
    for (int t = 0; t < 2 * G; ++t) {
        const int64_t row = (int64_t)expert * 2 * a.inter + (t < G ? 0 : a.inter) +
                            16 * (G * tile + t % G);
        w.w[t] = lane_codes<FMT>(a.w13, row, a.hidden);
        w.s[t] = lane_scales(a.w13_scales, row, a.hidden);
    }
    const uint16_t* xr[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
        xr[b] = a.x + (row[b] / a.topk) * a.ldx + 32 * g;

    f32x4 acc[NB][2 * G];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < 2 * G; ++t) acc[b][t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    auto use = [&](const Step<2 * G>& st, int c) {
#pragma unroll
        for (int i = 0; i < CS; ++i) {
            if (c + i >= c_to) break;
            bf16x8 ws[2 * G][4];
#pragma unroll
            for (int t = 0; t < 2 * G; ++t) convert<FMT>(st, t, i, ws[t]);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if (16 * b >= n) break;
                bf16x8 xs[4];
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    xs[s] = *reinterpret_cast<const bf16x8*>(xr[b] + (c + i) * 128 + 8 * s);
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int t = 0; t < 2 * G; ++t)
                        acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[t][s], xs[s],
                                                                            acc[b][t], 0, 0, 0);
            }
        }
    };
    if (c_from < c_to) {
        Step<2 * G> s0 = load_step<FMT>(w, c_from, chunks - 1), s1;
        for (int c = c_from;; c += 2 * CS) {
            // past the wave's last step its loads repeat that step
            s1 = load_step<FMT>(w, c + CS < c_to ? c + CS : c, chunks - 1);
            use(s0, c);
            if (c + CS >= c_to) break;
            s0 = load_step<FMT>(w, c + 2 * CS < c_to ? c + 2 * CS : c, chunks - 1);
            use(s1, c + CS);
            if (c + 2 * CS >= c_to) break;
        }
    }
    // the waves' sums in their order; lane l holds columns 4 g .. 4 g + 3 of row l % 16
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if (16 * b >= n) break;
        if (b > 0) __syncthreads();
#pragma unroll
        for (int t = 0; t < 2 * G; ++t) part[wave][t][lane] = acc[b][t];
        __syncthreads();
        if (wave >= G || 16 * b + r16 >= n) continue;
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
            const float h = gate[e] /
                            (1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * gate[e])) * up[e];
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

// ------------------------------------------------------------ down
//
// A workgroup owns 16 or 32 columns of y (NT blocks of 16) and walks every
// expert in use: no partial result leaves it.  The (expert, step) pairs,
// experts ascending, are dealt to the waves in contiguous runs; a wave adds an
// expert's part, times the tokens' weights, to sums of its own in LDS, and
// the waves' sums are added in their order at the end.

constexpr int kDownWaves = 8, kDownThreads = 64 * kDownWaves;

// FEW: the entries are in every wave's lanes, the experts in the order of their first
// entries; else in LDS, sorted by expert.
template <int FMT, int NB, int NT, bool FEW>
__global__ void __launch_bounds__(kDownThreads) moe_down_kernel(const MoeArgs a) {
    constexpr int kEntries = FEW ? 1 : kMoeMaxTokens * kMoeMaxTopk, kExperts = FEW ? 1 : kMoeMaxExperts;
    extern __shared__ float sums[];                // [kDownWaves][tokens][16 NT]
    __shared__ int16_t ids[kEntries];
    __shared__ uint16_t order[kEntries];           // entries, by expert
    __shared__ float weight[kEntries];
    __shared__ int count[kExperts];
    __shared__ uint16_t first[kExperts];           // an expert's first place in `order`
    __shared__ uint16_t active[kExperts];          // the experts in use, ascending
    __shared__ int n_active, n_entries;
    const int tid = (int)threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int entries = a.tokens * a.topk;
    float* mine = sums + wave * a.tokens * 16 * NT;
    for (int k = lane; k < a.tokens * 16 * NT; k += 64) mine[k] = 0.0f;
    FewEntries few{};
    uint64_t firsts = 0;                           // the first entry of each expert
    int act;
    if constexpr (FEW) {
        few = few_entries(a, lane < entries ? a.ids[lane] : -1, lane < entries ? a.weights[lane] : 0.0f);
        for (uint64_t m = few.counted; m;) {
            const int at = __ffsll((unsigned long long)m) - 1;
            firsts |= 1ull << at;
            m &= ~entries_of(few, expert_at(few, at));
        }
        act = __popcll(firsts);
    } else {
        for (int e = tid; e < a.experts; e += kDownThreads) count[e] = 0;
        for (int r = tid; r < entries; r += kDownThreads) {
            const int id = a.ids[r];
            const float w = a.weights[r];
            ids[r] = (int16_t)(id < 0 || id >= a.experts || w == 0.0f ? -1 : id);
            weight[r] = w;
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
        act = n_active;
    }
    // the ai-th expert in use
    auto expert_in_use = [&](int ai) {
        if constexpr (FEW) {
            uint64_t m = firsts;
            for (int i = 0; i < ai; ++i) m &= m - 1;
            return expert_at(few, __ffsll((unsigned long long)m) - 1);
        } else {
            return (int)active[ai];
        }
    };

    constexpr int CS = kStepChunks<FMT>;
    const int chunks = a.inter / 128, steps = (chunks + CS - 1) / CS;
    const int col0 = 16 * NT * (int)blockIdx.x;
    const int items = act * steps;                 // at most 2^20
    const int it_from = (int)((int64_t)items * wave / kDownWaves);
    const int it_to = (int)((int64_t)items * (wave + 1) / kDownWaves);
    f32x4 acc[NB][NT];
    auto clear = [&]() {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[b][t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    };
    auto load = [&](int it) {
        const int ai = it / steps, c = CS * (it - ai * steps), expert = expert_in_use(ai);
        Rows<NT> w;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int64_t row = (int64_t)expert * a.hidden + col0 + 16 * t;
            w.w[t] = lane_codes<FMT>(a.w2, row, a.inter);
            w.s[t] = lane_scales(a.w2_scales, row, a.inter);
        }
        return load_step<FMT>(w, c, chunks - 1);
    };
    auto use = [&](const Step<NT>& st, int it) {
        const int ai = it / steps, c = CS * (it - ai * steps);
        int n, row[NB];                            // the expert's entries, that of column 16 b + r16
        if constexpr (FEW) {
            const uint64_t m = entries_of(few, expert_in_use(ai));
            n = __popcll(m);
            columns_of<NB>(m, row);
        } else {
            const int begin = first[active[ai]];
            n = (ai + 1 < act ? (int)first[active[ai + 1]] : n_entries) - begin;
#pragma unroll
            for (int b = 0; b < NB; ++b) row[b] = order[begin + min(16 * b + r16, n - 1)];
        }
#pragma unroll
        for (int i = 0; i < CS; ++i) {
            if (c + i >= chunks) break;
            bf16x8 ws[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) convert<FMT>(st, t, i, ws[t]);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if (16 * b >= n) break;
                const uint16_t* h = a.h + (int64_t)row[b] * 2 * a.inter + 32 * g + (c + i) * 128;
                bf16x8 hi[4], lo[4];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    hi[s] = *reinterpret_cast<const bf16x8*>(h + 8 * s);
                    lo[s] = *reinterpret_cast<const bf16x8*>(h + a.inter + 8 * s);
                }
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[t][s], hi[s],
                                                                            acc[b][t], 0, 0, 0);
                        acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[t][s], lo[s],
                                                                            acc[b][t], 0, 0, 0);
                    }
            }
        }
        // the expert's (or the wave's) last step: its part goes to the tokens' sums
        if (it + 1 < it_to && it + 1 < (ai + 1) * steps) return;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int r = row[b], t = r / a.topk;
            float f;
            if constexpr (FEW) {
                f = __shfl(few.w, r);
            } else {
                f = weight[r];                     // and of equal entries after it
                for (int k = r + 1; k < (t + 1) * a.topk; ++k)
                    if (ids[k] == ids[r]) f += weight[k];
            }
            if (16 * b + r16 >= n) continue;
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                f32x4* s = reinterpret_cast<f32x4*>(mine + t * 16 * NT + 16 * u + 4 * g);
                *s = *s + acc[b][u] * f;
            }
        }
        clear();
    };
    clear();
    if (it_from < it_to) {
        Step<NT> s0 = load(it_from), s1;
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
    for (int k = tid; k < a.tokens * 16 * NT; k += kDownThreads) {
        float y = sums[k];
#pragma unroll
        for (int w = 1; w < kDownWaves; ++w) y += sums[w * a.tokens * 16 * NT + k];
        reinterpret_cast<__bf16*>(a.y)[k / (16 * NT) * a.ldy + col0 + k % (16 * NT)] = (__bf16)y;
    }
}

template <int FMT, int NB, int G>
void launch_up(const MoeArgs& a, bool few, bool routed, hipStream_t stream) {
    const int tiles = a.inter / (16 * G), entries = a.tokens * a.topk;
    const dim3 grid((uint32_t)(std::min(entries, a.experts) * tiles)), block(kUpThreads);
    const dim3 by_entry((uint32_t)(entries * tiles));
    if (few && !routed)
        hipLaunchKernelGGL((moe_up_kernel<FMT, NB, G, kRoute>), by_entry, block, 0, stream, a, tiles);
    else if (few)
        hipLaunchKernelGGL((moe_up_kernel<FMT, NB, G, kFew>), by_entry, block, 0, stream, a, tiles);
    else if (entries <= a.experts)
        hipLaunchKernelGGL((moe_up_kernel<FMT, NB, G, kEntry>), grid, block, 0, stream, a, tiles);
    else
        hipLaunchKernelGGL((moe_up_kernel<FMT, NB, G, kExpert>), grid, block, 0, stream, a, tiles);
}

template <int FMT, int NB, int NT>
void launch_down(const MoeArgs& a, bool few, hipStream_t stream) {
    const dim3 grid((uint32_t)(a.hidden / (16 * NT))), block(kDownThreads);
    const uint32_t lds = (uint32_t)(kDownWaves * a.tokens * 16 * NT * sizeof(float));
    if (few) hipLaunchKernelGGL((moe_down_kernel<FMT, NB, NT, true>), grid, block, lds, stream, a);
    else hipLaunchKernelGGL((moe_down_kernel<FMT, NB, NT, false>), grid, block, lds, stream, a);
}

template <int FMT, int NB>
hipError_t launch(const MoeArgs& a, hipStream_t stream) {
    const bool few = a.tokens * a.topk <= kFewEntries;
    bool routed = a.logits == nullptr;
    if (!routed && !(few && a.tokens <= kUpWaves)) {
        hipLaunchKernelGGL(moe_route_kernel, dim3((uint32_t)a.tokens), dim3(64), 0, stream, a);
        routed = true;
    }
    // wide tiles where there are workgroups enough for every CU
    const int units = std::min(a.experts, a.tokens * a.topk);
    if (units * (a.inter / 32) >= 1024) launch_up<FMT, NB, 2>(a, few, routed, stream);
    else launch_up<FMT, NB, 1>(a, few, routed, stream);
    if (NB == 1 && a.hidden >= 32 * 192) launch_down<FMT, NB, NB == 1 ? 2 : 1>(a, few, stream);
    else launch_down<FMT, NB, 1>(a, few, stream);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe(int fmt, const MoeArgs& a, hipStream_t stream) {
    if (a.tokens <= 16)
        return fmt == BSQ_MXFP8 ? launch<BSQ_MXFP8, 1>(a, stream) : launch<BSQ_MXFP4, 1>(a, stream);
    return fmt == BSQ_MXFP8 ? launch<BSQ_MXFP8, 4>(a, stream) : launch<BSQ_MXFP4, 4>(a, stream);
}

}  // namespace bsq
