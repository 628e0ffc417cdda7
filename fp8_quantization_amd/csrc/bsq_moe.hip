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

#include "bsq.h"
#include "bsq_serving_internal.h"

namespace bsq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// 16-byte loads of a lane's 32 codes
template <int FMT>
constexpr int kPieces = FMT == BSQ_MXFP8 ? 2 : 1;

template <int FMT>
struct Codes {
    u32x4 v[kPieces<FMT>];
};
// A lane's 32 codes of chunk c: `row` points at the row's codes
template <int FMT>
__device__ __forceinline__ Codes<FMT> load_codes(const uint8_t* row, int c, int g) {
    Codes<FMT> r;
    const uint8_t* p = row + (int64_t)c * (64 * kPieces<FMT>) + g * (16 * kPieces<FMT>);
#pragma unroll
    for (int i = 0; i < kPieces<FMT>; ++i)
        r.v[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + 16 * i));
    return r;
}
// 2^(b - 127); 255 is NaN
__device__ __forceinline__ float scale_of(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7FC00000u : b == 0u ? 0x00400000u : b << 23);
}
// Codes 8 s .. 8 s + 7 of the lane's 32, times the scale, as BF16
template <int FMT>
__device__ __forceinline__ bf16x8 step_codes(const Codes<FMT>& c, int s, float scale) {
    bf16x2 p[4];
    if constexpr (FMT == BSQ_MXFP8) {
        const uint32_t a = c.v[s / 2][2 * (s % 2)], b = c.v[s / 2][2 * (s % 2) + 1];
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true);
    } else {
        const uint32_t a = c.v[0][s];
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 0);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 1);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 2);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 3);
    }
    return (bf16x8){p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// ------------------------------------------------------------ routing

// NaN counts as -inf.
__device__ __forceinline__ float logit_of(float x) { return x == x ? x : -INFINITY; }

// One wave: the topk experts of a token, lane j getting the j-th and its
// logit.  Each round takes the largest left, the lowest expert among equals.
__device__ __forceinline__ void wave_topk(const float* logits, int experts, int topk, int& id,
                                          float& value) {
    constexpr int kRegs = kMoeMaxExperts / 64;
    const int lane = (int)threadIdx.x & 63;
    float v[kRegs];
    uint32_t left = 0;                             // bit k: expert 64 k + lane is still there
#pragma unroll
    for (int k = 0; k < kRegs; ++k) {
        v[k] = -INFINITY;
        if (64 * k + lane < experts) {
            v[k] = logit_of(logits[64 * k + lane]);
            left |= 1u << k;
        }
    }
    for (int j = 0; j < topk; ++j) {
        float best = -INFINITY;
        int at = 0x7FFFFFFF;                       // none
#pragma unroll
        for (int k = 0; k < kRegs; ++k)
            if (((left >> k) & 1u) && (at == 0x7FFFFFFF || v[k] > best)) {
                best = v[k];
                at = 64 * k + lane;
            }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const float ov = __shfl_xor(best, off);
            const int oa = __shfl_xor(at, off);
            if (oa != 0x7FFFFFFF && (at == 0x7FFFFFFF || ov > best || (ov == best && oa < at))) {
                best = ov;
                at = oa;
            }
        }
        if (lane == (at & 63)) left &= ~(1u << (at >> 6));
        if (lane == j) {
            id = at;
            value = best;
        }
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
    return v;
}

// One wave: the weights of a token whose experts wave_topk found (lane j: the j-th).
__device__ __forceinline__ float wave_weights(const MoeArgs& a, const float* logits, float v) {
    const int lane = (int)threadIdx.x & 63;
    const float top = __shfl(v, 0);
    // exp(x - top); +inf shares the whole weight among its equals
    auto share = [&](float x) {
        if (x == -INFINITY) return 0.0f;
        return x == top ? 1.0f : __builtin_amdgcn_exp2f((x - top) * 1.44269504088896340736f);
    };
    const float mine = lane < a.topk ? share(v) : 0.0f;
    float sum = mine;
    if (!a.renormalize) {
        sum = 0.0f;
        for (int e = lane; e < a.experts; e += 64) sum += share(logit_of(logits[e]));
    }
    sum = wave_sum(sum);
    return sum > 0.0f ? mine / sum : 0.0f;
}

// Whether entry r of a table of (expert, has a weight) counts: the expert
// exists, the weight is not 0 and no earlier such entry of the token names
// the same expert (the weights of equal entries add up in the first).
// `ids` holds -1 for entries without weight or expert.
__device__ __forceinline__ bool counts(const int16_t* ids, int r, int topk) {
    const int id = ids[r];
    if (id < 0) return false;
    for (int k = r - r % topk; k < r; ++k)
        if (ids[k] == id) return false;
    return true;
}

// ------------------------------------------------------------ gate and up
//
// A workgroup computes 16 columns of h for one expert: the 16 rows of W1 and
// the 16 of W3 that belong to them, over all of `hidden`, its waves taking
// contiguous runs of the 128-element chunks.  Columns past the expert's rows
// repeat its last one; no result of theirs is stored.

constexpr int kUpWaves = 4, kUpThreads = 64 * kUpWaves;

// How a workgroup knows its expert and the expert's rows (entries t * topk + j):
//  kGiven    a workgroup per entry of topk_ids; one whose expert an earlier
//            entry names has nothing to do
//  kFew      the same from logits, for at most kUpWaves tokens: every workgroup
//            routes them itself, a wave each
//  kExperts  from logits, a workgroup per expert: a token is the expert's if
//            fewer than topk others come before it, and that count is its place
//  kAll      from topk_ids, a workgroup per expert (more entries than experts)
enum RowsFrom { kGiven, kFew, kExperts, kAll };

template <int FMT, int NB, RowsFrom FROM>
__global__ void __launch_bounds__(kUpThreads) moe_up_kernel(const MoeArgs a, int tiles) {
    __shared__ int16_t ids[kMoeMaxTokens * kMoeMaxTopk];
    __shared__ uint16_t rows[kMoeMaxTokens];
    __shared__ int n_rows;
    __shared__ f32x4 part[kUpWaves][2][64];
    const int tid = (int)threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int unit = (int)(blockIdx.x / (uint32_t)tiles), tile = (int)(blockIdx.x % (uint32_t)tiles);
    const int entries = a.tokens * a.topk;
    if (tid == 0) n_rows = 0;
    int expert = unit;
    if constexpr (FROM == kFew) {
        if (wave < a.tokens) {
            const float* logits = a.logits + (int64_t)wave * a.experts;
            int id = 0;
            float v = -INFINITY;
            wave_topk(logits, a.experts, a.topk, id, v);
            if (lane < a.topk) ids[wave * a.topk + lane] = (int16_t)(v == -INFINITY ? -1 : id);
            if (blockIdx.x == 0) {
                const float w = wave_weights(a, logits, v);
                if (lane < a.topk) {
                    a.ids[wave * a.topk + lane] = id;
                    a.weights[wave * a.topk + lane] = w;
                }
            }
        }
    } else if constexpr (FROM == kExperts) {
        // the first column tile's workgroups write the tokens' routing too
        if (tile == 0)
            for (int t = unit + a.experts * wave; t < a.tokens; t += a.experts * kUpWaves) {
                const float* logits = a.logits + (int64_t)t * a.experts;
                int id = 0;
                float v = -INFINITY;
                wave_topk(logits, a.experts, a.topk, id, v);
                const float w = wave_weights(a, logits, v);
                if (lane < a.topk) {
                    a.ids[t * a.topk + lane] = id;
                    a.weights[t * a.topk + lane] = w;
                }
            }
    } else {
        for (int r = tid; r < entries; r += kUpThreads) {
            const int id = a.ids[r];
            ids[r] = (int16_t)(id < 0 || id >= a.experts || a.weights[r] == 0.0f ? -1 : id);
        }
    }
    __syncthreads();
    if constexpr (FROM == kExperts) {
        for (int t = wave; t < a.tokens; t += kUpWaves) {
            const float* logits = a.logits + (int64_t)t * a.experts;
            const float x = logit_of(logits[expert]);
            int before = 0;
            for (int e0 = 0; e0 < a.experts; e0 += 64) {
                const int e = e0 + lane;
                const float y = e < a.experts ? logit_of(logits[e]) : -INFINITY;
                before += __popcll(__ballot(y > x || (y == x && e < expert)));
            }
            if (lane == 0 && before < a.topk && x != -INFINITY)
                rows[atomicAdd(&n_rows, 1)] = (uint16_t)(t * a.topk + before);
        }
    } else {
        if constexpr (FROM != kAll) {
            // the first entry that names an expert does its work
            expert = ids[unit];
            bool later = expert < 0;
            for (int r = tid; r < unit; r += kUpThreads) later |= ids[r] == expert;
            if (__syncthreads_or(later)) return;
        }
        for (int r = tid; r < entries; r += kUpThreads)
            if (ids[r] == expert && counts(ids, r, a.topk))
                rows[atomicAdd(&n_rows, 1)] = (uint16_t)r;
    }
    __syncthreads();
    const int n = n_rows;
    if (n == 0) return;

    const int chunks = a.hidden / 128;
    const int c_from = chunks * wave / kUpWaves, c_to = chunks * (wave + 1) / kUpWaves;
    const int64_t row_bytes = (int64_t)chunks * 64 * kPieces<FMT>;
    const int64_t group_bytes = (int64_t)((a.hidden + 511) / 512) * 256;
    const int64_t gate_row = (int64_t)expert * 2 * a.inter + 16 * tile, up_row = gate_row + a.inter;
    const uint8_t* wg = a.w13 + (gate_row + r16) * row_bytes;
    const uint8_t* wu = a.w13 + (up_row + r16) * row_bytes;
    const uint8_t* sg = a.w13_scales + gate_row / 16 * group_bytes + 4 * lane;
    const uint8_t* su = a.w13_scales + up_row / 16 * group_bytes + 4 * lane;
    const uint16_t* xr[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
        xr[b] = a.x + (rows[min(16 * b + r16, n - 1)] / a.topk) * a.ldx + 32 * g;

    f32x4 gate[NB], up[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) gate[b] = up[b] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};

    for (int c = c_from; c < c_to; ++c) {
        const Codes<FMT> cg = load_codes<FMT>(wg, c, g), cu = load_codes<FMT>(wu, c, g);
        const float fg = scale_of(sg[(c / 4) * 256 + (c & 3)]);
        const float fu = scale_of(su[(c / 4) * 256 + (c & 3)]);
        bf16x8 wgs[4], wus[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            wgs[s] = step_codes<FMT>(cg, s, fg);
            wus[s] = step_codes<FMT>(cu, s, fu);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (16 * b >= n) break;
            bf16x8 xs[4];
#pragma unroll
            for (int s = 0; s < 4; ++s)
                xs[s] = *reinterpret_cast<const bf16x8*>(xr[b] + c * 128 + 8 * s);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                gate[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wgs[s], xs[s], gate[b], 0, 0, 0);
                up[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wus[s], xs[s], up[b], 0, 0, 0);
            }
        }
    }
    // the waves' sums in their order; lane l holds columns 4 g .. 4 g + 3 of row l % 16
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if (16 * b >= n) break;
        if (b > 0) __syncthreads();
        part[wave][0][lane] = gate[b];
        part[wave][1][lane] = up[b];
        __syncthreads();
        if (wave == b % kUpWaves && 16 * b + r16 < n) {
            f32x4 G = part[0][0][lane], U = part[0][1][lane];
#pragma unroll
            for (int w = 1; w < kUpWaves; ++w) {
                G += part[w][0][lane];
                U += part[w][1][lane];
            }
            float h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                h[e] = G[e] / (1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * G[e])) * U[e];
            // as the sum of two BF16 numbers, 16 bits in all: with one, its rounding
            // alone made y's error 1.4 to 1.5 times that of rounding y
            bf16x2 hi[2], lo[2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                hi[e / 2][e % 2] = (__bf16)h[e];
                lo[e / 2][e % 2] = (__bf16)(h[e] - (float)hi[e / 2][e % 2]);
            }
            uint16_t* dst = a.h + (int64_t)rows[16 * b + r16] * 2 * a.inter + 16 * tile + 4 * g;
            *reinterpret_cast<u32x2*>(dst) = (u32x2){__builtin_bit_cast(uint32_t, hi[0]),
                                                     __builtin_bit_cast(uint32_t, hi[1])};
            *reinterpret_cast<u32x2*>(dst + a.inter) = (u32x2){__builtin_bit_cast(uint32_t, lo[0]),
                                                               __builtin_bit_cast(uint32_t, lo[1])};
        }
    }
}

// ------------------------------------------------------------ down
//
// A workgroup owns 16 columns of y and walks every expert in use: no partial
// result leaves it.  The (expert, 128-element chunk) pairs, experts
// ascending, are dealt to the waves in contiguous runs; a wave adds an
// expert's part, times the tokens' weights, to sums of its own in LDS, and
// the waves' sums are added in their order at the end.

constexpr int kDownWaves = 8, kDownThreads = 64 * kDownWaves;

template <int FMT, int NB>
__global__ void __launch_bounds__(kDownThreads) moe_down_kernel(const MoeArgs a) {
    extern __shared__ float sums[];                // [kDownWaves][tokens][16]
    __shared__ int16_t ids[kMoeMaxTokens * kMoeMaxTopk];
    __shared__ uint16_t order[kMoeMaxTokens * kMoeMaxTopk];   // entries, by expert
    __shared__ float weight[kMoeMaxTokens * kMoeMaxTopk];
    __shared__ int count[kMoeMaxExperts];
    __shared__ uint16_t first[kMoeMaxExperts];     // an expert's first place in `order`
    __shared__ uint16_t active[kMoeMaxExperts];    // the experts in use, ascending
    __shared__ int n_active, n_entries;
    const int tid = (int)threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int entries = a.tokens * a.topk;
    for (int e = tid; e < a.experts; e += kDownThreads) count[e] = 0;
    for (int k = tid; k < kDownWaves * a.tokens * 16; k += kDownThreads) sums[k] = 0.0f;
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
        int base = 0, act = 0;
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
            if (c > 0) active[act + __popcll(used & ((1ull << lane) - 1))] = (uint16_t)e;
            act += __popcll(used);
            base += __shfl(x, 63);
        }
        if (lane == 0) {
            n_active = act;
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

    const int chunks = a.inter / 128, act = n_active;
    const int64_t row_bytes = (int64_t)chunks * 64 * kPieces<FMT>;
    const int64_t group_bytes = (int64_t)((a.inter + 511) / 512) * 256;
    const int col0 = 16 * (int)blockIdx.x;
    const int items = act * chunks;                // at most 2^20
    int it = (int)((int64_t)items * wave / kDownWaves);
    const int it_end = (int)((int64_t)items * (wave + 1) / kDownWaves);
    float* mine = sums + wave * a.tokens * 16;
    while (it < it_end) {
        const int ai = it / chunks, c_from = it - ai * chunks;
        const int c_to = min(chunks, c_from + it_end - it);
        it += c_to - c_from;
        const int expert = active[ai], begin = first[expert];
        const int n = (ai + 1 < act ? (int)first[active[ai + 1]] : n_entries) - begin;
        const int64_t row0 = (int64_t)expert * a.hidden + col0;
        const uint8_t* w2 = a.w2 + (row0 + r16) * row_bytes;
        const uint8_t* sc = a.w2_scales + row0 / 16 * group_bytes + 4 * lane;
        const uint16_t* hr[NB];
        f32x4 acc[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            acc[b] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
            hr[b] = a.h + (int64_t)order[begin + min(16 * b + r16, n - 1)] * 2 * a.inter + 32 * g;
        }

        for (int c = c_from; c < c_to; ++c) {
            const Codes<FMT> cw = load_codes<FMT>(w2, c, g);
            const float f = scale_of(sc[(c / 4) * 256 + (c & 3)]);
            bf16x8 ws[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) ws[s] = step_codes<FMT>(cw, s, f);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if (16 * b >= n) break;
                bf16x8 hs[4], ls[4];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    hs[s] = *reinterpret_cast<const bf16x8*>(hr[b] + c * 128 + 8 * s);
                    ls[s] = *reinterpret_cast<const bf16x8*>(hr[b] + a.inter + c * 128 + 8 * s);
                }
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[s], hs[s], acc[b], 0, 0, 0);
                    acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ws[s], ls[s], acc[b], 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (16 * b + r16 >= n) continue;
            const int r = order[begin + 16 * b + r16], t = r / a.topk;
            float w = weight[r];                   // and of equal entries after it
            for (int k = r + 1; k < (t + 1) * a.topk; ++k)
                if (ids[k] == ids[r]) w += weight[k];
            f32x4* s = reinterpret_cast<f32x4*>(mine + t * 16 + 4 * g);
            *s = *s + acc[b] * w;
        }
    }
    __syncthreads();
    // token k / 16, column k % 16
    for (int k = tid; k < a.tokens * 16; k += kDownThreads) {
        float y = sums[k];
#pragma unroll
        for (int w = 1; w < kDownWaves; ++w) y += sums[w * a.tokens * 16 + k];
        reinterpret_cast<__bf16*>(a.y)[(k / 16) * a.ldy + col0 + k % 16] = (__bf16)y;
    }
}

template <int FMT, int NB>
hipError_t launch(const MoeArgs& a, hipStream_t stream) {
    const int tiles = a.inter / 16, entries = a.tokens * a.topk;
    const bool few = a.logits && a.tokens <= kUpWaves;
    // a workgroup for each entry or for each expert, whichever are fewer
    const bool by_entry = few || (!a.logits && entries <= a.experts);
    const dim3 grid((uint32_t)((by_entry ? entries : a.experts) * tiles));
    if (few)
        hipLaunchKernelGGL((moe_up_kernel<FMT, NB, kFew>), grid, dim3(kUpThreads), 0, stream, a, tiles);
    else if (a.logits)
        hipLaunchKernelGGL((moe_up_kernel<FMT, NB, kExperts>), grid, dim3(kUpThreads), 0, stream, a,
                           tiles);
    else if (by_entry)
        hipLaunchKernelGGL((moe_up_kernel<FMT, NB, kGiven>), grid, dim3(kUpThreads), 0, stream, a,
                           tiles);
    else
        hipLaunchKernelGGL((moe_up_kernel<FMT, NB, kAll>), grid, dim3(kUpThreads), 0, stream, a, tiles);
    hipLaunchKernelGGL((moe_down_kernel<FMT, NB>), dim3((uint32_t)(a.hidden / 16)),
                       dim3(kDownThreads), (uint32_t)(kDownWaves * a.tokens * 16 * sizeof(float)),
                       stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe(int fmt, const MoeArgs& a, hipStream_t stream) {
    if (a.tokens <= 16)
        return fmt == BSQ_MXFP8 ? launch<BSQ_MXFP8, 1>(a, stream) : launch<BSQ_MXFP4, 1>(a, stream);
    return fmt == BSQ_MXFP8 ? launch<BSQ_MXFP8, 4>(a, stream) : launch<BSQ_MXFP4, 4>(a, stream);
}

}  // namespace bsq
