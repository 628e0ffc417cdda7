// bsq_wave.h -- reductions over the 64 lanes of a wave, for the kernels of
// bsq_route.hip and bsq_logprobs.hip.  Device code; not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bsq {

// A number's bits in an order of unsigned integers, -0 as 0, and back; 0 is below all numbers.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

template <int CTRL>
__device__ __forceinline__ uint32_t turned(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
// f over the numbers of a row of 16 lanes, in each of them: rotations by 8, 4, 2, 1.
template <class F>
__device__ __forceinline__ uint32_t row_all(uint32_t v, F f) {
    v = f(v, turned<0x128>(v));
    v = f(v, turned<0x124>(v));
    v = f(v, turned<0x122>(v));
    return f(v, turned<0x121>(v));
}
// f over the wave's numbers, in every lane.
template <class F>
__device__ __forceinline__ uint32_t wave_all(uint32_t v, F f) {
    v = row_all(v, f);
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = f(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return f(b[0], b[1]);
}
__device__ __forceinline__ float wave_max(float v) {
    return __uint_as_float(wave_all(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}
__device__ __forceinline__ float wave_sum(float v) {
    return __uint_as_float(wave_all(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
// Whole numbers' maxima are the same scalar in all lanes.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    return __builtin_amdgcn_readfirstlane(wave_all(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; }));
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
    const uint32_t hi = wave_max((uint32_t)(v >> 32));
    return (uint64_t)hi << 32 | wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}

}  // namespace bsq
