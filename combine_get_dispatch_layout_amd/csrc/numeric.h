// Element types of the router, expert-order and expert-product kernels
// (device code): bf16, fp16 and fp32 values, moved in 16-byte chunks and
// computed in fp32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moedx {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// N values of type S that fill one 16-byte chunk.
template <typename S>
struct Chunk {
    static constexpr int kN = 16 / (int)sizeof(S);
    typedef S vec __attribute__((ext_vector_type(kN)));
};

// The casts round to nearest even and keep NaN.
template <typename S>
__device__ __forceinline__ void chunk_to_f32(u32x4_t c, float (&f)[Chunk<S>::kN]) {
    const typename Chunk<S>::vec v = __builtin_bit_cast(typename Chunk<S>::vec, c);
#pragma unroll
    for (int i = 0; i < Chunk<S>::kN; ++i) f[i] = (float)v[i];
}

template <typename S>
__device__ __forceinline__ u32x4_t chunk_from_f32(const float (&f)[Chunk<S>::kN]) {
    typename Chunk<S>::vec v;
#pragma unroll
    for (int i = 0; i < Chunk<S>::kN; ++i) v[i] = (S)f[i];
    return __builtin_bit_cast(u32x4_t, v);
}

// v, rounded to fp32: the compiler may fold a product into its conversion to
// fp16 (one rounding instead of two), in one kernel and not in another.
__device__ __forceinline__ float in_fp32(float v) {
    asm("" : "+v"(v));
    return v;
}

// Reductions over the 64 lanes of a wave by lane-shifted operands (no LDS
// traffic): rows of 16 first, then across rows; lane 63 holds the result,
// which every lane gets.  The order is fixed.
template <int kCtrl, int kRows>
__device__ __forceinline__ int dpp(int old, int v) {
    return __builtin_amdgcn_update_dpp(old, v, kCtrl, kRows, 0xf, false);
}

#define MOEDX_DPP_STEPS(step) \
    step(0x111, 0xf);         \
    step(0x112, 0xf);         \
    step(0x114, 0xf);         \
    step(0x118, 0xf);         \
    step(0x142, 0xa);         \
    step(0x143, 0xc)

__device__ __forceinline__ float wave_sum(float v) {
#define MOEDX_STEP(c, r) v += __int_as_float(dpp<c, r>(0, __float_as_int(v)))
    MOEDX_DPP_STEPS(MOEDX_STEP);
#undef MOEDX_STEP
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

__device__ __forceinline__ double wave_sum(double v) {
#define MOEDX_STEP(c, r)                                                       \
    {                                                                          \
        const uint64_t b = __builtin_bit_cast(uint64_t, v);                    \
        const uint32_t lo = (uint32_t)dpp<c, r>(0, (int)(uint32_t)b);          \
        const uint32_t hi = (uint32_t)dpp<c, r>(0, (int)(uint32_t)(b >> 32));  \
        v += __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);            \
    }
    MOEDX_DPP_STEPS(MOEDX_STEP);
#undef MOEDX_STEP
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, 63);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define MOEDX_STEP(c, r) v = max(v, (uint32_t)dpp<c, r>((int)v, (int)v))
    MOEDX_DPP_STEPS(MOEDX_STEP);
#undef MOEDX_STEP
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float wave_max(float v) {
#define MOEDX_STEP(c, r) \
    v = fmaxf(v, __int_as_float(dpp<c, r>(__float_as_int(v), __float_as_int(v))))
    MOEDX_DPP_STEPS(MOEDX_STEP);
#undef MOEDX_STEP
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// The sum of v over this lane and those below it.
__device__ __forceinline__ int wave_scan(int v) {
#define MOEDX_STEP(c, r) v += dpp<c, r>(0, v)
    MOEDX_DPP_STEPS(MOEDX_STEP);
#undef MOEDX_STEP
    return v;
}

// v of the lane that kCtrl (a quad permutation or a mirror) names.
template <int kCtrl>
__device__ __forceinline__ double lane_swap(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)dpp<kCtrl, 0xf>(0, (int)(uint32_t)b);
    const uint32_t hi = (uint32_t)dpp<kCtrl, 0xf>(0, (int)(uint32_t)(b >> 32));
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Reductions over the 16 lanes of a row, by rotations: every lane ends with the
// same bits.
#define MOEDX_ROR_STEPS(step) \
    step(0x128);              \
    step(0x124);              \
    step(0x122);              \
    step(0x121)

__device__ __forceinline__ float row_sum(float v) {
#define MOEDX_STEP(c) v += __int_as_float(dpp<c, 0xf>(0, __float_as_int(v)))
    MOEDX_ROR_STEPS(MOEDX_STEP);
#undef MOEDX_STEP
    return v;
}

__device__ __forceinline__ float row_max(float v) {
#define MOEDX_STEP(c) v = fmaxf(v, __int_as_float(dpp<c, 0xf>(0, __float_as_int(v))))
    MOEDX_ROR_STEPS(MOEDX_STEP);
#undef MOEDX_STEP
    return v;
}

__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#define MOEDX_STEP(c) v = max(v, (uint32_t)dpp<c, 0xf>(0, (int)v))
    MOEDX_ROR_STEPS(MOEDX_STEP);
#undef MOEDX_STEP
    return v;
}

__device__ __forceinline__ uint64_t row_max(uint64_t v) {
#define MOEDX_STEP(c)                                                         \
    {                                                                         \
        const uint32_t lo = (uint32_t)dpp<c, 0xf>(0, (int)(uint32_t)v);       \
        const uint32_t hi = (uint32_t)dpp<c, 0xf>(0, (int)(uint32_t)(v >> 32)); \
        const uint64_t o = ((uint64_t)hi << 32) | lo;                         \
        v = o > v ? o : v;                                                    \
    }
    MOEDX_ROR_STEPS(MOEDX_STEP);
#undef MOEDX_STEP
    return v;
}

// The maximum over the wave's lanes, which every lane gets: rows of 16 by
// rotations, then rows and halves by exchanges.  No NaN.
__device__ __forceinline__ double wave_max(double v) {
    const auto join = [&](uint32_t lo, uint32_t hi) {
        const double o = __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
        v = o > v ? o : v;
    };
#define MOEDX_STEP(c)                                                              \
    {                                                                              \
        const uint64_t b = __builtin_bit_cast(uint64_t, v);                        \
        join((uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, c, 0xf, 0xf, true), \
             (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), c, 0xf, 0xf, true)); \
    }
    MOEDX_ROR_STEPS(MOEDX_STEP);
#undef MOEDX_STEP
    uint64_t b = __builtin_bit_cast(uint64_t, v);
    auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
    auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
    v = __builtin_bit_cast(double, ((uint64_t)hi[0] << 32) | lo[0]);
    join(lo[1], hi[1]);
    b = __builtin_bit_cast(uint64_t, v);
    lo = __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false);
    hi = __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
    v = __builtin_bit_cast(double, ((uint64_t)hi[0] << 32) | lo[0]);
    join(lo[1], hi[1]);
    return v;
}

// exp(x) for x <= 0 to about an fp32 rounding: x log2 e as a rounded product
// and its remainder, the hardware's 2^t, and 1 + r ln 2 for the remainder.
// Below the normal range (x < -87.3) the result is 0.
__device__ __forceinline__ float exp_neg(float x) {
    constexpr float kLog2e = 1.44269504088896341f;
    constexpr float kLog2eLow = (float)(1.44269504088896341 - (double)kLog2e);
    x = fmaxf(x, -150.0f);
    const float t = x * kLog2e;
    const float r = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, r * 0.693147180559945f, e);
}

}  // namespace moedx
