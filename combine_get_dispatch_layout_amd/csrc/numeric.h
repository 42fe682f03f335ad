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

// Sum over the 64 lanes of a wave, in a fixed order; every lane gets it.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}

}  // namespace moedx
