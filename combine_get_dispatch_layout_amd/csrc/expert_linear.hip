// The experts' products for gfx950: y = x w[e]^T over the rows of each expert,
// its two gradients, and the gated activation's gradient.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_launch.h"
#include "expert_map.h"
#include "moedx.h"
#include "numeric.h"

namespace moedx {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename S>
struct Mfma;
template <>
struct Mfma<__bf16> {
    typedef __bf16 vec __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 mul(vec a, vec b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Mfma<_Float16> {
    typedef _Float16 vec __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 mul(vec a, vec b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// Operand values of one lane: index i (row of p, or column if kStrided), 8
// values along the reduction from r0; zero outside [0, ni) x [0, nr).
template <typename S, bool kStrided>
__device__ __forceinline__ typename Mfma<S>::vec operand(const S* p, int64_t ld, int64_t i,
                                                         int64_t ni, int64_t r0, int64_t nr) {
    typename Mfma<S>::vec v{};
    if (i >= ni) return v;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (r0 + j < nr) v[j] = kStrided ? p[(r0 + j) * ld + i] : p[i * ld + r0 + j];
    return v;
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// One wave per 16 x 16 output tile; the D tile's lane holds 4 consecutive
// contiguous-dimension outputs of one row.
template <typename S, bool kSwiglu>
__global__ __launch_bounds__(64) void linear_kernel(const S* x, const S* w, ExpertRows er, int K,
                                                    int N, S* y, S* pre) {
    const RowTile tile = find_tile<16>(er, blockIdx.y);
    if (tile.e < 0) return;
    const int lane = threadIdx.x, i = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int64_t cols = kSwiglu ? 2 * (int64_t)N : N;
    const S* we = w + (int64_t)tile.e * cols * K;
    f32x4 acc{0, 0, 0, 0}, up{0, 0, 0, 0};
    for (int k0 = 0; k0 < K; k0 += 32) {
        const auto b = operand<S, false>(x, K, (int64_t)tile.begin + i, tile.end, k0 + g * 8, K);
        const auto a = operand<S, false>(we, K, n0 + i, N, k0 + g * 8, K);
        acc = Mfma<S>::mul(a, b, acc);
        if (kSwiglu) {
            const auto u = operand<S, false>(we + (int64_t)N * K, K, n0 + i, N, k0 + g * 8, K);
            up = Mfma<S>::mul(u, b, up);
        }
    }
    const int m = tile.begin + i;
    if (m >= tile.end) return;
    for (int j = 0; j < 4; ++j) {
        const int n = n0 + g * 4 + j;
        if (n >= N) continue;
        if (kSwiglu) {
            y[(int64_t)m * N + n] = (S)(silu(acc[j]) * up[j]);
            if (pre) {
                pre[(int64_t)m * cols + n] = (S)acc[j];
                pre[(int64_t)m * cols + N + n] = (S)up[j];
            }
        } else {
            y[(int64_t)m * N + n] = (S)acc[j];
        }
    }
}

template <typename S>
__global__ __launch_bounds__(64) void dgrad_kernel(const S* d_y, const S* w, ExpertRows er, int K,
                                                   int N, S* d_x) {
    const RowTile tile = find_tile<16>(er, blockIdx.y);
    if (tile.e < 0) return;
    const int lane = threadIdx.x, i = lane & 15, g = lane >> 4;
    const int k0 = blockIdx.x * 16;
    const S* we = w + (int64_t)tile.e * N * K;
    f32x4 acc{0, 0, 0, 0};
    for (int n0 = 0; n0 < N; n0 += 32) {
        const auto b = operand<S, false>(d_y, N, (int64_t)tile.begin + i, tile.end, n0 + g * 8, N);
        const auto a = operand<S, true>(we, K, k0 + i, K, n0 + g * 8, N);
        acc = Mfma<S>::mul(a, b, acc);
    }
    const int m = tile.begin + i;
    if (m >= tile.end) return;
    for (int j = 0; j < 4; ++j) {
        const int k = k0 + g * 4 + j;
        if (k < K) d_x[(int64_t)m * K + k] = (S)acc[j];
    }
}

template <typename S, typename D>
__global__ __launch_bounds__(64) void wgrad_kernel(const S* d_y, const S* x, ExpertRows er, int K,
                                                   int N, D* d_w) {
    const int e = blockIdx.z;
    const RowSpan s = expert_span(er, e);
    const int lane = threadIdx.x, i = lane & 15, g = lane >> 4;
    const int k0 = blockIdx.x * 16, n0 = blockIdx.y * 16;
    f32x4 acc{0, 0, 0, 0};
    for (int64_t m0 = s.begin; m0 < s.end; m0 += 32) {
        const auto b = operand<S, true>(d_y, N, n0 + i, N, m0 + g * 8, s.end);
        const auto a = operand<S, true>(x, K, k0 + i, K, m0 + g * 8, s.end);
        acc = Mfma<S>::mul(a, b, acc);
    }
    const int n = n0 + i;
    if (n >= N) return;
    for (int j = 0; j < 4; ++j) {
        const int k = k0 + g * 4 + j;
        if (k < K) d_w[((int64_t)e * N + n) * K + k] = (D)acc[j];
    }
}

constexpr int kActThreads = 256;

// One workgroup per row of the buffer; rows of no expert are left alone.
template <typename S>
__global__ __launch_bounds__(kActThreads) void swiglu_backward_kernel(
    const u32x4_t* __restrict__ d_h, const u32x4_t* __restrict__ pre, ExpertRows er, int chunks,
    u32x4_t* __restrict__ d_pre) {
    constexpr int C = Chunk<S>::kN;
    const int64_t row = blockIdx.x;
    bool live;
    if (er.offsets) {
        live = row >= er.offsets[0] && row < er.offsets[er.E];
    } else {
        const int e = (int)(row / er.cap);
        live = row - (int64_t)e * er.cap < er.counts[e];
    }
    if (!live) return;
    for (int c = threadIdx.x; c < chunks; c += kActThreads) {
        float d[C], g[C], u[C];
        chunk_to_f32<S>(d_h[row * chunks + c], d);
        chunk_to_f32<S>(pre[row * 2 * chunks + c], g);
        chunk_to_f32<S>(pre[row * 2 * chunks + chunks + c], u);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const float s = 1.0f / (1.0f + expf(-g[i]));
            const float du = d[i] * g[i] * s;
            g[i] = d[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
            u[i] = du;
        }
        d_pre[row * 2 * chunks + c] = chunk_from_f32<S>(g);
        d_pre[row * 2 * chunks + chunks + c] = chunk_from_f32<S>(u);
    }
}

template <typename S>
hipError_t linear_as(const void* x, const void* w, const ExpertRows& er, int K, int N, bool swiglu,
                     void* y, void* pre, const Launch& L) {
    const dim3 grid((N + 15) / 16, (unsigned)max_tiles(er, 16));
    const S* xs = static_cast<const S*>(x);
    const S* ws = static_cast<const S*>(w);
    if (swiglu)
        return launch_kernel(linear_kernel<S, true>, grid, dim3(64), L, xs, ws, er, K, N,
                             static_cast<S*>(y), static_cast<S*>(pre));
    return launch_kernel(linear_kernel<S, false>, grid, dim3(64), L, xs, ws, er, K, N,
                         static_cast<S*>(y), static_cast<S*>(pre));
}

template <typename S>
hipError_t dgrad_as(const void* d_y, const void* w, const ExpertRows& er, int K, int N, void* d_x,
                    const Launch& L) {
    const dim3 grid((K + 15) / 16, (unsigned)max_tiles(er, 16));
    return launch_kernel(dgrad_kernel<S>, grid, dim3(64), L, static_cast<const S*>(d_y),
                         static_cast<const S*>(w), er, K, N, static_cast<S*>(d_x));
}

template <typename S>
hipError_t wgrad_as(const void* d_y, const void* x, const ExpertRows& er, int K, int N, void* d_w,
                    bool f32_out, const Launch& L) {
    const dim3 grid((K + 15) / 16, (N + 15) / 16, er.E);
    const S* ds = static_cast<const S*>(d_y);
    const S* xs = static_cast<const S*>(x);
    if (f32_out)
        return launch_kernel(wgrad_kernel<S, float>, grid, dim3(64), L, ds, xs, er, K, N,
                             static_cast<float*>(d_w));
    return launch_kernel(wgrad_kernel<S, S>, grid, dim3(64), L, ds, xs, er, K, N,
                         static_cast<S*>(d_w));
}

template <typename S>
hipError_t swiglu_backward_as(const void* d_h, const void* pre, const ExpertRows& er, int N,
                              void* d_pre, const Launch& L) {
    return launch_kernel(swiglu_backward_kernel<S>, dim3((unsigned)er.rows), dim3(kActThreads), L,
                         static_cast<const u32x4_t*>(d_h), static_cast<const u32x4_t*>(pre), er,
                         N / Chunk<S>::kN, static_cast<u32x4_t*>(d_pre));
}

}  // namespace

hipError_t launch_expert_linear(const void* x, const void* w, int dtype, const ExpertRows& er,
                                int K, int N, bool swiglu, void* y, void* pre, const Launch& L) {
    if (dtype == MOEDX_F16) return linear_as<_Float16>(x, w, er, K, N, swiglu, y, pre, L);
    return linear_as<__bf16>(x, w, er, K, N, swiglu, y, pre, L);
}

hipError_t launch_expert_dgrad(const void* d_y, const void* w, int dtype, const ExpertRows& er,
                               int K, int N, void* d_x, const Launch& L) {
    if (dtype == MOEDX_F16) return dgrad_as<_Float16>(d_y, w, er, K, N, d_x, L);
    return dgrad_as<__bf16>(d_y, w, er, K, N, d_x, L);
}

hipError_t launch_expert_wgrad(const void* d_y, const void* x, int dtype, const ExpertRows& er,
                               int K, int N, void* d_w, bool f32_out, const Launch& L) {
    if (dtype == MOEDX_F16) return wgrad_as<_Float16>(d_y, x, er, K, N, d_w, f32_out, L);
    return wgrad_as<__bf16>(d_y, x, er, K, N, d_w, f32_out, L);
}

hipError_t launch_swiglu_backward(const void* d_h, const void* pre, int dtype,
                                  const ExpertRows& er, int N, void* d_pre, const Launch& L) {
    if (dtype == MOEDX_F16) return swiglu_backward_as<_Float16>(d_h, pre, er, N, d_pre, L);
    return swiglu_backward_as<__bf16>(d_h, pre, er, N, d_pre, L);
}

}  // namespace moedx
