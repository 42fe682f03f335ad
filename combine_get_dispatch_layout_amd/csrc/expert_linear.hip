// The experts' products for gfx950: y = x w[e]^T over the rows of each expert,
// its two gradients, and the gated activation's gradient.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_launch.h"
#include "expert_map.h"
#include "mma_tile.h"
#include "moedx.h"
#include "numeric.h"
#include "xcd.h"

namespace moedx {

namespace {

// Tile shapes (mma_tile.h): forward and input gradient 256 x 256 by 8 waves,
// weight gradient 256 x 128 by 4.
template <int BQ_, int WQ_, int BK_>
struct Shape {
    static constexpr int BP = 256, BQ = BQ_, WP = 2, WQ = WQ_, BK = BK_;
    static constexpr int kWaves = WP * WQ, kThreads = kWaves * 64;
    static constexpr int TP = BP / WP / 16, TQ = BQ / WQ / 16;
    static __device__ __forceinline__ int p_at(int wp, int i) { return p_block<BP, WP>(wp, i); }
    static __device__ __forceinline__ int q_at(int wq, int j) { return q_block<WQ>(wq, j); }
};
typedef Shape<256, 4, 64> Wide;
typedef Shape<128, 2, 32> Narrow;

constexpr int kRunLog2 = 5;  // an XCD takes runs of 32 tiles: one per CU, sharing operands in its L2
constexpr int kRowGroup = 8;  // row tiles that go through the columns together

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

template <typename S>
__device__ __forceinline__ void store4(S* at, const f32x4& v) {
    typedef S vec __attribute__((ext_vector_type(4)));
    vec o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (S)v[i];
    *reinterpret_cast<vec*>(at) = o;
}

// Runs f with the number of Q blocks per wave that `rows` rows need.
template <int WQ, typename F>
__device__ __forceinline__ void with_blocks(int rows, F&& f) {
    const int n = (rows + 16 * WQ - 1) / (16 * WQ);
    if (n >= 4) f(std::integral_constant<int, 4>{});
    else if (n == 3) f(std::integral_constant<int, 3>{});
    else if (n == 2) f(std::integral_constant<int, 2>{});
    else f(std::integral_constant<int, 1>{});
}

template <typename S, bool kSwiglu>
__global__ __launch_bounds__(Wide::kThreads, 2) void linear_kernel(const S* x, const S* w, ExpertRows er,
                                                             int K, int N, int cols, S* y, S* pre) {
    typedef Wide T;
    __shared__ __align__(16) S lp0[T::BP * T::BK], lp1[T::BP * T::BK];
    __shared__ __align__(16) S lq0[T::BQ * T::BK], lq1[T::BQ * T::BK];
    const RowTile tile = find_block<T::BQ, kRowGroup>(
        er, xcd_run_block<kRunLog2>((int)blockIdx.x, (int)gridDim.x), cols);
    if (tile.e < 0) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave % T::WP, wq = wave / T::WP;
    const int n0 = tile.col * (kSwiglu ? T::BP / 2 : T::BP);
    const S* we = w + (int64_t)tile.e * (kSwiglu ? 2 : 1) * N * K + (int64_t)n0 * K;
    Along<T::BP, T::kWaves, T::BK, kSwiglu ? 2 : 1> gp;
    gp.init(K * 2, K, wave, lane);
    gp.half(0, we, N - n0);
    if constexpr (kSwiglu) gp.half(1, we + (int64_t)N * K, N - n0);
    Along<T::BQ, T::kWaves, T::BK, 1> gq;
    gq.init(K * 2, K, wave, lane);
    gq.half(0, x + (int64_t)tile.begin * K, tile.end - tile.begin);
    with_blocks<T::WQ>(tile.end - tile.begin, [&](auto nq) {
        constexpr int NQ = decltype(nq)::value;
        f32x4 acc[T::TP][T::TQ] = {};
        WholeCuLoop<S, T::BP, T::BQ, T::WP, T::WQ, NQ, decltype(gp), decltype(gq)>(wp, wq, lane).run(
            gp, gq, (lds_char*)lp0, (lds_char*)lq0, (lds_char*)lp1, (lds_char*)lq1,
            (K + T::BK - 1) / T::BK, wave, acc);
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int m = tile.begin + T::q_at(wq, j) + (lane & 15);
            if (m >= tile.end) continue;
            if constexpr (kSwiglu) {
#pragma unroll
                for (int i = 0; i < T::TP / 2; ++i) {
                    const int n = n0 + T::p_at(wp, i) + 4 * (lane >> 4);
                    if (n >= N) continue;
                    const f32x4 g = acc[i][j], u = acc[i + T::TP / 2][j];
                    f32x4 h;
#pragma unroll
                    for (int r = 0; r < 4; ++r) h[r] = silu(g[r]) * u[r];
                    store4(y + (int64_t)m * N + n, h);
                    if (pre) {
                        store4(pre + (int64_t)m * 2 * N + n, g);
                        store4(pre + (int64_t)m * 2 * N + N + n, u);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < T::TP; ++i) {
                    const int n = n0 + T::p_at(wp, i) + 4 * (lane >> 4);
                    if (n < N) store4(y + (int64_t)m * N + n, acc[i][j]);
                }
            }
        }
    });
}

template <typename S>
__global__ __launch_bounds__(Wide::kThreads, 2) void dgrad_kernel(const S* d_y, const S* w, ExpertRows er,
                                                            int K, int N, int cols, S* d_x) {
    typedef Wide T;
    __shared__ __align__(16) S lp0[T::BP * T::BK], lp1[T::BP * T::BK];
    __shared__ __align__(16) S lq0[T::BQ * T::BK], lq1[T::BQ * T::BK];
    const RowTile tile = find_block<T::BQ, kRowGroup>(
        er, xcd_run_block<kRunLog2>((int)blockIdx.x, (int)gridDim.x), cols);
    if (tile.e < 0) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave % T::WP, wq = wave / T::WP;
    const int k0 = tile.col * T::BP;
    Across<T::BP, T::kWaves, T::BK> gp;
    gp.init(w + (int64_t)tile.e * N * K, K * 2, N, k0, K, wave, lane);
    Along<T::BQ, T::kWaves, T::BK, 1> gq;
    gq.init(N * 2, N, wave, lane);
    gq.half(0, d_y + (int64_t)tile.begin * N, tile.end - tile.begin);
    with_blocks<T::WQ>(tile.end - tile.begin, [&](auto nq) {
        constexpr int NQ = decltype(nq)::value;
        f32x4 acc[T::TP][T::TQ] = {};
        WholeCuLoop<S, T::BP, T::BQ, T::WP, T::WQ, NQ, decltype(gp), decltype(gq)>(wp, wq, lane).run(
            gp, gq, (lds_char*)lp0, (lds_char*)lq0, (lds_char*)lp1, (lds_char*)lq1,
            (N + T::BK - 1) / T::BK, wave, acc);
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int m = tile.begin + T::q_at(wq, j) + (lane & 15);
            if (m >= tile.end) continue;
#pragma unroll
            for (int i = 0; i < T::TP; ++i) {
                const int k = k0 + T::p_at(wp, i) + 4 * (lane >> 4);
                if (k < K) store4(d_x + (int64_t)m * K + k, acc[i][j]);
            }
        }
    });
}

template <typename S, typename D>
__global__ __launch_bounds__(Narrow::kThreads, 2) void wgrad_kernel(const S* d_y, const S* x, ExpertRows er,
                                                            int K, int N, int cols, int rows,
                                                            D* d_w) {
    typedef Narrow T;
    __shared__ __align__(16) S lp0[T::BP * T::BK], lp1[T::BP * T::BK], lp2[T::BP * T::BK];
    __shared__ __align__(16) S lq0[T::BQ * T::BK], lq1[T::BQ * T::BK], lq2[T::BQ * T::BK];
    int b = xcd_run_block<kRunLog2>((int)blockIdx.x, (int)gridDim.x);
    const int e = b / (cols * rows);
    b -= e * cols * rows;
    // row tiles in groups, each through all columns
    const int grp = b / (kRowGroup * cols);
    b -= grp * kRowGroup * cols;
    const int in_grp = min(kRowGroup, rows - grp * kRowGroup);
    const int k0 = b / in_grp * T::BP, n0 = (grp * kRowGroup + b % in_grp) * T::BQ;
    const RowSpan s = expert_span(er, e);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave % T::WP, wq = wave / T::WP;
    const int count = s.end - s.begin;
    Across<T::BP, T::kWaves, T::BK> gp;
    gp.init(x + (int64_t)s.begin * K, K * 2, count, k0, K, wave, lane);
    Across<T::BQ, T::kWaves, T::BK> gq;
    gq.init(d_y + (int64_t)s.begin * N, N * 2, count, n0, N, wave, lane);
    with_blocks<T::WQ>(N - n0, [&](auto nq) {
        constexpr int NQ = decltype(nq)::value;
        f32x4 acc[T::TP][T::TQ] = {};
        SharedCuLoop<S, T::BP, T::BQ, T::WP, T::WQ, NQ, decltype(gp), decltype(gq)>(wp, wq, lane).run(
            gp, gq, (lds_char*)lp0, (lds_char*)lq0, (lds_char*)lp1, (lds_char*)lq1,
            (lds_char*)lp2, (lds_char*)lq2,
            (count + T::BK - 1) / T::BK, wave, acc);
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int n = n0 + T::q_at(wq, j) + (lane & 15);
            if (n >= N) continue;
#pragma unroll
            for (int i = 0; i < T::TP; ++i) {
                const int k = k0 + T::p_at(wp, i) + 4 * (lane >> 4);
                if (k < K) store4(d_w + ((int64_t)e * N + n) * K + k, acc[i][j]);
            }
        }
    });
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

int tiles_of(int n, int b) { return (n + b - 1) / b; }

template <typename S>
hipError_t linear_as(const void* x, const void* w, const ExpertRows& er, int K, int N, bool swiglu,
                     void* y, void* pre, const Launch& L) {
    const int cols = tiles_of(N, swiglu ? Wide::BP / 2 : Wide::BP);
    const dim3 grid((unsigned)(max_tiles(er, Wide::BQ) * cols));
    const S* xs = static_cast<const S*>(x);
    const S* ws = static_cast<const S*>(w);
    if (swiglu)
        return launch_kernel(linear_kernel<S, true>, grid, dim3(Wide::kThreads), L, xs, ws, er, K, N,
                             cols, static_cast<S*>(y), static_cast<S*>(pre));
    return launch_kernel(linear_kernel<S, false>, grid, dim3(Wide::kThreads), L, xs, ws, er, K, N, cols,
                         static_cast<S*>(y), static_cast<S*>(pre));
}

template <typename S>
hipError_t dgrad_as(const void* d_y, const void* w, const ExpertRows& er, int K, int N, void* d_x,
                    const Launch& L) {
    const int cols = tiles_of(K, Wide::BP);
    const dim3 grid((unsigned)(max_tiles(er, Wide::BQ) * cols));
    return launch_kernel(dgrad_kernel<S>, grid, dim3(Wide::kThreads), L, static_cast<const S*>(d_y),
                         static_cast<const S*>(w), er, K, N, cols, static_cast<S*>(d_x));
}

template <typename S>
hipError_t wgrad_as(const void* d_y, const void* x, const ExpertRows& er, int K, int N, void* d_w,
                    bool f32_out, const Launch& L) {
    const int cols = tiles_of(K, Narrow::BP), rows = tiles_of(N, Narrow::BQ);
    const dim3 grid((unsigned)((int64_t)cols * rows * er.E));
    const S* ds = static_cast<const S*>(d_y);
    const S* xs = static_cast<const S*>(x);
    if (f32_out)
        return launch_kernel(wgrad_kernel<S, float>, grid, dim3(Narrow::kThreads), L, ds, xs, er, K, N,
                             cols, rows, static_cast<float*>(d_w));
    return launch_kernel(wgrad_kernel<S, S>, grid, dim3(Narrow::kThreads), L, ds, xs, er, K, N, cols, rows,
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
