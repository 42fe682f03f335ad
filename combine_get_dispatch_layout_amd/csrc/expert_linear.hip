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

// The forward product where experts have few rows: the weights' bytes are all
// that counts, so they go from memory straight into registers, with no LDS and
// no barrier on the way.  A workgroup takes NP blocks of 16 weight rows (half
// of them gate, half up rows in a gated product) and up to 32 rows of x; its 4
// waves take turns along the reduction, 128 values each, and their sums are
// added in LDS in wave order.  x comes from the caches.  64 experts of 4096 x
// 7168, one row each: 602 us, the weights at 6.25 TB/s (a large copy reaches
// 6.3); 12 rows each: 659 us.
constexpr int kFewRows = 32, kFewBlocks = kFewRows / 16, kFewWaves = 4, kFewThreads = kFewWaves * 64;
constexpr int kFewRunLog2 = 3;

// 16 rows of an operand along r, read by the whole wave: lane l takes row
// l & 15, reduction values 8 (l >> 4) .. + 7 of each 32; zeros outside.
struct FewRows {
    __amdgpu_buffer_rsrc_t rs;
    int off;
    __device__ __forceinline__ void init(const void* first, int rows, int K, int lane) {
        rs = make_rsrc(first, rows * K * 2);
        off = (lane & 15) * K * 2 + (lane >> 4) * 16;
    }
    __device__ __forceinline__ s16x8 load(int k, bool inside) const {
        return __builtin_bit_cast(s16x8, __builtin_amdgcn_raw_buffer_load_b128(
                                             rs, inside ? off + k * 2 : (int)kOutside, 0, 0));
    }
};

// NP blocks of 16 weight rows times NQ blocks of 16 rows of x.
template <typename S, int NP, int NQ>
__device__ __forceinline__ void few_products(const FewRows* ws, const FewRows* xs, int K, int wave,
                                             int lane, f32x4 (&acc)[NP][kFewBlocks]) {
    constexpr int kU = 4, kStep = 32 * kU * kFewWaves;
    s16x8 a[2][NP][kU], b[2][NQ][kU];
    const int first = wave * 32 * kU, in = (lane >> 4) * 8;
    // The scheduling barriers keep the loads of one step ahead of the products
    // of the other.
    const auto fetch = [&](int s, int k0) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int k = k0 + u * 32;
            const bool inside = k + in < K;
#pragma unroll
            for (int i = 0; i < NP; ++i) a[s][i][u] = ws[i].load(k, inside);
#pragma unroll
            for (int j = 0; j < NQ; ++j) b[s][j][u] = xs[j].load(k, inside);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    const auto multiply = [&](int s) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int j = 0; j < NQ; ++j)
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    acc[i][j] = Mfma<S>::mul(a[s][i][u], b[s][j][u], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
    };
    fetch(0, first);
    for (int k0 = first; k0 < K; k0 += 2 * kStep) {
        fetch(1, k0 + kStep);
        multiply(0);
        fetch(0, k0 + 2 * kStep);
        multiply(1);
    }
}

// NP: blocks of 16 weight rows; with kSwiglu the first half are gate rows.
template <typename S, bool kSwiglu, int NP>
__global__ __launch_bounds__(kFewThreads) void linear_few_kernel(const S* x, const S* w,
                                                                 ExpertRows er, int K, int N,
                                                                 int cols, S* y, S* pre) {
    constexpr int kOut = kSwiglu ? NP / 2 : NP;  // blocks of outputs
    __shared__ f32x4 part[kFewWaves][kFewBlocks][NP][64];
    const RowTile tile = find_block<kFewRows, kRowGroup>(
        er, xcd_run_block<kFewRunLog2>((int)blockIdx.x, (int)gridDim.x), cols);
    if (tile.e < 0) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = tile.col * kOut * 16;
    const S* we = w + (int64_t)tile.e * (kSwiglu ? 2 : 1) * N * K;
    const int rows = tile.end - tile.begin;
    FewRows ws[NP], xs[kFewBlocks];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int n = n0 + i % kOut * 16;
        ws[i].init(we + (int64_t)(i < kOut ? n : N + n) * K, min(N - n, 16), K, lane);
    }
#pragma unroll
    for (int j = 0; j < kFewBlocks; ++j)
        xs[j].init(x + (int64_t)(tile.begin + 16 * j) * K, min(rows - 16 * j, 16), K, lane);
    f32x4 acc[NP][kFewBlocks] = {};
    if (rows > 16)
        few_products<S, NP, 2>(ws, xs, K, wave, lane, acc);
    else
        few_products<S, NP, 1>(ws, xs, K, wave, lane, acc);
#pragma unroll
    for (int j = 0; j < kFewBlocks; ++j)
#pragma unroll
        for (int i = 0; i < NP; ++i) part[wave][j][i][lane] = acc[i][j];
    __syncthreads();
    // wave j finishes block j of 16 rows
    if (wave >= kFewBlocks) return;
    const int m = tile.begin + wave * 16 + (lane & 15);
    if (m >= tile.end) return;
    f32x4 sum[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        sum[i] = part[0][wave][i][lane];
#pragma unroll
        for (int v = 1; v < kFewWaves; ++v) {
            const f32x4 a = part[v][wave][i][lane];
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[i][r] += a[r];
        }
    }
#pragma unroll
    for (int i = 0; i < kOut; ++i) {
        const int n = n0 + i * 16 + 4 * (lane >> 4);
        if (n >= N) return;
        if constexpr (kSwiglu) {
            const f32x4 g = sum[i], u = sum[kOut + i];
            f32x4 h;
#pragma unroll
            for (int r = 0; r < 4; ++r) h[r] = silu(g[r]) * u[r];
            store4(y + (int64_t)m * N + n, h);
            if (pre) {
                store4(pre + (int64_t)m * 2 * N + n, g);
                store4(pre + (int64_t)m * 2 * N + N + n, u);
            }
        } else {
            store4(y + (int64_t)m * N + n, sum[i]);
        }
    }
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
        chunk_to_f32<S>(__builtin_nontemporal_load(d_h + row * chunks + c), d);
        chunk_to_f32<S>(__builtin_nontemporal_load(pre + row * 2 * chunks + c), g);
        chunk_to_f32<S>(__builtin_nontemporal_load(pre + row * 2 * chunks + chunks + c), u);
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

// Rows an expert is likely to have, from what the host knows.  A capacity
// buffer holds at most cap tokens, each with a few experts: 8 are taken, the
// top-k of the wide routings (more only moves where the kernels change).
int64_t expected_rows(const ExpertRows& er) {
    if (er.offsets) return er.rows / er.E;
    return er.E > 8 ? (int64_t)er.cap * 8 / er.E : er.cap;
}

template <typename S>
hipError_t linear_as(const void* x, const void* w, const ExpertRows& er, int K, int N, bool swiglu,
                     void* y, void* pre, const Launch& L) {
    const S* xs = static_cast<const S*>(x);
    const S* ws = static_cast<const S*>(w);
    // 64 experts, 7168 -> 4096, us at 1 / 12 / 24 / 40 rows each: 2 blocks 602 /
    // 659 / 821 / 988, 4 blocks 629 / 644 / 695 / 765, tiles 731 / 721 / 727 / 740.
    // Fewer columns per workgroup also means more workgroups for a few experts.
    const int64_t likely = expected_rows(er);
    if (likely <= 32) {
        const int np = likely <= 16 ? 2 : 4;
        const int cols = tiles_of(N, swiglu ? np * 8 : np * 16);
        const dim3 grid((unsigned)(max_tiles(er, kFewRows) * cols));
        const auto two = swiglu ? linear_few_kernel<S, true, 2> : linear_few_kernel<S, false, 2>;
        const auto four = swiglu ? linear_few_kernel<S, true, 4> : linear_few_kernel<S, false, 4>;
        return launch_kernel(np == 2 ? two : four, grid, dim3(kFewThreads), L, xs, ws, er, K, N,
                             cols, static_cast<S*>(y), static_cast<S*>(pre));
    }
    const int cols = tiles_of(N, swiglu ? Wide::BP / 2 : Wide::BP);
    const dim3 grid((unsigned)(max_tiles(er, Wide::BQ) * cols));
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
