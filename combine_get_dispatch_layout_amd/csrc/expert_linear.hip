// The experts' products for gfx950: y = x w[e]^T over the rows of each expert,
// its two gradients, and the gated activation's gradient.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_launch.h"
#include "expert_map.h"
#include "expert_tile.h"
#include "mma_tile.h"
#include "moedx.h"
#include "numeric.h"
#include "xcd.h"

namespace moedx {

namespace {

template <typename S, bool kSwiglu, typename T>
__global__ __launch_bounds__(T::kThreads, 2) void linear_kernel(const S* x, const S* w,
                                                                ExpertRows er, int K, int N,
                                                                int cols, S* y, S* pre,
                                                                bool rotate) {
    // One array: with two, the compiler reads LDS before it asks for the next
    // stage of Q (64 experts of about 182 rows, 4096 -> 4096: 555 and 534 us).
    __shared__ __align__(16) S lp[T::kP * T::BP * T::BK + T::kQ * T::BQ * T::BK];
    S* const lq = lp + T::kP * T::BP * T::BK;
    const int blk = xcd_run_block<kRunLog2>((int)blockIdx.x, (int)gridDim.x);
    const RowTile tile = find_block<T::BQ, kRowGroup>(er, blk, cols);
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
        const int nk = (K + T::BK - 1) / T::BK;
        RingLoop<S, T::BP, T::BQ, T::WP, T::WQ, NQ, T::kP, T::kQ, true, decltype(gp),
                 decltype(gq)>(
            wp, wq, lane, rotate ? scattered(blk, nk) : 0, nk)
            .run(gp, gq, (lds_char*)lp, (lds_char*)lq, wave, acc);
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const uint32_t m = (uint32_t)tile.begin + T::q_at(wq, j) + (lane & 15);
            const bool row = m < (uint32_t)tile.end;  // unsigned: past 2^31 for the last tiles
            S* const ym = y + (int64_t)m * N;
            if constexpr (kSwiglu) {
                S* const gm = pre + (int64_t)m * 2 * N;
#pragma unroll
                for (int i = 0; i < T::TP / 2; i += 2) {
                    const int n = n0 + T::p_at(wp, i) + pair_at(lane);
                    const f32x4 g[2] = {acc[i][j], acc[i + 1][j]};
                    const f32x4 u[2] = {acc[i + T::TP / 2][j], acc[i + 1 + T::TP / 2][j]};
                    f32x4 h[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int r = 0; r < 4; ++r) h[b][r] = silu(g[b][r]) * u[b][r];
                    const bool in = row && n < N;
                    const u32x4_t hv = pack_pair<S>(h[0], h[1]);
                    if (in) store8(ym + n, hv);
                    if (pre) {
                        const u32x4_t gv = pack_pair<S>(g[0], g[1]), uv = pack_pair<S>(u[0], u[1]);
                        if (in) {
                            store8(gm + n, gv);
                            store8(gm + N + n, uv);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < T::TP; i += 2) {
                    const int n = n0 + T::p_at(wp, i) + pair_at(lane);
                    const u32x4_t v = pack_pair<S>(acc[i][j], acc[i + 1][j]);
                    if (row && n < N) store8(ym + n, v);
                }
            }
        }
    });
}

// The forward product where experts have few rows: the weights' bytes are all
// that counts, so they go from memory straight into registers, with no LDS and
// no barrier on the way.  A workgroup takes 32 weight rows (16 gate
// and 16 up rows in a gated product) and up to 32 rows of x; its 4
// waves take turns along the reduction, 128 values each, and their sums are
// added in LDS in wave order.  x comes from the caches.  64 experts of 4096 x
// 7168, one row each: 602 us, the weights at 6.25 TB/s (a large copy reaches
// 6.3); 12 rows each: 659 us.
constexpr int kFewP = 2;  // blocks of 16 weight rows
constexpr int kFewRows = 32, kFewBlocks = kFewRows / 16, kFewWaves = 4, kFewThreads = kFewWaves * 64,
              kFewStep = 128 * kFewWaves;
constexpr int kFewRunLog2 = 3;
static_assert(same({kFewRows, kFewP * 16, kFewThreads}, kFewTile), "the plan's tile is the kernel's");

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

// Two blocks of 16 weight rows times NQ blocks of 16 rows of x.
template <typename S, int NQ>
__device__ __forceinline__ void few_products(const FewRows* ws, const FewRows* xs, int K, int shift,
                                             int wave, int lane, f32x4 (&acc)[kFewP][kFewBlocks]) {
    constexpr int kU = 4, kStep = kFewStep;
    static_assert(kStep == 32 * kU * kFewWaves, "a step of all waves");
    const int steps = (K + kStep - 1) / kStep;
    s16x8 a[2][kFewP][kU], b[2][NQ][kU];
    const int in = (lane >> 4) * 8;
    // Steps go around the reduction from `shift` on; past the last one nothing
    // is read.  The scheduling barriers keep the loads of one step ahead of the
    // products of the other.
    const auto fetch = [&](int s, int step) {
        int at = step + shift;
        at -= at >= steps ? steps : 0;
        const int k0 = step < steps ? at * kStep + wave * 32 * kU : K;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int k = k0 + u * 32;
            const bool inside = k + in < K;
#pragma unroll
            for (int i = 0; i < kFewP; ++i) a[s][i][u] = ws[i].load(k, inside);
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
                for (int i = 0; i < kFewP; ++i)
                    acc[i][j] = Mfma<S>::mul(a[s][i][u], b[s][j][u], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
    };
    fetch(0, 0);
    for (int step = 0; step < steps; step += 2) {
        fetch(1, step + 1);
        multiply(0);
        fetch(0, step + 2);
        multiply(1);
    }
}

template <typename S, bool kSwiglu>
__global__ __launch_bounds__(kFewThreads) void linear_few_kernel(const S* x, const S* w,
                                                                 ExpertRows er, int K, int N,
                                                                 int cols, S* y, S* pre, bool rotate) {
    constexpr int kOut = kSwiglu ? kFewP / 2 : kFewP;  // blocks of outputs
    __shared__ f32x4 part[kFewWaves][kFewBlocks][kFewP][64];
    const int blk = xcd_run_block<kFewRunLog2>((int)blockIdx.x, (int)gridDim.x);
    const RowTile tile = find_block<kFewRows, kRowGroup>(er, blk, cols);
    if (tile.e < 0) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = tile.col * kOut * 16;
    const S* we = w + (int64_t)tile.e * (kSwiglu ? 2 : 1) * N * K;
    const int rows = tile.end - tile.begin;
    FewRows ws[kFewP], xs[kFewBlocks];
#pragma unroll
    for (int i = 0; i < kFewP; ++i) {
        const int n = n0 + i % kOut * 16;
        ws[i].init(we + (int64_t)(i < kOut ? n : N + n) * K, min(N - n, 16), K, lane);
    }
#pragma unroll
    for (int j = 0; j < kFewBlocks; ++j)
        xs[j].init(x + ((int64_t)tile.begin + 16 * j) * K, min(rows - 16 * j, 16), K, lane);
    f32x4 acc[kFewP][kFewBlocks] = {};
    const int shift = rotate ? scattered(blk, (K + kFewStep - 1) / kFewStep) : 0;
    if (rows > 16)
        few_products<S, 2>(ws, xs, K, shift, wave, lane, acc);
    else
        few_products<S, 1>(ws, xs, K, shift, wave, lane, acc);
#pragma unroll
    for (int j = 0; j < kFewBlocks; ++j)
#pragma unroll
        for (int i = 0; i < kFewP; ++i) part[wave][j][i][lane] = acc[i][j];
    __syncthreads();
    // wave j finishes block j of 16 rows
    if (wave >= kFewBlocks) return;
    const uint32_t m = (uint32_t)tile.begin + wave * 16 + (lane & 15);
    if (m >= (uint32_t)tile.end) return;
    f32x4 sum[kFewP];
#pragma unroll
    for (int i = 0; i < kFewP; ++i) {
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

template <typename S, typename T>
__global__ __launch_bounds__(T::kThreads, 2) void dgrad_kernel(const S* d_y, const S* w, ExpertRows er,
                                                            int K, int N, int cols, S* d_x) {
    __shared__ __align__(16) S lp[T::kP * T::BP * T::BK];
    __shared__ __align__(16) S lq[T::kQ * T::BQ * T::BK];
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
        RingLoop<S, T::BP, T::BQ, T::WP, T::WQ, NQ, T::kP, T::kQ, false, decltype(gp),
                 decltype(gq)>(
            wp, wq, lane, 0, (N + T::BK - 1) / T::BK)
            .run(gp, gq, (lds_char*)lp, (lds_char*)lq, wave, acc);
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const uint32_t m = (uint32_t)tile.begin + T::q_at(wq, j) + (lane & 15);
#pragma unroll
            for (int i = 0; i < T::TP; i += 2) {
                const int k = k0 + T::p_at(wp, i) + pair_at(lane);
                const u32x4_t v = pack_pair<S>(acc[i][j], acc[i + 1][j]);
                if (m < (uint32_t)tile.end && k < K) store8(d_x + (int64_t)m * K + k, v);
            }
        }
    });
}

template <typename S, typename D>
__global__ __launch_bounds__(WeightGrad::kThreads, 2) void wgrad_kernel(const S* d_y, const S* x,
                                                                        ExpertRows er, int K, int N,
                                                                        int cols, int rows, D* d_w) {
    typedef WeightGrad T;
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
            row_tiles<T::BK>(count), wave, acc);
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int n = n0 + T::q_at(wq, j) + (lane & 15);
            D* const row = d_w + ((int64_t)e * N + n) * K;
            if constexpr (sizeof(D) == 2) {
#pragma unroll
                for (int i = 0; i < T::TP; i += 2) {
                    const int k = k0 + T::p_at(wp, i) + pair_at(lane);
                    const u32x4_t v = pack_pair<D>(acc[i][j], acc[i + 1][j]);
                    if (n < N && k < K) store8(row + k, v);
                }
            } else {
#pragma unroll
                for (int i = 0; i < T::TP; ++i) {
                    const int k = k0 + T::p_at(wp, i) + 4 * (lane >> 4);
                    if (n < N && k < K) store4(row + k, acc[i][j]);
                }
            }
        }
    });
}

constexpr int kActThreads = 256;
constexpr int64_t kActGrid = 1 << 20;  // workgroups at most

// Workgroups go through the buffer's rows, one row at a time; rows of no expert
// are left alone.  Bound by memory from rows of 1024 values on: 65536 x 1024
// bf16 110 us (6.1 TB/s), 49152 x 2048 169 (6.0), 32768 x 4096 224 (6.0), 16384 x
// 7168 217 (5.4).  Narrower rows leave threads idle: 65536 x 768 105 us (4.8
// TB/s), 65536 x 256 61 us (2.8).
template <typename S>
__global__ __launch_bounds__(kActThreads) void swiglu_backward_kernel(
    const u32x4_t* __restrict__ d_h, const u32x4_t* __restrict__ pre, ExpertRows er, int chunks,
    u32x4_t* __restrict__ d_pre) {
    constexpr int C = Chunk<S>::kN;
    for (int64_t row = blockIdx.x; row < er.rows; row += gridDim.x) {
        bool live;
        if (er.offsets) {
            live = row >= er.offsets[0] && row < er.offsets[er.E];
        } else {
            const int e = (int)(row / er.cap);
            live = row - (int64_t)e * er.cap < er.counts[e];
        }
        if (!live) continue;
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
}

dim3 grid_of(int64_t workgroups) { return dim3((unsigned)workgroups); }

template <typename S, typename T>
hipError_t linear_tiles(const S* x, const S* w, const ExpertRows& er, int K, int N, bool swiglu,
                        bool rotate, S* y, S* pre, const Launch& L) {
    const int outs = swiglu ? 2 * N : N, cols = (int)tiles_of(outs, T::kTile.outs);
    return launch_kernel(swiglu ? linear_kernel<S, true, T> : linear_kernel<S, false, T>,
                         grid_of(workgroups(er, T::kTile, outs)), dim3(T::kThreads), L, x, w, er, K,
                         N, cols, y, pre, rotate);
}

template <typename S>
hipError_t linear_as(const void* x, const void* w, const ExpertRows& er, int K, int N, bool swiglu,
                     void* y, void* pre, const Launch& L) {
    const S* xs = static_cast<const S*>(x);
    const S* ws = static_cast<const S*>(w);
    S* ys = static_cast<S*>(y);
    S* ps = static_cast<S*>(pre);
    const int outs = swiglu ? 2 * N : N;
    const bool rotate = rotates(expected_rows(er), K);
    switch (forward_tiles(er, outs)) {
        case Tiles::kFew:
            return launch_kernel(swiglu ? linear_few_kernel<S, true> : linear_few_kernel<S, false>,
                                 grid_of(workgroups(er, kFewTile, outs)), dim3(kFewThreads), L, xs,
                                 ws, er, K, N, (int)tiles_of(outs, kFewTile.outs), ys, ps, rotate);
        case Tiles::kSmall:
            return linear_tiles<S, Small>(xs, ws, er, K, N, swiglu, rotate, ys, ps, L);
        case Tiles::kWide:
            return linear_tiles<S, Wide>(xs, ws, er, K, N, swiglu, rotate, ys, ps, L);
        default:
            return hipErrorInvalidValue;  // refused before
    }
}

template <typename S, typename T>
hipError_t dgrad_tiles(const S* d_y, const S* w, const ExpertRows& er, int K, int N, S* d_x,
                       const Launch& L) {
    return launch_kernel(dgrad_kernel<S, T>, grid_of(workgroups(er, T::kTile, K)),
                         dim3(T::kThreads), L, d_y, w, er, K, N, (int)tiles_of(K, T::kTile.outs),
                         d_x);
}

template <typename S>
hipError_t dgrad_as(const void* d_y, const void* w, const ExpertRows& er, int K, int N, void* d_x,
                    const Launch& L) {
    const S* ds = static_cast<const S*>(d_y);
    const S* ws = static_cast<const S*>(w);
    switch (input_gradient_tiles(er, K)) {
        case Tiles::kSmall:
            return dgrad_tiles<S, Small>(ds, ws, er, K, N, static_cast<S*>(d_x), L);
        case Tiles::kWide:
            return dgrad_tiles<S, Wide>(ds, ws, er, K, N, static_cast<S*>(d_x), L);
        default:
            return hipErrorInvalidValue;  // refused before
    }
}

template <typename S>
hipError_t wgrad_as(const void* d_y, const void* x, const ExpertRows& er, int K, int N, void* d_w,
                    bool f32_out, const Launch& L) {
    const int cols = (int)tiles_of(K, WeightGrad::BP), rows = (int)tiles_of(N, WeightGrad::BQ);
    const dim3 grid = grid_of(weight_workgroups(er, K, N));
    const S* ds = static_cast<const S*>(d_y);
    const S* xs = static_cast<const S*>(x);
    if (f32_out)
        return launch_kernel(wgrad_kernel<S, float>, grid, dim3(WeightGrad::kThreads), L, ds, xs,
                             er, K, N, cols, rows, static_cast<float*>(d_w));
    return launch_kernel(wgrad_kernel<S, S>, grid, dim3(WeightGrad::kThreads), L, ds, xs, er, K,
                         N, cols, rows, static_cast<S*>(d_w));
}

template <typename S>
hipError_t swiglu_backward_as(const void* d_h, const void* pre, const ExpertRows& er, int N,
                              void* d_pre, const Launch& L) {
    const dim3 grid((unsigned)(er.rows < kActGrid ? er.rows : kActGrid));
    return launch_kernel(swiglu_backward_kernel<S>, grid, dim3(kActThreads), L,
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
