// The experts' products in int8 for gfx950, y = (c v^T) scaled by row and by
// output, and the weight gradient from saved int8 rows.
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

// The tiles are those of the 16-bit product (mma_tile.h) over Codes2: the same
// bytes per stage and the same instructions, each of twice the multiplications.
// Sums are exact integers, so a row's outputs depend on nothing but the row and
// its expert: not on the tile, the buffer or where the workgroup starts.

// Four neighbouring outputs of one row: (sum * row's scale) * output's scale.
__device__ __forceinline__ f32x4 scaled(const i32x4& sum, float xs, const f32x4& ws) {
    f32x4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = in_fp32((float)sum[r] * xs * ws[r]);
    return v;
}
__device__ __forceinline__ f32x4 scales4(const float* ws, int n, int N) {
    f32x4 v = {};
    if (n < N) v = *reinterpret_cast<const f32x4*>(ws + n);
    return v;
}

template <typename S, bool kSwiglu, typename T>
__global__ __launch_bounds__(T::kThreads, 2) void linear_int8_kernel(
    const int8_t* x, const float* xs, const int8_t* w, const float* ws, ExpertRows er, int K, int N,
    int cols, S* y, bool rotate) {
    __shared__ __align__(16) Codes2 lp[T::kP * T::BP * T::BK + T::kQ * T::BQ * T::BK];
    Codes2* const lq = lp + T::kP * T::BP * T::BK;
    const int blk = xcd_run_block<kRunLog2>((int)blockIdx.x, (int)gridDim.x);
    const RowTile tile = find_block<T::BQ, kRowGroup>(er, blk, cols);
    if (tile.e < 0) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave % T::WP, wq = wave / T::WP;
    const int n0 = tile.col * (kSwiglu ? T::BP / 2 : T::BP);
    const int64_t first = (int64_t)tile.e * (kSwiglu ? 2 : 1) * N;  // the expert's weight rows
    const int8_t* we = w + (first + n0) * K;
    Along<T::BP, T::kWaves, T::BK, kSwiglu ? 2 : 1> gp;
    gp.init(K, K / 2, wave, lane);
    gp.half(0, we, N - n0);
    if constexpr (kSwiglu) gp.half(1, we + (int64_t)N * K, N - n0);
    Along<T::BQ, T::kWaves, T::BK, 1> gq;
    gq.init(K, K / 2, wave, lane);
    gq.half(0, x + (int64_t)tile.begin * K, tile.end - tile.begin);
    with_blocks<T::WQ>(tile.end - tile.begin, [&](auto nq) {
        constexpr int NQ = decltype(nq)::value;
        i32x4 acc[T::TP][T::TQ] = {};
        const int nk = (K / 2 + T::BK - 1) / T::BK;
        RingLoop<Codes2, T::BP, T::BQ, T::WP, T::WQ, NQ, T::kP, T::kQ, true, decltype(gp),
                 decltype(gq)>(wp, wq, lane, rotate ? scattered(blk, nk) : 0, nk)
            .run(gp, gq, (lds_char*)lp, (lds_char*)lq, wave, acc);
        const float* const wse = ws + first;
        const int mine = 4 * (lane >> 4);  // this lane's first output of a block of 16
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const uint32_t m = (uint32_t)tile.begin + T::q_at(wq, j) + (lane & 15);
            const bool row = m < (uint32_t)tile.end;  // unsigned: past 2^31 for the last tiles
            const float xm = row ? xs[m] : 0.0f;
            S* const ym = y + (int64_t)m * N;
            if constexpr (kSwiglu) {
#pragma unroll
                for (int i = 0; i < T::TP / 2; i += 2) {
                    f32x4 h[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int n = n0 + T::p_at(wp, i + b) + mine;
                        const f32x4 g = scaled(acc[i + b][j], xm, scales4(wse, n, N));
                        const f32x4 u =
                            scaled(acc[i + b + T::TP / 2][j], xm, scales4(wse + N, n, N));
#pragma unroll
                        for (int r = 0; r < 4; ++r) h[b][r] = in_fp32(silu(g[r]) * u[r]);
                    }
                    const int n = n0 + T::p_at(wp, i) + pair_at(lane);
                    const u32x4_t hv = pack_pair<S>(h[0], h[1]);
                    if (row && n < N) store8(ym + n, hv);
                }
            } else {
#pragma unroll
                for (int i = 0; i < T::TP; i += 2) {
                    const int a = n0 + T::p_at(wp, i) + mine, b = n0 + T::p_at(wp, i + 1) + mine;
                    const u32x4_t v = pack_pair<S>(scaled(acc[i][j], xm, scales4(wse, a, N)),
                                                   scaled(acc[i + 1][j], xm, scales4(wse, b, N)));
                    const int n = n0 + T::p_at(wp, i) + pair_at(lane);
                    if (row && n < N) store8(ym + n, v);
                }
            }
        }
    });
}

// Few rows per expert: weights straight into registers (few_products).
template <typename S, bool kSwiglu>
__global__ __launch_bounds__(kFewThreads) void linear_int8_few_kernel(
    const int8_t* x, const float* xs, const int8_t* w, const float* ws, ExpertRows er, int K, int N,
    int cols, S* y, bool rotate) {
    constexpr int kOut = kSwiglu ? kFewP / 2 : kFewP;  // blocks of outputs
    __shared__ i32x4 part[kFewWaves][kFewBlocks][kFewP][64];
    const int blk = xcd_run_block<kFewRunLog2>((int)blockIdx.x, (int)gridDim.x);
    const RowTile tile = find_block<kFewRows, kRowGroup>(er, blk, cols);
    if (tile.e < 0) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = tile.col * kOut * 16;
    const int64_t first = (int64_t)tile.e * (kSwiglu ? 2 : 1) * N;
    const int rows = tile.end - tile.begin;
    FewRows wr[kFewP], xr[kFewBlocks];
#pragma unroll
    for (int i = 0; i < kFewP; ++i) {
        const int n = n0 + i % kOut * 16;
        wr[i].init(w + (first + (i < kOut ? n : N + n)) * K, min(N - n, 16), K / 2, lane);
    }
#pragma unroll
    for (int j = 0; j < kFewBlocks; ++j)
        xr[j].init(x + ((int64_t)tile.begin + 16 * j) * K, min(rows - 16 * j, 16), K / 2, lane);
    i32x4 acc[kFewP][kFewBlocks] = {};
    const int shift = rotate ? scattered(blk, (K / 2 + kFewStep - 1) / kFewStep) : 0;
    if (rows > 16)
        few_products<Codes2, 2>(wr, xr, K / 2, shift, wave, lane, acc);
    else
        few_products<Codes2, 1>(wr, xr, K / 2, shift, wave, lane, acc);
#pragma unroll
    for (int j = 0; j < kFewBlocks; ++j)
#pragma unroll
        for (int i = 0; i < kFewP; ++i) part[wave][j][i][lane] = acc[i][j];
    __syncthreads();
    // wave j finishes block j of 16 rows
    if (wave >= kFewBlocks) return;
    const uint32_t m = (uint32_t)tile.begin + wave * 16 + (lane & 15);
    if (m >= (uint32_t)tile.end) return;
    const float xm = xs[m];
    const float* const wse = ws + first;
    f32x4 v[kFewP];
#pragma unroll
    for (int i = 0; i < kFewP; ++i) {
        i32x4 sum = part[0][wave][i][lane];
#pragma unroll
        for (int u = 1; u < kFewWaves; ++u) sum += part[u][wave][i][lane];
        const int n = n0 + i % kOut * 16 + 4 * (lane >> 4);
        v[i] = scaled(sum, xm, scales4(wse + (i < kOut ? 0 : N), n, N));
    }
#pragma unroll
    for (int i = 0; i < kOut; ++i) {
        const int n = n0 + i * 16 + 4 * (lane >> 4);
        if (n >= N) return;
        if constexpr (kSwiglu) {
            f32x4 h;
#pragma unroll
            for (int r = 0; r < 4; ++r) h[r] = in_fp32(silu(v[i][r]) * v[kOut + i][r]);
            store4(y + (int64_t)m * N + n, h);
        } else {
            store4(y + (int64_t)m * N + n, v[i]);
        }
    }
}

// An operand across r whose memory holds int8 codes and their scales: as Across
// in LDS, but its values come through registers, restored and rounded to S (the
// matrix instruction's type: what expert_dequantize gives).
template <typename S, int B, int NW, int BK>
struct AcrossCodes {
    typedef Across<B, NW, BK> Whole;
    static constexpr int kLoads = Whole::kLoads, kFragReads = Whole::kFragReads;
    typedef typename Whole::At At;
    typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
    struct Stage {
        u32x2_t c[kLoads];
        float s[kLoads];
    };
    const int8_t* base;
    const float* scales;
    int ld, groups, nr, skip, srow;
    uint32_t voff, soff;

    // groups: scales of a row; 0: one, for all of it.
    __device__ __forceinline__ void init(const int8_t* first, const float* first_scale, int ld_bytes,
                                         int per_row, int reduction, int c0, int nc, int wave,
                                         int lane) {
        base = first + c0;
        scales = first_scale;
        ld = ld_bytes;
        groups = per_row ? per_row : 1;
        nr = reduction;
        skip = c0;
        srow = wave * Whole::kRowsPerLoad + lane / Whole::kRowChunks;
        const int c = (lane & (Whole::kRowChunks - 1)) ^ Whole::swizzle(srow);
        const bool in = c0 + c * 8 < nc;
        const int row = Whole::stage_row(srow);
        voff = in ? (uint32_t)(row * ld) + c * 8 : kOutside;
        soff = in ? (uint32_t)(row * groups + (per_row ? (c0 + c * 8) >> 7 : 0)) * 4 : kOutside;
    }
    __device__ __forceinline__ void fetch(Stage& st, uint32_t k0) const {
        const bool any = k0 < (uint32_t)nr;
        const int rows = min((int)((uint32_t)nr - k0), BK);
        const __amdgpu_buffer_rsrc_t rc = make_rsrc(base + (int64_t)k0 * ld, rows * ld - skip);
        const __amdgpu_buffer_rsrc_t rs =
            make_rsrc(scales + (int64_t)k0 * groups, rows * groups * 4);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int row = Whole::stage_row(j * Whole::kStep);
            st.c[j] = __builtin_bit_cast(
                u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(
                             rc, (int)((any ? voff : kOutside) + row * ld), 0, 0));
            st.s[j] = __builtin_bit_cast(
                float, __builtin_amdgcn_raw_buffer_load_b32(
                           rs, (int)((any ? soff : kOutside) + row * groups * 4), 0, 0));
        }
    }
    __device__ __forceinline__ void store(const Stage& st, lds_char* lds, int wave,
                                          int lane) const {
        typedef __attribute__((address_space(3))) u32x4_t lds_u32x4;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = in_fp32((float)(int8_t)(st.c[j][i >> 2] >> (8 * (i & 3))) * st.s[j]);
            *(lds_u32x4*)(lds + (j * NW + wave) * 1024 + lane * 16) = chunk_from_f32<S>(f);
        }
    }
};

template <typename S, typename D>
__global__ __launch_bounds__(Narrow::kThreads, 2) void wgrad_int8_kernel(
    const S* d_y, const int8_t* x, const float* scales, int groups, ExpertRows er, int K, int N,
    int cols, int rows, D* d_w) {
    typedef Narrow T;
    __shared__ __align__(16) S lp[T::BP * T::BK];
    __shared__ __align__(16) S lq[T::BQ * T::BK];
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
    typedef AcrossCodes<S, T::BP, T::kWaves, T::BK> GP;
    typedef Across<T::BQ, T::kWaves, T::BK> GQ;
    GP gp;
    gp.init(x + (int64_t)s.begin * K, scales + (int64_t)s.begin * (groups ? groups : 1), K, groups,
            count, k0, K, wave, lane);
    GQ gq;
    gq.init(d_y + (int64_t)s.begin * N, N * 2, count, n0, N, wave, lane);
    with_blocks<T::WQ>(N - n0, [&](auto nq) {
        constexpr int NQ = decltype(nq)::value;
        f32x4 acc[T::TP][T::TQ] = {};
        typename GP::At ap;
        typename GQ::At aq;
        ap.init(wp * (T::BP / 2 / T::WP), lane);
        aq.init(wq * 16, lane);
        const int nk = row_tiles<T::BK>(count);
        for (int it = 0; it < nk; ++it) {
            typename GP::Stage st;
            gq.load((lds_char*)lq, (uint32_t)it * T::BK, wave);
            gp.fetch(st, (uint32_t)it * T::BK);
            gp.store(st, (lds_char*)lp, wave, lane);
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            s16x8 p[T::TP], q[NQ];
#pragma unroll
            for (int j = 0; j < NQ; ++j) q[j] = aq.frag((lds_char*)lq, j * 16 * T::WQ, 0);
#pragma unroll
            for (int i = 0; i < T::TP; ++i)
                p[i] = ap.frag((lds_char*)lp, p_step<T::BP, T::WP>(i), 0);
#pragma unroll
            for (int i = 0; i < T::TP; ++i)
#pragma unroll
                for (int j = 0; j < NQ; ++j) acc[i][j] = Mfma<S>::mul(p[i], q[j], acc[i][j]);
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
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

dim3 grid_of(int64_t workgroups) { return dim3((unsigned)workgroups); }

template <typename S, typename T>
hipError_t linear_int8_tiles(const int8_t* x, const float* xs, const int8_t* w, const float* ws,
                             const ExpertRows& er, int K, int N, bool swiglu, bool rotate, S* y,
                             const Launch& L) {
    const int outs = swiglu ? 2 * N : N, cols = (int)tiles_of(outs, T::kTile.outs);
    return launch_kernel(swiglu ? linear_int8_kernel<S, true, T> : linear_int8_kernel<S, false, T>,
                         grid_of(workgroups(er, T::kTile, outs)), dim3(T::kThreads), L, x, xs, w, ws,
                         er, K, N, cols, y, rotate);
}

template <typename S>
hipError_t linear_int8_as(const int8_t* x, const float* xs, const int8_t* w, const float* ws,
                          const ExpertRows& er, int K, int N, bool swiglu, void* y,
                          const Launch& L) {
    S* ys = static_cast<S*>(y);
    const int outs = swiglu ? 2 * N : N;
    const bool rotate = rotates(expected_rows(er), K / 2);
    switch (forward_tiles(er, outs)) {
        case Tiles::kFew:
            return launch_kernel(
                swiglu ? linear_int8_few_kernel<S, true> : linear_int8_few_kernel<S, false>,
                grid_of(workgroups(er, kFewTile, outs)), dim3(kFewThreads), L, x, xs, w, ws, er, K,
                N, (int)tiles_of(outs, kFewTile.outs), ys, rotate);
        case Tiles::kSmall:
            return linear_int8_tiles<S, Small>(x, xs, w, ws, er, K, N, swiglu, rotate, ys, L);
        case Tiles::kWide:
            return linear_int8_tiles<S, Wide>(x, xs, w, ws, er, K, N, swiglu, rotate, ys, L);
        default:
            return hipErrorInvalidValue;  // refused before
    }
}

template <typename S>
hipError_t wgrad_int8_as(const void* d_y, const int8_t* x, const float* scales, int groups,
                         const ExpertRows& er, int K, int N, void* d_w, bool f32_out,
                         const Launch& L) {
    const int cols = (int)tiles_of(K, Narrow::BP), rows = (int)tiles_of(N, Narrow::BQ);
    const dim3 grid = grid_of(weight_workgroups(er, K, N));
    const S* ds = static_cast<const S*>(d_y);
    if (f32_out)
        return launch_kernel(wgrad_int8_kernel<S, float>, grid, dim3(Narrow::kThreads), L, ds, x,
                             scales, groups, er, K, N, cols, rows, static_cast<float*>(d_w));
    return launch_kernel(wgrad_int8_kernel<S, S>, grid, dim3(Narrow::kThreads), L, ds, x, scales,
                         groups, er, K, N, cols, rows, static_cast<S*>(d_w));
}

}  // namespace

hipError_t launch_expert_linear_int8(const int8_t* x, const float* x_scales, const int8_t* w,
                                     const float* w_scales, const ExpertRows& er, int K, int N,
                                     bool swiglu, void* y, int dtype, const Launch& L) {
    if (dtype == MOEDX_F16)
        return linear_int8_as<_Float16>(x, x_scales, w, w_scales, er, K, N, swiglu, y, L);
    return linear_int8_as<__bf16>(x, x_scales, w, w_scales, er, K, N, swiglu, y, L);
}

hipError_t launch_expert_wgrad_int8(const void* d_y, const int8_t* x, const float* x_scales,
                                    int block, int dtype, const ExpertRows& er, int K, int N,
                                    void* d_w, bool f32_out, const Launch& L) {
    const int groups = block ? (K + 127) / 128 : 0;
    if (dtype == MOEDX_F16)
        return wgrad_int8_as<_Float16>(d_y, x, x_scales, groups, er, K, N, d_w, f32_out, L);
    return wgrad_int8_as<__bf16>(d_y, x, x_scales, groups, er, K, N, d_w, f32_out, L);
}

}  // namespace moedx
