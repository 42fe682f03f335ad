// What the experts' products share beside the tiles' loops (device code): the
// tile shapes, the epilogue's stores, and the loop of a product of few rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "expert_plan.h"
#include "mma_tile.h"
#include "numeric.h"

namespace moedx {

// Tile shapes (mma_tile.h): forward and input gradient 256 x 256 by 8 waves,
// weight gradient 256 x 128 by 4.
template <int BP_, int BQ_, int WQ_, int BK_, int kP_, int kQ_>
struct Shape {
    static constexpr int BP = BP_, BQ = BQ_, WP = 2, WQ = WQ_, BK = BK_;
    static constexpr int kP = kP_, kQ = kQ_;  // stages of either operand in LDS
    static constexpr int kWaves = WP * WQ, kThreads = kWaves * 64;
    static constexpr int TP = BP / WP / 16, TQ = BQ / WQ / 16;
    static constexpr TileShape kTile{BQ, BP, kThreads};
    static __device__ __forceinline__ int p_at(int wp, int i) { return p_block<BP, WP>(wp, i); }
    static __device__ __forceinline__ int q_at(int wq, int j) { return q_block<WQ>(wq, j); }
};
typedef Shape<256, 256, 4, 64, 3, 2> Wide;
typedef Shape<256, 128, 2, 32, 3, 3> Narrow;
typedef Shape<128, 128, 2, 64, 2, 2> Small;

constexpr bool same(const TileShape& a, const TileShape& b) {
    return a.rows == b.rows && a.outs == b.outs && a.threads == b.threads;
}
static_assert(same(Wide::kTile, kWideTile) && same(Small::kTile, kSmallTile) &&
                  same(Narrow::kTile, kWeightTile),
              "the plan's tiles are the kernels'");

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

// Outputs of two neighbouring blocks of 16: the lane groups trade halves, so
// that each lane holds 8 consecutive outputs (16 bytes) and a row's 32 outputs
// are 64 contiguous bytes.  They start pair_at(lane) outputs into the blocks.
template <typename S>
__device__ __forceinline__ u32x4_t pack_pair(const f32x4& a, const f32x4& b) {
    typedef S vec __attribute__((ext_vector_type(4)));
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    vec va, vb;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        va[i] = (S)a[i];
        vb[i] = (S)b[i];
    }
    const u32x2 ua = __builtin_bit_cast(u32x2, va), ub = __builtin_bit_cast(u32x2, vb);
    // swaps the odd rows of 16 lanes of one operand with the even ones of the other
    const auto lo = __builtin_amdgcn_permlane16_swap(ua[0], ub[0], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(ua[1], ub[1], false, false);
    return u32x4_t{lo[0], hi[0], lo[1], hi[1]};
}
__device__ __forceinline__ int pair_at(int lane) {
    return ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
}
template <typename S>
__device__ __forceinline__ void store8(S* at, u32x4_t v) {
    *reinterpret_cast<u32x4_t*>(at) = v;
}

// One of n starting points for tile i, scattered (a multiplicative hash).  Rows
// a multiple of 4 KiB apart start on the same memory channels, and so do
// workgroups that all begin at the reduction's start; where a weight row is
// read by one workgroup only, each may begin elsewhere.  64 experts of 12 rows,
// 4096 -> 4096: 454 us from the start, 366 us scattered.  Where several row
// tiles share the weights, it would cost them the sharing.
__device__ __forceinline__ int scattered(int i, int n) {
    return (int)__umulhi((uint32_t)i * 2654435761u, (uint32_t)n);
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
                                             int wave, int lane,
                                             typename Mfma<S>::Acc (&acc)[kFewP][kFewBlocks]) {
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

}  // namespace moedx
