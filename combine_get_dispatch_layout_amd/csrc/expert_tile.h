// What the experts' products share beside the tiles' loops (device code): the
// tile shapes and the epilogue's pieces.
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
typedef Shape<256, 128, 2, 32, 3, 3> WeightGrad;
typedef Shape<128, 128, 2, 64, 2, 2> Small;

constexpr bool same(const TileShape& a, const TileShape& b) {
    return a.rows == b.rows && a.outs == b.outs && a.threads == b.threads;
}
static_assert(same(Wide::kTile, kWideTile) && same(Small::kTile, kSmallTile) &&
                  same(WeightGrad::kTile, kWeightTile),
              "the plan's tiles are the kernels'");

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

}  // namespace moedx
