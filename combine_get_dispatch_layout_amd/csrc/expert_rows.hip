// Rows in expert order for gfx950: the order itself, the rows moved there and
// back, and the gradients of both moves.
//
// A pair p = t * K + k is a filled slot of topk_idx.  In expert order the
// pairs are sorted by expert and, inside one, by p:
//   row(p) = offsets[e(p)] + #{p' < p : e(p') = e(p)}.
// The order is a counting sort: every tile of pairs counts its experts, one
// workgroup turns the counts into prefixes, every tile ranks its pairs.  Ranks
// come from wave ballots (the lanes that hold the same expert), not from
// atomics, so the order is the same on every run.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_launch.h"
#include "moedx.h"
#include "numeric.h"

namespace moedx {

namespace {

constexpr int kOrderThreads = 256;
constexpr int kOrderWaves = kOrderThreads / 64;

// The global expert id of pair i, or -1 (empty, out of range, or a receive row
// past the last one).  prefix: the buckets' inclusive row prefix in LDS.
__device__ __forceinline__ int pair_expert(const OrderArgs& a, const int32_t* prefix, int64_t i,
                                           int64_t pairs) {
    if (i >= pairs) return -1;
    const int64_t e = a.topk_idx[i];
    if (!a.rank_prefix_matrix) return (e >= 0 && e < a.E) ? (int)e : -1;
    const int row = (int)(i / a.K);
    if (e < 0 || e >= a.P || row >= prefix[a.R - 1]) return -1;
    int r = 0;
    while (prefix[r] <= row) ++r;  // the bucket of the row: r < R by the test above
    return r * a.P + (int)e;
}

__device__ __forceinline__ void load_prefix(const OrderArgs& a, int32_t* prefix) {
    if (a.rank_prefix_matrix && (int)threadIdx.x < a.R)
        prefix[threadIdx.x] = a.rank_prefix_matrix[threadIdx.x];
}

// Lanes of this wave whose e equals this lane's (e < 2^bits).
__device__ __forceinline__ uint64_t same_lanes(int e, int bits) {
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const uint64_t s = __ballot((e >> b) & 1);
        m &= ((e >> b) & 1) ? s : ~s;
    }
    return m;
}

__global__ __launch_bounds__(kOrderThreads) void order_count_kernel(OrderArgs a) {
    __shared__ int32_t hist[kMaxExperts];
    __shared__ int32_t prefix[kMaxRanks];
    const int64_t pairs = (int64_t)a.T * a.K;
    const int64_t tile = (int64_t)kOrderTile * a.iters;
    load_prefix(a, prefix);
    for (int e = threadIdx.x; e < a.E; e += kOrderThreads) hist[e] = 0;
    __syncthreads();
    const int64_t b = blockIdx.x * tile;
    for (int64_t i = b + threadIdx.x; i < b + tile; i += kOrderThreads) {
        const int e = pair_expert(a, prefix, i, pairs);
        if (e >= 0) atomicAdd(&hist[e], 1);  // a sum of ones: any order gives it
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kOrderThreads)
        a.tile_counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
}

// One workgroup, thread e per expert: counts become exclusive prefixes over
// the tiles plus the expert's offset.
__global__ __launch_bounds__(kMaxExperts) void order_scan_kernel(OrderArgs a) {
    __shared__ int32_t total[kMaxExperts];
    const int e = threadIdx.x;
    int sum = 0;
    if (e < a.E)
        for (int t = 0; t < a.tiles; ++t) sum += a.tile_counts[(int64_t)t * a.E + e];
    total[e] = sum;
    __syncthreads();
    for (int d = 1; d < kMaxExperts; d <<= 1) {
        const int v = e >= d ? total[e - d] : 0;
        __syncthreads();
        total[e] += v;
        __syncthreads();
    }
    if (e >= a.E) return;
    int at = total[e] - sum;
    a.expert_offsets[e] = at;
    if (e == a.E - 1) a.expert_offsets[a.E] = total[e];
    for (int t = 0; t < a.tiles; ++t) {
        int32_t* c = &a.tile_counts[(int64_t)t * a.E + e];
        const int n = *c;
        *c = at;
        at += n;
    }
}

// Waves take contiguous quarters of the tile, so that ranks ascend with p.
__global__ __launch_bounds__(kOrderThreads) void order_rank_kernel(OrderArgs a, int bits) {
    __shared__ int32_t base[kOrderWaves][kMaxExperts];
    __shared__ int32_t prefix[kMaxRanks];
    const int64_t pairs = (int64_t)a.T * a.K;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t span = (int64_t)kOrderTile / kOrderWaves * a.iters;
    const int64_t b = ((int64_t)blockIdx.x * kOrderWaves + wave) * span;
    load_prefix(a, prefix);
    for (int e = threadIdx.x; e < kOrderWaves * kMaxExperts; e += kOrderThreads)
        (&base[0][0])[e] = 0;
    __syncthreads();
    for (int64_t i = b + lane; i < b + span; i += 64) {
        const int e = pair_expert(a, prefix, i, pairs);
        if (e >= 0) atomicAdd(&base[wave][e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kOrderThreads) {
        int at = a.tile_counts[(int64_t)blockIdx.x * a.E + e];
        for (int w = 0; w < kOrderWaves; ++w) {
            const int n = base[w][e];
            base[w][e] = at;
            at += n;
        }
    }
    __syncthreads();
    const int filled = a.expert_offsets[a.E];
    for (int64_t i0 = b; i0 < b + span; i0 += 64) {
        const int64_t i = i0 + lane;
        const int e = pair_expert(a, prefix, i, pairs);
        const uint64_t same = same_lanes(e, bits) & __ballot(e >= 0);
        int row = -1;
        if (e >= 0) {
            const uint64_t below = same & ((1ull << lane) - 1);
            row = base[wave][e] + __popcll(below);
        }
        __builtin_amdgcn_wave_barrier();
        if (e >= 0 && (same >> lane) == 1ull) base[wave][e] = row + 1;  // the last of them
        __builtin_amdgcn_wave_barrier();
        if (i < pairs) {
            a.row_of_slot[i] = row;
            if (row >= 0) a.slot_of_row[row] = (int32_t)i;
            if (i >= filled) a.slot_of_row[i] = -1;
        }
    }
}

// One wave per (token, slice of 64 chunks): the chunk is read once and stored
// to every row of the token.
__global__ __launch_bounds__(kRowThreads) void expert_sort_kernel(
    const u32x4_t* __restrict__ x, int T, int K, int chunks, int64_t n_rows,
    const int32_t* __restrict__ row_of_slot, u32x4_t* __restrict__ rows, RowSplit rs) {
    int t, part;
    row_part(rs, &t, &part);
    if (t >= T) return;
    const int lane = threadIdx.x & 63;
    const int c = part * 64 + lane;
    int row = -1;
    if (lane < K) row = row_of_slot[(int64_t)t * K + lane];
    u32x4_t v{};
    if (c < chunks) v = x[(int64_t)t * chunks + c];
    uint64_t m = __ballot(row >= 0 && row < n_rows);
    while (m) {
        const int k = __builtin_ctzll(m);
        m &= m - 1;
        const int64_t r = __builtin_amdgcn_readlane(row, k);
        if (c < chunks) rows[r * chunks + c] = v;
    }
}

// One wave per (token, slice): out = sum over the filled slots, in ascending
// slot order, of weight * row, in fp32 from +0; one rounding.
template <typename S>
__global__ __launch_bounds__(kRowThreads) void expert_unsort_kernel(
    const u32x4_t* __restrict__ rows, int T, int K, int chunks, int64_t n_rows,
    const int32_t* __restrict__ row_of_slot, const float* __restrict__ weights,
    u32x4_t* __restrict__ out, RowSplit rs) {
    constexpr int N = Chunk<S>::kN;
    int t, part;
    row_part(rs, &t, &part);
    if (t >= T) return;
    const int lane = threadIdx.x & 63;
    const int c = part * 64 + lane;
    int row = -1;
    float w = 1.0f;
    if (lane < K) {
        row = row_of_slot[(int64_t)t * K + lane];
        if (weights) w = weights[(int64_t)t * K + lane];
    }
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    uint64_t m = __ballot(row >= 0 && row < n_rows);
    while (m) {
        const int k = __builtin_ctzll(m);
        m &= m - 1;
        const int64_t r = __builtin_amdgcn_readlane(row, k);
        const float wk = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), k));
        if (c < chunks) {
            float f[N];
            chunk_to_f32<S>(rows[r * chunks + c], f);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(wk, f[i], acc[i]);
        }
    }
    if (c < chunks) out[(int64_t)t * chunks + c] = chunk_from_f32<S>(acc);
}

// One workgroup per token: d_rows[row] = w * d_out and the dot product of
// d_out with the row, which is read in the same pass.
constexpr int kBackThreads = 256;

template <typename S>
__global__ __launch_bounds__(kBackThreads) void expert_unsort_backward_kernel(
    const u32x4_t* __restrict__ d_out, const u32x4_t* __restrict__ rows, int K, int chunks,
    int64_t n_rows, const int32_t* __restrict__ row_of_slot, const float* __restrict__ weights,
    u32x4_t* __restrict__ d_rows, float* __restrict__ d_weights) {
    constexpr int N = Chunk<S>::kN;
    __shared__ float part[kBackThreads / 64][kMaxTopk];
    const int t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int k = 0; k < K; ++k) {
        const int64_t r = row_of_slot[(int64_t)t * K + k];
        float dot = 0.0f;
        if (r >= 0 && r < n_rows) {
            const float w = weights[(int64_t)t * K + k];
            for (int c = threadIdx.x; c < chunks; c += kBackThreads) {
                float d[N], y[N];
                chunk_to_f32<S>(d_out[(int64_t)t * chunks + c], d);
                chunk_to_f32<S>(rows[r * chunks + c], y);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    dot = fmaf(d[i], y[i], dot);
                    d[i] *= w;
                }
                d_rows[r * chunks + c] = chunk_from_f32<S>(d);
            }
        }
        dot = wave_sum(dot);
        if (lane == 0) part[wave][k] = dot;
    }
    __syncthreads();
    if ((int)threadIdx.x < K) {
        float s = 0.0f;
        for (int i = 0; i < kBackThreads / 64; ++i) s += part[i][threadIdx.x];
        d_weights[(int64_t)t * K + threadIdx.x] = s;
    }
}

}  // namespace

hipError_t launch_expert_order(const OrderArgs& a, const Launch& L) {
    const Launch first{L.stream, L.start, nullptr, 0u}, mid{L.stream, nullptr, nullptr, 0u},
        last{L.stream, nullptr, L.stop, 0u};
    hipError_t e = hipSuccess;
    if (a.tiles > 0) e = launch_kernel(order_count_kernel, dim3(a.tiles), dim3(kOrderThreads), first, a);
    if (e == hipSuccess)
        e = launch_kernel(order_scan_kernel, dim3(1), dim3(kMaxExperts), a.tiles > 0 ? mid : L, a);
    if (e != hipSuccess || a.tiles == 0) return e;
    int bits = 0;
    while ((1 << bits) < a.E) ++bits;
    return launch_kernel(order_rank_kernel, dim3(a.tiles), dim3(kOrderThreads), last, a, bits);
}

hipError_t launch_expert_sort(const void* x, int T, int K, int64_t row_bytes,
                              const int32_t* row_of_slot, void* rows, const Launch& L) {
    const int chunks = (int)(row_bytes / 16);
    const int slices = (chunks + 63) / 64;
    return launch_kernel(expert_sort_kernel, dim3((int)row_blocks(T, slices)), dim3(kRowThreads), L,
                         static_cast<const u32x4_t*>(x), T, K, chunks, (int64_t)T * K, row_of_slot,
                         static_cast<u32x4_t*>(rows), make_row_split(chunks, slices));
}

namespace {

template <typename S>
hipError_t unsort_as(const void* rows, int T, int K, int chunks, const int32_t* row_of_slot,
                     const float* weights, void* out, const Launch& L) {
    const int slices = (chunks + 63) / 64;
    return launch_kernel(expert_unsort_kernel<S>, dim3((int)row_blocks(T, slices)),
                         dim3(kRowThreads), L, static_cast<const u32x4_t*>(rows), T, K, chunks,
                         (int64_t)T * K, row_of_slot, weights, static_cast<u32x4_t*>(out),
                         make_row_split(chunks, slices));
}

template <typename S>
hipError_t unsort_backward_as(const void* d_out, const void* rows, int T, int K, int chunks,
                              const int32_t* row_of_slot, const float* weights, void* d_rows,
                              float* d_weights, const Launch& L) {
    return launch_kernel(expert_unsort_backward_kernel<S>, dim3(T), dim3(kBackThreads), L,
                         static_cast<const u32x4_t*>(d_out), static_cast<const u32x4_t*>(rows), K,
                         chunks, (int64_t)T * K, row_of_slot, weights,
                         static_cast<u32x4_t*>(d_rows), d_weights);
}

}  // namespace

hipError_t launch_expert_unsort(const void* rows, int dtype, int T, int K, int H,
                                const int32_t* row_of_slot, const float* weights, void* out,
                                const Launch& L) {
    if (dtype == MOEDX_F32)
        return unsort_as<float>(rows, T, K, H / 4, row_of_slot, weights, out, L);
    if (dtype == MOEDX_F16)
        return unsort_as<_Float16>(rows, T, K, H / 8, row_of_slot, weights, out, L);
    return unsort_as<__bf16>(rows, T, K, H / 8, row_of_slot, weights, out, L);
}

hipError_t launch_expert_unsort_backward(const void* d_out, const void* rows, int dtype, int T,
                                         int K, int H, const int32_t* row_of_slot,
                                         const float* weights, void* d_rows, float* d_weights,
                                         const Launch& L) {
    if (dtype == MOEDX_F32)
        return unsort_backward_as<float>(d_out, rows, T, K, H / 4, row_of_slot, weights, d_rows,
                                         d_weights, L);
    if (dtype == MOEDX_F16)
        return unsort_backward_as<_Float16>(d_out, rows, T, K, H / 8, row_of_slot, weights, d_rows,
                                            d_weights, L);
    return unsort_backward_as<__bf16>(d_out, rows, T, K, H / 8, row_of_slot, weights, d_rows,
                                      d_weights, L);
}

}  // namespace moedx
