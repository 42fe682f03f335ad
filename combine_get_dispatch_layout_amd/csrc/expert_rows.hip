// Rows in expert order for gfx950: the order itself, the rows moved there and
// back, and the gradients of both moves.
//
// A pair p = t * K + k is a filled slot of topk_idx.  In expert order the
// pairs are sorted by expert and, inside one, by p:
//   row(p) = offsets[e(p)] + #{p' < p : e(p') = e(p)}.
// The order is a counting sort in two launches (one for up to 1024 pairs):
// every tile of pairs counts its experts; then every tile sums the counts it
// needs, all experts' totals and its own prefix, and ranks its pairs.  Ranks
// come from wave ballots (the lanes that hold the same expert), not from
// atomics, so the order is the same on every run.
//
// The moves are bound by memory.  Rows are streamed past the caches (every
// one is read and written once): of 16-byte chunks, one wave per token and 64.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_launch.h"
#include "moedx.h"
#include "numeric.h"
#include "xcd.h"

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

constexpr int kOrderUnroll = kOrderTile / kOrderThreads;

__global__ __launch_bounds__(kOrderThreads) void order_count_kernel(OrderArgs a) {
    __shared__ int32_t hist[kMaxExperts];
    __shared__ int32_t prefix[kMaxRanks];
    const int64_t pairs = (int64_t)a.T * a.K;
    load_prefix(a, prefix);
    for (int e = threadIdx.x; e < a.E; e += kOrderThreads) hist[e] = 0;
    __syncthreads();
    for (int it = 0; it < a.iters; ++it) {
        const int64_t b = ((int64_t)blockIdx.x * a.iters + it) * kOrderTile + threadIdx.x;
        int e[kOrderUnroll];
#pragma unroll
        for (int u = 0; u < kOrderUnroll; ++u)
            e[u] = pair_expert(a, prefix, b + u * kOrderThreads, pairs);
#pragma unroll
        for (int u = 0; u < kOrderUnroll; ++u)
            if (e[u] >= 0) atomicAdd(&hist[e[u]], 1);  // a sum of ones: any order gives it
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kOrderThreads)
        a.tile_counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
}

// Exclusive prefix of v over the workgroup's threads; *total gets the sum.
__device__ __forceinline__ int block_prefix(int v, int32_t* wave_sums, int* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int incl = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d, 64);
        if (lane >= d) incl += o;
    }
    if (lane == 63) wave_sums[wave] = incl;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kOrderWaves; ++w) {
        before += w < wave ? wave_sums[w] : 0;
        sum += wave_sums[w];
    }
    *total = sum;
    return before + incl - v;
}

// Adds an expert's counts in tiles t .. t + N - 1, all asked for at once, to the
// sum over all tiles and, of those before this one, to its own.
template <int N>
__device__ __forceinline__ void add_counts(const int32_t*& at, int E, int t, int& all, int& mine) {
    int c[N];
#pragma unroll
    for (int u = 0; u < N; ++u) c[u] = at[u * E];
    at += N * E;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        all += c[u];
        mine += t + u < (int)blockIdx.x ? c[u] : 0;
    }
}

// Waves take contiguous quarters of the tile, so that ranks ascend with p.
// A wave's lane holds 4 pairs, 64 apart, per kOrderTile pairs of the tile.
__global__ __launch_bounds__(kOrderThreads) void order_rank_kernel(OrderArgs a, int bits) {
    constexpr int kPer = kMaxExperts / kOrderThreads;  // experts t, t + 256, ... of thread t
    __shared__ int32_t base[kOrderWaves][kMaxExperts];
    __shared__ int32_t prefix[kMaxRanks];
    __shared__ int32_t wave_sums[kOrderWaves];
    const int64_t pairs = (int64_t)a.T * a.K;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t span = (int64_t)kOrderTile / kOrderWaves * a.iters;
    const int64_t b = ((int64_t)blockIdx.x * kOrderWaves + wave) * span + lane;
    load_prefix(a, prefix);
    for (int e = threadIdx.x; e < kOrderWaves * kMaxExperts; e += kOrderThreads)
        (&base[0][0])[e] = 0;
    __syncthreads();
    int e[kOrderUnroll];
    for (int it = 0; it < a.iters; ++it) {
        const int64_t i = b + (int64_t)it * (64 * kOrderUnroll);
#pragma unroll
        for (int u = 0; u < kOrderUnroll; ++u) e[u] = pair_expert(a, prefix, i + u * 64, pairs);
#pragma unroll
        for (int u = 0; u < kOrderUnroll; ++u)
            if (e[u] >= 0) atomicAdd(&base[wave][e[u]], 1);
    }
    __syncthreads();
    // Totals over all tiles, and over those before this one.
    int all[kPer], mine[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int x = j * kOrderThreads + threadIdx.x;
        all[j] = mine[j] = 0;
        if (a.tiles == 1) {  // no counts were taken: this tile's are all
            for (int w = 0; w < kOrderWaves; ++w) all[j] += base[w][x];
        } else if (x < a.E) {
            const int32_t* at = a.tile_counts + x;
            int t = 0;
            for (; t + 32 <= a.tiles; t += 32) add_counts<32>(at, a.E, t, all[j], mine[j]);
            for (; t + 8 <= a.tiles; t += 8) add_counts<8>(at, a.E, t, all[j], mine[j]);
            for (; t < a.tiles; ++t) add_counts<1>(at, a.E, t, all[j], mine[j]);
        }
    }
    int filled = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if (j * kOrderThreads >= a.E) break;
        const int x = j * kOrderThreads + threadIdx.x;
        int layer;
        const int at = filled + block_prefix(all[j], wave_sums, &layer);
        filled += layer;
        if (blockIdx.x == 0 && x < a.E) a.expert_offsets[x] = at;
        int p = at + mine[j];
        for (int w = 0; w < kOrderWaves; ++w) {
            const int n = base[w][x];
            base[w][x] = p;
            p += n;
        }
        __syncthreads();
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.expert_offsets[a.E] = filled;
    for (int it = 0; it < a.iters; ++it) {
        const int64_t i0 = b + (int64_t)it * (64 * kOrderUnroll);
        if (a.iters > 1) {  // else they are at hand
#pragma unroll
            for (int u = 0; u < kOrderUnroll; ++u) e[u] = pair_expert(a, prefix, i0 + u * 64, pairs);
        }
#pragma unroll
        for (int u = 0; u < kOrderUnroll; ++u) {
            const int64_t i = i0 + u * 64;
            const uint64_t same = same_lanes(e[u], bits) & __ballot(e[u] >= 0);
            int row = -1;
            if (e[u] >= 0) row = base[wave][e[u]] + __popcll(same & ((1ull << lane) - 1));
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            // the last of them moves the expert on
            if (e[u] >= 0 && (same >> lane) == 1ull) base[wave][e[u]] = row + 1;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (i < pairs) {
                a.row_of_slot[i] = row;
                if (row >= 0) a.slot_of_row[row] = (int32_t)i;
                if (i >= filled) a.slot_of_row[i] = -1;
            }
        }
    }
}

// No pairs at all: every offset is zero.
__global__ __launch_bounds__(kOrderThreads) void order_empty_kernel(OrderArgs a) {
    for (int e = threadIdx.x; e <= a.E; e += kOrderThreads) a.expert_offsets[e] = 0;
}

// One wave per (token, slice of 64 chunks): the chunk is read once and stored
// to every row of the token.  The stores stay in the caches for the product
// that reads the rows next (4096 x 7168 to half of 8 slots: 46 us, 55 us with
// streaming stores), and LDS that nothing touches keeps it to 6 workgroups per
// CU: more rows in flight spread over more of memory (8191 x 7168 to 8 skewed
// slots: 182 us at 4 to 6, 193 at 7, 198 without; 2 to 14 chunks per lane 195
// to 205).
constexpr int kSortWorkgroupsPerCu = 6;

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
    const u32x4_t v = __builtin_nontemporal_load(x + (int64_t)t * chunks + min(c, chunks - 1));
    uint64_t m = __ballot(row >= 0 && row < n_rows);
    while (m) {
        const int k = __builtin_ctzll(m);
        m &= m - 1;
        const int64_t r = __builtin_amdgcn_readlane(row, k);
        if (c < chunks) rows[r * chunks + c] = v;
    }
}

// The next NB filled slots of *m: all their chunks are loaded, then added.
template <typename S, int NB>
__device__ __forceinline__ void unsort_batch(const u32x4_t* __restrict__ rows, int chunks, int c,
                                             int row, float w, uint64_t* m,
                                             float (&acc)[Chunk<S>::kN]) {
    constexpr int N = Chunk<S>::kN;
    u32x4_t v[NB];
    float wt[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int k = __builtin_ctzll(*m);
        *m &= *m - 1;
        const int64_t r = __builtin_amdgcn_readlane(row, k);
        wt[b] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), k));
        v[b] = __builtin_nontemporal_load(rows + r * chunks + c);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        float f[N];
        chunk_to_f32<S>(v[b], f);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(wt[b], f[i], acc[i]);
    }
}

// One wave per (token, slice): out = sum over the filled slots, in ascending
// slot order, of weight * row, in fp32 from +0; one rounding.  Workgroups go to
// the XCDs in short runs, so that a token's slots and weights stay in one L2.
constexpr int kUnsortRunLog2 = 4;

template <typename S>
__global__ __launch_bounds__(kRowThreads) void expert_unsort_kernel(
    const u32x4_t* __restrict__ rows, int T, int K, int chunks, int64_t n_rows,
    const int32_t* __restrict__ row_of_slot, const float* __restrict__ weights,
    u32x4_t* __restrict__ out, RowSplit rs) {
    constexpr int N = Chunk<S>::kN;
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(
        xcd_run_block<kUnsortRunLog2>((int)blockIdx.x, (int)gridDim.x) * kRowWavesPerBlock +
        (int)(threadIdx.x >> 6));
    const int t = (int)rs.div.div((uint32_t)wv);
    if (t >= T) return;
    const int c = (wv - t * rs.split) * 64 + lane;
    const int at = min(c, chunks - 1);  // lanes past the row's end store nothing
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
    while (__popcll(m) >= 4) unsort_batch<S, 4>(rows, chunks, at, row, w, &m, acc);
    if (__popcll(m) >= 2) unsort_batch<S, 2>(rows, chunks, at, row, w, &m, acc);
    if (m) unsort_batch<S, 1>(rows, chunks, at, row, w, &m, acc);
    if (c < chunks)
        __builtin_nontemporal_store(chunk_from_f32<S>(acc), out + (int64_t)t * chunks + c);
}

// One wave per row, in row order: the row and its gradient pass as two
// streams, and its token's d_out comes from the caches after the first of the
// token's rows; the dot product ends in the wave.  16384 x 4096 x top-6: 1.75
// GB in 334 us (5.2 TB/s); by token, with d_out held and the rows gathered, 346
// us, and with cached instead of streaming stores 343 us.  (All-zero data takes
// 290 us: what memory reaches depends on the bits.)
//
// A turn of the loop takes kBackChunks chunks per lane.  fp32 has their loads in
// flight together (43 registers); for bf16 and fp16 the compiler moves each pair
// of loads behind the end-of-row test, so that a lane loads, waits and stores
// chunk by chunk (27 and 21 registers), and only other waves cover the wait.
constexpr int kBackChunks = 4;

template <typename S>
__global__ __launch_bounds__(kRowThreads) void expert_unsort_backward_kernel(
    const u32x4_t* __restrict__ d_out, const u32x4_t* __restrict__ rows, int K, FastDiv by_k,
    int chunks, int n_rows, const int32_t* __restrict__ row_of_slot,
    const int32_t* __restrict__ slot_of_row, const float* __restrict__ weights,
    u32x4_t* __restrict__ d_rows, float* __restrict__ d_weights) {
    constexpr int N = Chunk<S>::kN, C = kBackChunks;
    const int r = row_wave();
    if (r >= n_rows) return;
    const int lane = threadIdx.x & 63;
    // pair r, if its slot is empty (or its row outside), has no row to get its
    // gradient from
    if (lane == 0 && (uint32_t)row_of_slot[r] >= (uint32_t)n_rows) d_weights[r] = 0.0f;
    const int slot = slot_of_row[r];
    if (slot < 0 || slot >= n_rows) return;
    const float w = weights[slot];
    const u32x4_t* d0 = d_out + (int64_t)by_k.div((uint32_t)slot) * chunks;
    const u32x4_t* y0 = rows + (int64_t)r * chunks;
    u32x4_t* g0 = d_rows + (int64_t)r * chunks;
    float dot = 0.0f;
    for (int c0 = lane; c0 < chunks; c0 += 64 * C) {
        u32x4_t dv[C], yv[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = min(c0 + 64 * i, chunks - 1);
            yv[i] = __builtin_nontemporal_load(y0 + c);
            dv[i] = d0[c];
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (c0 + 64 * i >= chunks) break;
            float d[N], y[N];
            chunk_to_f32<S>(dv[i], d);
            chunk_to_f32<S>(yv[i], y);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                dot = fmaf(d[j], y[j], dot);
                d[j] *= w;
            }
            __builtin_nontemporal_store(chunk_from_f32<S>(d), g0 + c0 + 64 * i);
        }
    }
    dot = wave_sum(dot);
    if (lane == 0) d_weights[slot] = dot;
}

}  // namespace

hipError_t launch_expert_order(const OrderArgs& a, const Launch& L) {
    if (a.tiles == 0)
        return launch_kernel(order_empty_kernel, dim3(1), dim3(kOrderThreads), L, a);
    int bits = 0;
    while ((1 << bits) < a.E) ++bits;
    const bool counted = a.tiles > 1;
    if (counted) {
        const hipError_t e = launch_kernel(order_count_kernel, dim3(a.tiles), dim3(kOrderThreads),
                                           Launch{L.stream, L.start, nullptr, 0u}, a);
        if (e != hipSuccess) return e;
    }
    return launch_kernel(order_rank_kernel, dim3(a.tiles), dim3(kOrderThreads),
                         Launch{L.stream, counted ? nullptr : L.start, L.stop, 0u}, a, bits);
}

hipError_t launch_expert_sort(const void* x, int T, int K, int64_t row_bytes,
                              const int32_t* row_of_slot, void* rows, const Launch& L) {
    const int chunks = (int)(row_bytes / 16);
    const int slices = (chunks + 63) / 64;
    Launch capped = L;
    capped.lds_bytes = occupancy_lds(kSortWorkgroupsPerCu, 0);
    return launch_kernel(expert_sort_kernel, dim3((int)row_blocks(T, slices)), dim3(kRowThreads),
                         capped, static_cast<const u32x4_t*>(x), T, K, chunks, (int64_t)T * K,
                         row_of_slot, static_cast<u32x4_t*>(rows), make_row_split(chunks, slices));
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
hipError_t unsort_backward_as(const void* d_out, const void* rows, int T, int K, int H,
                              const int32_t* row_of_slot, const int32_t* slot_of_row,
                              const float* weights, void* d_rows, float* d_weights,
                              const Launch& L) {
    return launch_kernel(expert_unsort_backward_kernel<S>, dim3((int)row_blocks(T, K)),
                         dim3(kRowThreads), L, static_cast<const u32x4_t*>(d_out),
                         static_cast<const u32x4_t*>(rows), K, make_fastdiv((uint32_t)K),
                         H / Chunk<S>::kN, T * K, row_of_slot, slot_of_row, weights,
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
                                         const int32_t* slot_of_row, const float* weights,
                                         void* d_rows, float* d_weights, const Launch& L) {
    const auto as = dtype == MOEDX_F32   ? unsort_backward_as<float>
                    : dtype == MOEDX_F16 ? unsort_backward_as<_Float16>
                                         : unsort_backward_as<__bf16>;
    return as(d_out, rows, T, K, H, row_of_slot, slot_of_row, weights, d_rows, d_weights, L);
}

}  // namespace moedx
