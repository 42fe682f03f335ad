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

constexpr int kStream = 2;  // a load's policy: past the caches

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

typedef Shape<128, 128, 2, 64, 3, 2> Deep;  // 80 KB of LDS: two workgroups share a CU
static_assert(same(Deep::kTile, kSmallTile), "the plan's tile is the kernel's");

// A value in LDS that no load on its way into LDS writes: told so, the compiler
// does not wait for those.
template <typename V>
__device__ __forceinline__ V in_lds(const lds_char* __restrict at) {
    return *(const __attribute__((address_space(3))) V*)at;
}

// The lane, as known from here on: neither it nor what is computed from it is kept
// in registers from before.
__device__ __forceinline__ int lane_here() {
    int zero = 0;
    asm volatile("" : "+v"(zero));
    return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, zero));
}

// Tiles of 256 x 256, one workgroup per CU, and of 128 x 128, two.  A workgroup goes
// through tiles: under one's last products the next one's first two stages are
// asked for, and its outputs are on their way to memory while the next one
// multiplies its first stage.  64 experts, us, a workgroup to each tile and this
// way: 192 rows, 1424 -> 4096: 133, 123; 512 rows, 2048 -> 7168: 479, 450; 256 rows,
// 4096 -> 2 x 2048, gated: 324, 303; 512 rows, 7168 -> 2 x 2048, gated: 822, 815 (power
// bounds it: 2360 TOP/s; one expert of 8192 rows, 8192 -> 8192: 388, 384, 2860
// TOP/s); 128 x 128: 48 rows, 2048 -> 1408: 41.8, 39.1; 64 rows, 4096 -> 2048: 91.9, 88.7.
// In the first of each pair for 256 x 256 loads past a reduction's last stage
// start over; left out (kStop), they save the first two products 3 and 7 of these
// us, and 48 rows, 2048 -> 1408, 44.5 to 41.8.
//
// Outputs change lanes in LDS and are stored past the caches, as whole cache lines
// (half ones in 128 x 128 tiles), the scales come through LDS.  With a workgroup
// to each tile, in 64-byte pieces through the caches, as lines through them and
// past them: 192 rows, 1424 -> 4096: 157, 152, 143 (the scales asked for at once: 134);
// 64 rows, 4096 -> 4096: 207, 205, 181.
//
// Waits count loads and stores in order, so every tile issues the same number:
// stores of rows that it does not have fall outside its descriptor's range, as do
// those ahead of the first tile.
template <typename S, bool kSwiglu, typename T, int kPolicy>
__global__ __launch_bounds__(T::kThreads, 2) void linear_int8_kernel(
    const int8_t* x, const float* xs, const int8_t* w, const float* ws, ExpertRows er, int K, int N,
    int cols, S* y, bool rotate, int total) {
    constexpr int kP = T::kP, kQ = T::kQ;
    constexpr int kPBytes = T::BP * T::BK * 2, kQBytes = T::BQ * T::BK * 2;
    // A wave's strip of 16 rows, and the scales of its rows and outputs.
    constexpr int kRun = T::BP / 2 / T::WP, kRunBlocks = kRun / 16, kRowBytes = kRun * 2 + 16;
    constexpr int kOwn = 16 * kRowBytes + T::TQ * 64 + 2 * kRun * 4;
    // They have P's last place until the outputs are out, or one of their own.
    constexpr bool kApart = kP == kQ;
    constexpr int kAsked = kApart ? kP : kP - 1;  // stages asked for under the last products
    static_assert(kAsked == 2 && kQ == 2, "as the waits count them");
    static_assert(kApart || T::kWaves * kOwn <= kPBytes, "they fit");
    __shared__ __align__(16) char lds[kP * kPBytes + kQ * kQBytes + (kApart ? T::kWaves * kOwn : 0)];
    lds_char* const lp = (lds_char*)lds;
    lds_char* const lq = lp + kP * kPBytes;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wp = wave % T::WP, wq = wave / T::WP;
    const int nk = (K / 2 + T::BK - 1) / T::BK;
    constexpr int kOuts = kSwiglu ? T::BP / 2 : T::BP;

    int blk = 0;
    TileSearch search(er);
    const auto tile_at = [&](int v, const TileSearch::Entries& n, int ln) {
        if (v >= total) return RowTile{-1, 0, 0, 0};
        blk = xcd_run_block<kRunLog2>(v, total);
        return search.find<T::BQ, kRowGroup>(er, n, ln, blk, cols);
    };
    typedef Along<T::BP, T::kWaves, T::BK, kSwiglu ? 2 : 1, kPolicy> GP;
    typedef Along<T::BQ, T::kWaves, T::BK, 1> GQ;
    GP gp;
    GQ gq;
    gp.init(K, K / 2, wave, lane);
    gq.init(K, K / 2, wave, lane);
    int shift = 0;
    const auto aim = [&](const RowTile& t) {
        const int n0 = t.col * kOuts;
        const int8_t* const we = w + ((int64_t)t.e * (kSwiglu ? 2 : 1) * N + n0) * K;
        gp.half(0, we, N - n0);
        if constexpr (kSwiglu) gp.half(1, we + (int64_t)N * K, N - n0);
        gq.half(0, x + (int64_t)t.begin * K, t.end - t.begin);
        shift = rotate ? scattered(blk, nk) : 0;
    };
    const auto place = [&](int i) {
        return (i >= nk ? nk : shift + i >= nk ? shift + i - nk : shift + i) * T::BK;
    };
    const auto ask = [&] {
#pragma unroll
        for (int i = 0; i < kAsked; ++i) {
            if (i < kQ) gq.load(lq + i * kQBytes, place(i), wave);
            __builtin_amdgcn_sched_barrier(0);
            gp.load(lp + i * kPBytes, place(i), wave);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    const auto ask_last = [&] {
        if constexpr (!kApart) gp.load(lp + (kP - 1) * kPBytes, place(kP - 1), wave);
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int kStage = GQ::kLoads + GP::kLoads, kLast = kApart ? 0 : GP::kLoads;

    constexpr int kLanes = kRun / 8, kRows = 64 / kLanes, kHalves = kSwiglu ? 1 : 2;
    constexpr int kStores = T::TQ * kHalves * (16 / kRows);
    typedef S vec4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) vec4 lds_vec4;
    lds_char* const strip = (kApart ? lq + kQ * kQBytes : lp + (kP - 1) * kPBytes) + wave * kOwn;
    lds_char* const own = strip + 16 * kRowBytes;
    lds_char* const own_w = own + T::TQ * 64;
    static_assert(T::TQ == 4, "64 rows: a scale each for a lane");
    const auto load_scale = [&](__amdgpu_buffer_rsrc_t rs, lds_char* to, int i) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)to, 4, i * 4, 0, 0, 0);
    };

    int v = (int)blockIdx.x;
    RowTile tile = tile_at(v, search.ask(lane), lane);
    if (tile.e < 0) return;
    aim(tile);
    ask();
    // the stores of the tile before, as the waits count them: outside any range
#pragma unroll
    for (int i = 0; i < kStores; ++i)
        __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{}, make_rsrc(y, 0), (int)(kOutside + i * 16), 0,
                                               kStream);
    __builtin_amdgcn_sched_barrier(0);
    ask_last();
    for (;;) {
        const RowTile cur = tile;
        with_blocks<T::WQ>(cur.end - cur.begin, [&](auto nq) {
            constexpr int NQ = decltype(nq)::value;
            typedef RingLoop<Codes2, T::BP, T::BQ, T::WP, T::WQ, NQ, kP, kQ, true, GP, GQ, true> Loop;
            const Loop loop(wp, wq, lane_here(), shift, nk);
            i32x4 acc[T::TP][T::TQ] = {};
            s16x8 p0[T::TP], q0[T::TQ], p1[T::TP], q1[T::TQ];
            Loop::template barrier<kStage + kStores + kLast>();
            loop.frags(lp, lq, 0, p0, q0);
            int pb = 0, qb = 0;
            const auto stage = [&](int it) {
                lds_char* const rp = lp + pb * kPBytes;
                lds_char* const rq = lq + qb * kQBytes;
                pb = pb + 1 == kP ? 0 : pb + 1;
                qb = qb + 1 == kQ ? 0 : qb + 1;
                loop.first(rp, rq, p0, q0, p1, q1, acc);
                if (it == 0) Loop::template barrier<kStores + kLast>();
                else Loop::template barrier<kLast>();
                loop.second(gp, gq, lp + pb * kPBytes, lq + qb * kQBytes, rp, rq, it, wave, p0, q0,
                            p1, q1, acc);
            };
            // Small tiles: the compiler takes stage 0 out of the loop (8 experts of 256
            // rows, 7168 -> 4096: 78 us; 81 with it inside); wide ones have no
            // registers for that.
            if constexpr (same(T::kTile, kWideTile)) {
#pragma clang loop unroll(disable)
                for (int it = 0; it + 1 < nk; ++it) stage(it);
            } else {
                for (int it = 0; it + 1 < nk; ++it) stage(it);
            }
            const int ln = lane_here();
            const TileSearch::Entries entries = search.ask(ln);
            loop.first(lp + pb * kPBytes, lq + qb * kQBytes, p0, q0, p1, q1, acc);
            Loop::template barrier<0>();  // no load is in flight, every place has been read
            v += (int)gridDim.x;
            tile = tile_at(v, entries, ln);
            __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt 0, where the compiler sees it
            const int mine = 4 * (ln >> 4);  // this lane's first output of a block of 16
            const int n0 = cur.col * kOuts, rows = cur.end - cur.begin;
            const float* const wse = ws + (int64_t)cur.e * (kSwiglu ? 2 : 1) * N;
            {
                const __amdgpu_buffer_rsrc_t rx = make_rsrc(xs + cur.begin, rows * 4);
                load_scale(rx, own, T::q_at(wq, ln >> 4) + (ln & 15));
                // run after run of the outputs, gate and up in a gated product
                const __amdgpu_buffer_rsrc_t rw =
                    make_rsrc(wse + n0, ((kSwiglu ? 2 * N : N) - n0) * 4);
#pragma unroll
                for (int l = 0; l < 2 * kRun; l += 64) {
                    const int i = l + ln, at = wp * kRun + i % kRun;
                    load_scale(rw, own_w + l * 4, i < kRun ? at : at + (kSwiglu ? N : T::BP / 2));
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            const bool more = tile.e >= 0;
            if (more) {
                aim(tile);
                ask();
            }
            Loop::products(p1, q1, acc);
            __builtin_amdgcn_sched_barrier(0);
            // the scales are here
            if (more) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kAsked * kStage) : "memory");
            else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            const __amdgpu_buffer_rsrc_t out = make_rsrc(y + (int64_t)cur.begin * N, rows * N * 2);
#pragma unroll
            for (int j = 0; j < T::TQ; ++j) {
#pragma unroll
                for (int half = 0; half < kHalves; ++half) {
                    if (j < NQ) {
#pragma unroll
                        for (int b = 0; b < kRunBlocks; ++b) {
                            const int i = half * kRunBlocks + b;
                            const float xm = in_lds<float>(own + (j * 16 + (ln & 15)) * 4);
                            f32x4 f = scaled(acc[i][j], xm,
                                             in_lds<f32x4>(own_w + (i * 16 + mine) * 4));
                            if constexpr (kSwiglu) {
                                const f32x4 u = scaled(
                                    acc[i + kRunBlocks][j], xm,
                                    in_lds<f32x4>(own_w + kRun * 4 + (i * 16 + mine) * 4));
#pragma unroll
                                for (int r = 0; r < 4; ++r) f[r] = in_fp32(silu(f[r]) * u[r]);
                            }
                            vec4 o;
#pragma unroll
                            for (int r = 0; r < 4; ++r) o[r] = (S)f[r];
                            *(lds_vec4*)(strip + (ln & 15) * kRowBytes + (b * 16 + mine) * 2) = o;
                            if constexpr (kSwiglu) __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                    // the wave's own strip: its LDS accesses are in order, the compiler's are
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                    for (int h = 0; h < 16 / kRows; ++h) {
                        const int r = h * kRows + ln / kLanes, c = ln % kLanes;
                        const u32x4_t o = in_lds<u32x4_t>(strip + r * kRowBytes + c * 16);
                        const int m = T::q_at(wq, j) + r;
                        const int n = n0 + T::p_at(wp, half * kRunBlocks) + c * 8;
                        // stores outside have places of their own: the compiler keeps each
                        const uint32_t outside =
                            kOutside + ((j * kHalves + half) * (16 / kRows) + h) * 16;
                        const bool in = j < NQ && n < N;
                        __builtin_amdgcn_raw_buffer_store_b128(
                            o, out, (int)(in ? (uint32_t)(m * N + n) * 2 : outside), 0, kStream);
                    }
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        });
        if (tile.e < 0) break;
        if constexpr (!kApart) {  // every wave has read its strip
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        }
        ask_last();
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS is left in flight
}

// Few rows of few experts: the weights' bytes are all that counts.  A tile has 64
// weight rows (gate and up halves in a gated product) and up to 32 rows of x;
// each of its 4 waves multiplies a quarter of the weight rows with all of x.
// Stages of 128 codes go straight into a ring of 6 LDS buffers, all but one of
// them in flight, the weights in whole cache lines past the caches.  64 experts of
// 7168 -> 4096, one row each: 267 us, the weights at 7.04 TB/s (loaded through the
// caches, in pieces of 64 bytes: 318).
constexpr int kThinRunLog2 = 3;  // as in the 16-bit few-row kernel
struct Thin {
    static constexpr int BP = 64, BQ = 32, kStages = 6, kWaves = 4;
    static constexpr TileShape kTile{BQ, BP, kWaves * 64};  // 72 KB of LDS: two share a CU
};
static_assert(same(Thin::kTile, kNarrowTile), "the plan's tile is the kernel's");

template <typename S, bool kSwiglu>
__global__ __launch_bounds__(Thin::kTile.threads) void linear_int8_thin_kernel(
    const int8_t* x, const float* xs, const int8_t* w, const float* ws, ExpertRows er, int K, int N,
    int cols, S* y, bool rotate) {
    typedef Thin T;
    constexpr int BP = T::BP, BQ = T::BQ, BK = 64, NW = T::kWaves, R = T::kStages;
    constexpr int TP = BP / 64, TQ = BQ / 16;
    constexpr int kPBytes = BP * BK * 2, kQBytes = BQ * BK * 2;
    __shared__ __align__(16) char lds[R * (kPBytes + kQBytes)];
    const int blk = xcd_run_block<kThinRunLog2>((int)blockIdx.x, (int)gridDim.x);
    const RowTile tile = find_block<BQ, kRowGroup>(er, blk, cols);
    if (tile.e < 0) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int kOuts = kSwiglu ? BP / 2 : BP;
    const int n0 = tile.col * kOuts;
    const int64_t first = (int64_t)tile.e * (kSwiglu ? 2 : 1) * N;
    const int rows = tile.end - tile.begin;
    typedef Along<BP, NW, BK, kSwiglu ? 2 : 1, kStream> GP;
    typedef Along<BQ, NW, BK, 1> GQ;
    GP gp;
    gp.init(K, K / 2, wave, lane);
    gp.half(0, w + (first + n0) * K, N - n0);
    if constexpr (kSwiglu) gp.half(1, w + (first + N + n0) * K, N - n0);
    GQ gq;
    gq.init(K, K / 2, wave, lane);
    gq.half(0, x + (int64_t)tile.begin * K, rows);
    typename GP::At ap;
    ap.init(wave * 16, lane);
    typename GQ::At aq;
    aq.init(0, lane);
    const int nk = (K / 2 + BK - 1) / BK, shift = rotate ? scattered(blk, nk) : 0;
    lds_char* const lp = (lds_char*)lds;
    lds_char* const lq = lp + R * kPBytes;
    const auto ask = [&](int it, int buf) {
        int s = it + shift;
        s -= s >= nk ? nk : 0;
        const int k0 = (it < nk ? s : nk) * BK;  // past the last stage: nothing
        gp.load(lp + buf * kPBytes, k0, wave);
        gq.load(lq + buf * kQBytes, k0, wave);
        __builtin_amdgcn_sched_barrier(0);
    };
    i32x4 acc[TP][TQ] = {};
    for (int s = 0; s < R - 1; ++s) ask(s, s);
    int buf = 0;
    for (int it = 0; it < nk; ++it) {
        // this stage has arrived, and every wave has read the one before it
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(
                         (R - 2) * (GP::kLoads + GQ::kLoads))
                     : "memory");
        __builtin_amdgcn_sched_barrier(0);
        const lds_char* const rp = lp + buf * kPBytes;
        const lds_char* const rq = lq + buf * kQBytes;
        s16x8 p[2][TP], q[2][TQ];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
            for (int i = 0; i < TP; ++i) p[kk][i] = ap.frag(rp, i * 64, kk);
#pragma unroll
            for (int j = 0; j < TQ; ++j) q[kk][j] = aq.frag(rq, j * 16, kk);
        }
        ask(it + R - 1, buf == 0 ? R - 1 : buf - 1);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int j = 0; j < TQ; ++j)
#pragma unroll
                for (int i = 0; i < TP; ++i)
                    acc[i][j] = Mfma<Codes2>::mul(p[kk][i], q[kk][j], acc[i][j]);
        buf = buf + 1 == R ? 0 : buf + 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS is left in flight
    __syncthreads();
    // block b of 16 weight rows and q of 16 rows of x: sums[b][q]
    static_assert(BP / 16 * TQ * 1024 <= R * (kPBytes + kQBytes), "the sums fit");
    typedef __attribute__((address_space(3))) i32x4 lds_i32x4;
    lds_i32x4* const sums = (lds_i32x4*)lp;
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
        for (int j = 0; j < TQ; ++j) sums[((i * 4 + wave) * TQ + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    const float* const wse = ws + first;
    constexpr int kBlocks = kOuts / 16;
    for (int t = wave; t < kBlocks * TQ; t += NW) {
        const int b = t % kBlocks, j = t / kBlocks;
        const uint32_t m = (uint32_t)tile.begin + j * 16 + (lane & 15);
        const int n = n0 + b * 16 + 4 * (lane >> 4);
        if (m >= (uint32_t)tile.end || n >= N) continue;
        const float xm = xs[m];
        const i32x4 g = sums[(b * TQ + j) * 64 + lane];
        f32x4 v = scaled(g, xm, scales4(wse, n, N));
        if constexpr (kSwiglu) {
            const i32x4 us = sums[((b + kBlocks) * TQ + j) * 64 + lane];
            const f32x4 u = scaled(us, xm, scales4(wse + N, n, N));
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = in_fp32(silu(v[r]) * u[r]);
        }
        store4(y + (int64_t)m * N + n, v);
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

// The weight gradient's loop with P in codes.  Q's stages go straight into one of
// four LDS buffers, three stages ahead; P's come into registers as far ahead and
// are restored into the other of two LDS buffers one stage ahead, under the
// products.  Buffers are arrays of their own and stages a compile-time place
// among them: then the compiler knows which one a load into LDS writes and adds
// no wait before the reads of another.
template <typename S, int BP, int BQ, int WP, int WQ, int NQ, typename LP, typename LQ>
struct SavedLoop {
    typedef typename Mfma<S>::Acc Acc;
    typedef typename LP::Stage Hold;
    static constexpr int TP = BP / WP / 16, TQ = BQ / WQ / 16;
    static constexpr int kBK = 32, kAhead = 3, kQ = kAhead + 1, kP = 2;
    static constexpr int kStageLoads = LQ::kLoads + 2 * LP::kLoads;
    typename LP::At ap;
    typename LQ::At aq;
    lds_char *lp[kP], *lq[kQ];
    int wave, lane;

    __device__ __forceinline__ SavedLoop(int wp, int wq, int wave_, int lane_)
        : wave(wave_), lane(lane_) {
        ap.init(wp * (BP / WP), lane);
        aq.init(wq * 16, lane);
    }
    // Past this only the kAhead - 1 stages after the next one are in flight.
    static __device__ __forceinline__ void arrive() {
        constexpr int kLeft = (kAhead - 1) * kStageLoads;
        static_assert(kLeft < 64, "the wait's count has 6 bits");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt((kLeft & 15) | (kLeft >> 4) << 14 | 0x70);  // lgkmcnt 0
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
    // Asks for stage `it`, whose place is V.
    template <int V>
    __device__ __forceinline__ void ask(const LP& gp, const LQ& gq, Hold& hold, int it) const {
        gq.load(lq[V % kQ], (uint32_t)it * kBK, wave);
        gp.fetch(hold, (uint32_t)it * kBK);
    }
    // Multiplies stage `it` (place V), restores stage it + 1 and asks for stage it
    // + kAhead.
    template <int V>
    __device__ __forceinline__ void stage(const LP& gp, const LQ& gq, Hold (&hold)[2], int it,
                                          Acc (&acc)[TP][TQ]) const {
        s16x8 p[TP], q[NQ];
#pragma unroll
        for (int j = 0; j < NQ; ++j) q[j] = aq.frag(lq[V % kQ], j * 16 * WQ, 0);
#pragma unroll
        for (int i = 0; i < TP; ++i) p[i] = ap.frag(lp[V % kP], i * 16, 0);
        gp.store(hold[(V + 1) % 2], lp[(V + 1) % kP], wave, lane);
        ask<V + kAhead>(gp, gq, hold[(V + kAhead) % 2], it + kAhead);
        // The products in one go, ahead of the other workgroup's reads and
        // conversions (spread among them instead, by scheduling groups: 5 to 50% slower;
        // without the priority 957 us for 917, 64 experts of 768 rows, 4096 x 2048).
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < TP; ++i)
#pragma unroll
            for (int j = 0; j < NQ; ++j) acc[i][j] = Mfma<S>::mul(p[i], q[j], acc[i][j]);
        __builtin_amdgcn_s_setprio(0);
        arrive();
    }
    // Stages 0 .. kAhead - 1 at places V ..
    template <int V>
    __device__ __forceinline__ void begin(const LP& gp, const LQ& gq, Hold (&hold)[2]) const {
        Hold first;
        ask<V>(gp, gq, first, 0);
        __builtin_amdgcn_sched_barrier(0);
        ask<V + 1>(gp, gq, hold[(V + 1) % 2], 1);
        __builtin_amdgcn_sched_barrier(0);
        ask<V + 2>(gp, gq, hold[(V + 2) % 2], 2);
        __builtin_amdgcn_sched_barrier(0);
        gp.store(first, lp[V % kP], wave, lane);
        arrive();
    }
    __device__ __forceinline__ void run(const LP& gp, const LQ& gq, int nk,
                                        Acc (&acc)[TP][TQ]) const {
        if (nk <= 0) return;
        Hold hold[2];
        // Stages past a multiple of four go first, at the last places, so that the
        // loop always starts at place 0.  Each number has a path of its own: where
        // paths with different loads in flight meet, the compiler waits for all.
        int it = nk % 4;
        if (it == 0) {
            begin<0>(gp, gq, hold);
        } else if (it == 1) {
            begin<3>(gp, gq, hold);
            stage<3>(gp, gq, hold, 0, acc);
        } else if (it == 2) {
            begin<2>(gp, gq, hold);
            stage<2>(gp, gq, hold, 0, acc);
            stage<3>(gp, gq, hold, 1, acc);
        } else {
            begin<1>(gp, gq, hold);
            stage<1>(gp, gq, hold, 0, acc);
            stage<2>(gp, gq, hold, 1, acc);
            stage<3>(gp, gq, hold, 2, acc);
        }
        for (; it < nk; it += 4) {
            stage<0>(gp, gq, hold, it, acc);
            stage<1>(gp, gq, hold, it + 1, acc);
            stage<2>(gp, gq, hold, it + 2, acc);
            stage<3>(gp, gq, hold, it + 3, acc);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS is left in flight
    }
};

// 128 x 256: the P side, which is restored, is the narrow one (256 x 128: 1015 us
// for 966 at 64 experts of 768 rows, 4096 x 2048, 917 by now); two workgroups share a CU.
typedef Shape<128, 256, 2, 32, 2, 4> Saved;
static_assert(same(Saved::kTile, kSavedTile), "the plan's tile is the kernel's");

// Runs f with the number of Q blocks per wave that `rows` rows need, made even.
template <int WQ, typename F>
__device__ __forceinline__ void with_even_blocks(int rows, F&& f) {
    const int n = (rows + 16 * WQ - 1) / (16 * WQ);
    if (n > 6) f(std::integral_constant<int, 8>{});
    else if (n > 4) f(std::integral_constant<int, 6>{});
    else if (n > 2) f(std::integral_constant<int, 4>{});
    else f(std::integral_constant<int, 2>{});
}

// The gradient is written once, as whole cache lines past the caches: a wave's
// sums go through LDS in strips of 16 rows.  64 experts, 4096 x 2048, us per
// call with lines, with 64-byte pieces from the registers, and what writing the
// gradient alone takes at 6.5 TB/s (165; fp32 330):
//   rows each    16       48       96       192      384      768
//   bf16       166 249  195 298  246 368  330 470  597 626  942 975
//   fp32       447 503  425 429  422 539  454 715  788 886 1126 1174
// (both before the products' raised priority, which takes the longest to 917 and
// 1081).
template <typename S, typename D>
__global__ __launch_bounds__(Saved::kThreads, 2) void wgrad_int8_kernel(
    const S* d_y, const int8_t* x, const float* scales, int groups, ExpertRows er, int K, int N,
    int cols, int rows, D* d_w) {
    typedef Saved T;
    __shared__ __align__(16) S lp0[T::BP * T::BK], lp1[T::BP * T::BK];
    __shared__ __align__(16) S lq0[T::BQ * T::BK], lq1[T::BQ * T::BK], lq2[T::BQ * T::BK],
        lq3[T::BQ * T::BK];
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
    AcrossCodes<S, T::BP, T::kWaves, T::BK> gp;
    gp.init(x + (int64_t)s.begin * K, scales + (int64_t)s.begin * (groups ? groups : 1), K, groups,
            count, k0, K, wave, lane);
    Across<T::BQ, T::kWaves, T::BK> gq;
    gq.init(d_y + (int64_t)s.begin * N, N * 2, count, n0, N, wave, lane);
    with_even_blocks<T::WQ>(N - n0, [&](auto nq) {
        constexpr int NQ = decltype(nq)::value;
        f32x4 acc[T::TP][T::TQ] = {};
        SavedLoop<S, T::BP, T::BQ, T::WP, T::WQ, NQ, decltype(gp), decltype(gq)> loop(wp, wq, wave,
                                                                                      lane);
        loop.lp[0] = (lds_char*)lp0;
        loop.lp[1] = (lds_char*)lp1;
        loop.lq[0] = (lds_char*)lq0;
        loop.lq[1] = (lds_char*)lq1;
        loop.lq[2] = (lds_char*)lq2;
        loop.lq[3] = (lds_char*)lq3;
        loop.run(gp, gq, row_tiles<T::BK>(count), acc);
        __syncthreads();  // every wave's reads and loads are done: Q's buffers are free
        lds_char* const mine = wave == 0   ? loop.lq[0]
                               : wave == 1 ? loop.lq[1]
                               : wave == 2 ? loop.lq[2]
                                           : loop.lq[3];
        constexpr int kCols = T::BP / T::WP, kRow = kCols * (int)sizeof(D) + 16;
        constexpr int kLanes = kCols * (int)sizeof(D) / 16, kRows = 64 / kLanes;
        static_assert(2 * 16 * kRow <= T::BQ * T::BK * 2, "two strips in a buffer");
        typedef __attribute__((address_space(3))) u32x4_t lds_u32x4;
        typedef D vec4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) vec4 lds_vec4;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            lds_char* const strip = mine + j % 2 * 16 * kRow;
#pragma unroll
            for (int i = 0; i < T::TP; ++i) {
                vec4 v;
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = (D)acc[i][j][r];
                *(lds_vec4*)(strip + (lane & 15) * kRow +
                             (i * 16 + 4 * (lane >> 4)) * (int)sizeof(D)) = v;
            }
            // the wave's own strip: its LDS accesses are in order, the compiler's are
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int h = 0; h < 16 / kRows; ++h) {
                const int row = h * kRows + lane / kLanes, c = lane % kLanes;
                const u32x4_t v = *(lds_u32x4*)(strip + row * kRow + c * 16);
                const int n = n0 + T::q_at(wq, j) + row;
                const int k = k0 + wp * kCols + c * (16 / (int)sizeof(D));
                if (n < N && k < K)
                    __builtin_nontemporal_store(
                        v, reinterpret_cast<u32x4_t*>(d_w + ((int64_t)e * N + n) * K + k));
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    });
}

dim3 grid_of(int64_t workgroups) { return dim3((unsigned)workgroups); }

template <typename S>
struct Int8Product {
    const int8_t* x;
    const float* xs;
    const int8_t* w;
    const float* ws;
    const ExpertRows& er;
    int K, N;
    bool swiglu;
    S* y;
    const Launch& L;

    int outs() const { return swiglu ? 2 * N : N; }
    hipError_t thin(bool rotate) const {
        return launch_kernel(
            swiglu ? linear_int8_thin_kernel<S, true> : linear_int8_thin_kernel<S, false>,
            grid_of(workgroups(er, kNarrowTile, outs())), dim3(kNarrowTile.threads), L, x, xs, w, ws,
            er, K, N, (int)tiles_of(outs(), kNarrowTile.outs), y, rotate);
    }
    template <typename T, int kPolicy>
    hipError_t tiles(bool rotate) const {
        const int64_t total = workgroups(er, T::kTile, outs());
        return launch_kernel(swiglu ? linear_int8_kernel<S, true, T, kPolicy>
                                    : linear_int8_kernel<S, false, T, kPolicy>,
                             grid_of(workgroups_through(T::kTile, total)), dim3(T::kThreads), L, x, xs,
                             w, ws, er, K, N, (int)tiles_of(outs(), T::kTile.outs), y, rotate,
                             (int)total);
    }
};

template <typename S>
hipError_t linear_int8_as(const int8_t* x, const float* xs, const int8_t* w, const float* ws,
                          const ExpertRows& er, int K, int N, bool swiglu, void* y,
                          const Launch& L) {
    const Int8Product<S> p{x, xs, w, ws, er, K, N, swiglu, static_cast<S*>(y), L};
    const bool rotate = rotates(expected_rows(er), K / 2);
    switch (int8_tiles(er, p.outs())) {
        case Int8Tiles::kNarrow: return p.thin(rotate);
        case Int8Tiles::kOnce: return p.template tiles<Small, kStream>(rotate);
        case Int8Tiles::kDeepOnce: return p.template tiles<Deep, kStream>(rotate);
        case Int8Tiles::kDeep: return p.template tiles<Deep, 0>(rotate);
        case Int8Tiles::kWide: return p.template tiles<Wide, 0>(rotate);
        default: return hipErrorInvalidValue;  // refused before
    }
}

template <typename S>
hipError_t wgrad_int8_as(const void* d_y, const int8_t* x, const float* scales, int groups,
                         const ExpertRows& er, int K, int N, void* d_w, bool f32_out,
                         const Launch& L) {
    const int cols = (int)tiles_of(K, Saved::BP), rows = (int)tiles_of(N, Saved::BQ);
    const dim3 grid = grid_of(weight_workgroups(er, K, N, kSavedTile));
    const S* ds = static_cast<const S*>(d_y);
    if (f32_out)
        return launch_kernel(wgrad_int8_kernel<S, float>, grid, dim3(Saved::kThreads), L, ds, x,
                             scales, groups, er, K, N, cols, rows, static_cast<float*>(d_w));
    return launch_kernel(wgrad_int8_kernel<S, S>, grid, dim3(Saved::kThreads), L, ds, x, scales,
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
