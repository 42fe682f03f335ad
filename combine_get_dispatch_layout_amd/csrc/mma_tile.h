// One output tile of a product on the matrix cores (device code).
//
//   D[q, p] = sum_r P(p, r) Q(q, r)
//
// p is the output's contiguous dimension (BP of it per tile), q its row
// dimension (BQ), r the reduction, taken 64 at a time.  An operand is either
// "along" (its memory runs along r: [B rows][64 r]) or "across" (its memory
// runs along p or q: [64 r][B columns]).  Stages of both operands go from
// global memory straight into LDS; the buffer descriptors' range gives zeros
// for rows past an operand's end, so ragged tiles need no branch.
//
// LDS holds 16-byte chunks, permuted so that the reads of a wave spread over
// the banks.  Along: row r's chunk c sits at c ^ (r & 7), read with 16-byte
// loads, 8 reduction values of one row per lane.  Across: row r's chunk c sits
// at c ^ 2 f(r); the transposing LDS read hands a lane 4 reduction values of
// one column, so a column-major operand costs no pass of its own.
//
// The matrix instruction is 16 x 16 x 32 with P as its A operand: a lane ends
// up with 4 consecutive p of one q.  Two LDS buffers alternate.  A stage is
// multiplied in two halves of 32: while the first half's products run, the
// second half is read, then the stage after next starts loading into the
// buffer just read, and the next stage's first half is read under the second
// half's products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moedx {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

template <typename S>
struct Mfma;
template <>
struct Mfma<__bf16> {
    typedef __bf16 vec __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 mul(s16x8 a, s16x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(vec, a),
                                                       __builtin_bit_cast(vec, b), c, 0, 0, 0);
    }
};
template <>
struct Mfma<_Float16> {
    typedef _Float16 vec __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 mul(s16x8 a, s16x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(vec, a),
                                                      __builtin_bit_cast(vec, b), c, 0, 0, 0);
    }
};

constexpr int kBK = 64;  // reduction values per stage

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0,
                                             (int)(bytes > 0 ? bytes : 0), 0x00020000);
}

constexpr uint32_t kOutside = 0x80000000u;  // past any descriptor's range (below 2^31 bytes)

// An operand along r: `halves` blocks of B / halves rows, each with its own
// first row (a gated product's gate and up rows), ld values per row.
template <int B, int NW, int kHalves>
struct Along {
    static constexpr int kLoads = B / (8 * NW);  // 16-byte loads per lane and stage
    static_assert(B % (8 * NW * kHalves) == 0, "a wave's 8 rows lie in one half");
    const char* base[kHalves];
    int valid[kHalves];  // rows of each half inside the operand
    int64_t ld2;         // bytes per row
    int nr;              // reduction length
    uint32_t voff[kLoads / kHalves];
    int col;             // this lane's first reduction value within a stage

    __device__ __forceinline__ void init(int64_t ld_bytes, int reduction, int wave, int lane) {
        ld2 = ld_bytes;
        nr = reduction;
        const int r = wave * 8 + (lane >> 3);
        const int c = (lane & 7) ^ ((lane >> 3) & 7);
        col = c * 8;
#pragma unroll
        for (int j = 0; j < kLoads / kHalves; ++j)
            voff[j] = (uint32_t)((r + j * 8 * NW) * ld2) + c * 16;
    }
    __device__ __forceinline__ void half(int h, const void* first, int rows) {
        base[h] = static_cast<const char*>(first);
        valid[h] = min(max(rows, 0), B / kHalves);
    }
    // Stage at reduction value k0 into lds (this wave's part of it).
    template <typename S>
    __device__ __forceinline__ void load(S* lds, int k0, int wave) const {
        const uint32_t out = k0 + col < nr ? 0u : kOutside;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            const int64_t bytes = valid[h] * ld2 - (int64_t)k0 * 2;
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(base[h] + (int64_t)k0 * 2, bytes);
#pragma unroll
            for (int j = 0; j < kLoads / kHalves; ++j) {
                const int row = h * (B / kHalves) + (j * NW + wave) * 8;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rs, (lds_void*)(lds + row * kBK), 16, (int)(voff[j] | out), 0, 0, 0);
            }
        }
    }
    // Lane's 8 reduction values (half kk) of row `row` (+ lane & 15).
    template <typename S>
    static __device__ __forceinline__ s16x8 frag(const S* lds, int row, int kk, int lane) {
        const int r = row + (lane & 15);
        const int c = (kk * 4 + (lane >> 4)) ^ (r & 7);
        return *reinterpret_cast<const s16x8*>(lds + r * kBK + c * 8);
    }
};

// An operand across r: 64 rows of the reduction, B columns from column c0 of
// nc; ld values per row.
template <int B, int NW>
struct Across {
    static constexpr int kLoads = B / (8 * NW);
    static constexpr int kRowChunks = B / 8;           // 16-byte chunks per LDS row
    static constexpr int kRowsPerLoad = 64 / kRowChunks;  // LDS rows one wave load fills
    static constexpr int kUnits = B / 16;              // 32-byte units per LDS row
    static_assert(kRowChunks <= 64, "an LDS row is one wave load at most");
    const char* base;
    int64_t ld2;
    int nr;
    int skip2;  // bytes before column c0
    uint32_t voff[kLoads];

    static __device__ __forceinline__ int swizzle(int row) {
        return (((row & 3) | ((row >> 1) & 12)) & (kUnits - 1)) * 2;
    }
    __device__ __forceinline__ void init(const void* first, int64_t ld_bytes, int reduction,
                                         int c0, int nc, int wave, int lane) {
        base = static_cast<const char*>(first) + (int64_t)c0 * 2;
        ld2 = ld_bytes;
        nr = reduction;
        skip2 = c0 * 2;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int row = (j * NW + wave) * kRowsPerLoad + lane / kRowChunks;
            const int c = (lane & (kRowChunks - 1)) ^ swizzle(row);
            voff[j] = (uint32_t)(row * ld2) + c * 16;
            if (c0 + c * 8 >= nc) voff[j] = kOutside;
        }
    }
    template <typename S>
    __device__ __forceinline__ void load(S* lds, int k0, int wave) const {
        const int rows = min(nr - k0, kBK);
        const __amdgpu_buffer_rsrc_t rs =
            make_rsrc(base + (int64_t)k0 * ld2, rows > 0 ? rows * ld2 - skip2 : 0);
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rs, (lds_void*)(lds + (j * NW + wave) * 512), 16, (int)voff[j], 0, 0, 0);
    }
    template <typename S>
    static __device__ __forceinline__ s16x8 frag(const S* lds, int col, int kk, int lane) {
        s16x8 v;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = kk * 32 + (lane >> 4) * 8 + h * 4 + ((lane >> 2) & 3);
            const int c = (col / 8 + ((lane >> 1) & 1)) ^ swizzle(row);
            const S* at = lds + row * B + c * 8 + (lane & 1) * 4;
            const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
            v[4 * h] = t[0];
            v[4 * h + 1] = t[1];
            v[4 * h + 2] = t[2];
            v[4 * h + 3] = t[3];
        }
        return v;
    }
};

// Waves of a tile: WP x WQ.  Wave (wp, wq) has the P blocks of 16 at
//   p = (i / (TP / 2)) * BP / 2 + wp * BP / 2 / WP + (i % (TP / 2)) * 16
// (its share of both halves of the tile) and the Q blocks at
//   q = j * 16 * WQ + wq * 16
// (dealt out in turn, so that a tile with few rows keeps every wave equally
// busy and leaves out whole blocks).
template <int BP, int WP>
__device__ __forceinline__ int p_block(int wp, int i) {
    constexpr int TP = BP / WP / 16;
    return (i / (TP / 2)) * (BP / 2) + wp * (BP / 2 / WP) + (i % (TP / 2)) * 16;
}
template <int WQ>
__device__ __forceinline__ int q_block(int wq, int j) {
    return j * 16 * WQ + wq * 16;
}

template <typename S, int BP, int BQ, int WP, int WQ, int NQ, typename LP, typename LQ>
struct TileLoop {
    static constexpr int TP = BP / WP / 16, TQ = BQ / WQ / 16;

    static __device__ __forceinline__ void frags(const S* lp, const S* lq, int kk, int wp, int wq,
                                                 int lane, s16x8 (&p)[TP], s16x8 (&q)[TQ]) {
#pragma unroll
        for (int i = 0; i < TP; ++i) p[i] = LP::frag(lp, p_block<BP, WP>(wp, i), kk, lane);
#pragma unroll
        for (int j = 0; j < NQ; ++j) q[j] = LQ::frag(lq, q_block<WQ>(wq, j), kk, lane);
    }
    static __device__ __forceinline__ void products(const s16x8 (&p)[TP], const s16x8 (&q)[TQ],
                                                    f32x4 (&acc)[TP][TQ]) {
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int i = 0; i < TP; ++i) acc[i][j] = Mfma<S>::mul(p[i], q[j], acc[i][j]);
    }
    // Stage `it` (in lp, lq; its first half already in p0, q0); the next one is
    // in np, nq.
    static __device__ __forceinline__ void stage(const LP& gp, const LQ& gq, S* lp, S* lq,
                                                 const S* np, const S* nq, int it, int nk, int wp,
                                                 int wq, int wave, int lane, s16x8 (&p0)[TP],
                                                 s16x8 (&q0)[TQ], f32x4 (&acc)[TP][TQ]) {
        s16x8 p1[TP], q1[TQ];
        frags(lp, lq, 1, wp, wq, lane, p1, q1);
        products(p0, q0, acc);
        __syncthreads();  // this buffer is read, the next stage has arrived
        frags(np, nq, 0, wp, wq, lane, p0, q0);
        __builtin_amdgcn_sched_barrier(0);
        if (it + 2 < nk) {
            gp.load(lp, (it + 2) * kBK, wave);
            gq.load(lq, (it + 2) * kBK, wave);
        }
        products(p1, q1, acc);
    }
    static __device__ __forceinline__ void run(const LP& gp, const LQ& gq, S* lp0, S* lq0, S* lp1,
                                               S* lq1, int nk, int wp, int wq, int wave, int lane,
                                               f32x4 (&acc)[TP][TQ]) {
        if (nk <= 0) return;
        gp.load(lp0, 0, wave);
        gq.load(lq0, 0, wave);
        __syncthreads();
        if (nk > 1) {
            gp.load(lp1, kBK, wave);
            gq.load(lq1, kBK, wave);
        }
        s16x8 p0[TP], q0[TQ];
        frags(lp0, lq0, 0, wp, wq, lane, p0, q0);
        for (int it = 0; it < nk; it += 2) {
            stage(gp, gq, lp0, lq0, lp1, lq1, it, nk, wp, wq, wave, lane, p0, q0, acc);
            if (it + 1 < nk)
                stage(gp, gq, lp1, lq1, lp0, lq0, it + 1, nk, wp, wq, wave, lane, p0, q0, acc);
        }
    }
};

}  // namespace moedx
