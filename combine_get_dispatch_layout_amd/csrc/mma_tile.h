// One output tile of a product on the matrix cores (device code).
//
//   D[q, p] = sum_r P(p, r) Q(q, r)
//
// p is the output's contiguous dimension (BP of it per tile), q its row
// dimension (BQ), r the reduction, taken BK at a time.  An operand is either
// "along" (its memory runs along r: [B rows][BK]) or "across" (its memory
// runs along p or q: [BK][B columns]).  Stages of both operands go from
// global memory straight into LDS; the buffer descriptors' range gives zeros
// for rows past an operand's end, so ragged tiles need no branch.
//
// LDS holds 16-byte chunks, permuted so that the reads of a wave spread over
// the banks (no bank conflict is counted in any of the three products).  Along:
// read with 16-byte loads, 8 reduction values of one row per lane.  Across: the
// transposing LDS read hands a lane 4 reduction values of one column, so a
// column-major operand costs no pass of its own.
//
// The matrix instruction is 16 x 16 x 32 with P as its A operand: a lane ends
// up with 4 consecutive p of one q.  (32 x 32 x 16 was 6 to 14% slower here.)
//
// What bounds the two loops below on random data is power as much as issue: an
// 8192^3 product that takes 775 us (1420 TFLOP/s; the library's takes 756) is
// 19% faster on zeros, whose clocks are higher.
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


// LDS is addressed through pointers of its own address space, one offset from
// the array's start per access: the compiler then knows which array a load
// into LDS writes and waits only for reads of that one.
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) s16x8 lds_s16x8;

// A value the compiler takes as it is: an address made of it stays one offset.
__device__ __forceinline__ int opaque(int v) {
    asm("" : "+v"(v));
    return v;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, max(bytes, 0),
                                             0x00020000);
}

constexpr uint32_t kOutside = 0x80000000u;  // past any descriptor's range (below 2^31 bytes)

// Both loaders keep one offset per lane; a load adds a wave-uniform step to it
// (an offset outside the range stays outside: steps are below 2^30).

// An operand along r: `halves` blocks of B / halves rows, each with its own
// first row (a gated product's gate and up rows).
template <int B, int NW, int BK, int kHalves>
struct Along {
    static constexpr int kRow = BK * 2;                // bytes per LDS row
    static constexpr int kRowChunks = BK / 8;
    static constexpr int kLoadRows = 64 / kRowChunks;  // rows of one wave load
    static constexpr int kLoads = B / (kLoadRows * NW);  // 16-byte loads per lane and stage
    static constexpr int kFragReads = 1;  // LDS reads per block of 16 and 32 values of r
    static_assert(B % (kLoadRows * NW * kHalves) == 0, "a wave's rows lie in one half");
    const char* base[kHalves];
    int valid[kHalves];  // rows of each half inside the operand
    int ld2;             // bytes per row
    int nr;              // reduction length
    uint32_t voff;
    int col;             // this lane's first reduction value within a stage

    // Rows 0, 1, ... take turns over the chunk positions, 128 bytes of LDS apart.
    static __device__ __forceinline__ int swizzle(int row) {
        return (BK == 64 ? row : row >> 1) & (kRowChunks - 1);
    }
    __device__ __forceinline__ void init(int ld_bytes, int reduction, int wave, int lane) {
        ld2 = ld_bytes;
        nr = reduction;
        const int row = lane / kRowChunks;
        const int c = (lane & (kRowChunks - 1)) ^ swizzle(row);
        col = c * 8;
        voff = (uint32_t)((wave * kLoadRows + row) * ld2) + c * 16;
    }
    __device__ __forceinline__ void half(int h, const void* first, int rows) {
        base[h] = static_cast<const char*>(first);
        valid[h] = min(max(rows, 0), B / kHalves);
    }
    // Stage at reduction value k0 into lds (this wave's part of it): all of it,
    // or of one half the first kSome loads of every wave, kSome * kLoadRows * NW
    // rows.
    template <int kSome = kLoads>
    __device__ __forceinline__ void load(lds_char* lds, int k0, int wave) const {
        static_assert(kSome == kLoads || kHalves == 1, "a part of one half");
        const uint32_t v = k0 + col < nr ? voff : kOutside;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            const __amdgpu_buffer_rsrc_t rs =
                make_rsrc(base[h] + (int64_t)k0 * 2, valid[h] * ld2 - k0 * 2);
#pragma unroll
            for (int j = 0; j < kSome / kHalves; ++j) {
                const int row = h * (B / kHalves) + (j * NW + wave) * kLoadRows;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + row * kRow), 16,
                                                         (int)(v + j * kLoadRows * NW * ld2), 0, 0,
                                                         0);
            }
        }
    }
    // Where a lane reads: 8 reduction values (of the kk-th 32) of row `first` +
    // (lane & 15).
    struct At {
        int at[BK / 32];
        __device__ __forceinline__ void init(int first, int lane) {
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk) {
                const int c = (kk * 4 + (lane >> 4)) ^ swizzle(lane & 15);  // first is 16 x
                at[kk] = opaque((first + (lane & 15)) * kRow + c * 16);
            }
        }
        // `off` rows further (a constant)
        __device__ __forceinline__ s16x8 frag(const lds_char* lds, int off, int kk) const {
            return *(const lds_s16x8*)(lds + at[kk] + off * kRow);
        }
    };
};

// An operand across r: BK rows of the reduction, B columns from column c0 of
// nc.  A lane group g of 16 takes reduction values 32 kk + 8 g + 4 h + i (h = 0,
// 1; i = 0..3); that row of the stage sits in LDS row i + 4 g + 16 h + 32 kk.  Its chunk c sits at c ^ 2 (row & 7): the 8
// rows that half a wave's transposing read touches lie in different banks.
template <int B, int NW, int BK>
struct Across {
    static constexpr int kLoads = B * BK / (512 * NW);
    static constexpr int kFragReads = 2;
    static constexpr int kRowChunks = B / 8;              // 16-byte chunks per LDS row
    static constexpr int kRowsPerLoad = 64 / kRowChunks;  // LDS rows one wave load fills
    static constexpr int kStep = NW * kRowsPerLoad;       // LDS rows of one load of all waves

    const char* base;
    int ld2;
    int nr;
    int skip2;  // bytes before column c0
    uint32_t voff;

    static __device__ __forceinline__ int swizzle(int lds_row) { return (lds_row & 7) * 2; }
    // The reduction row of an LDS row.
    static __device__ __forceinline__ constexpr int stage_row(int lds_row) {
        return (lds_row & 3) | ((lds_row & 12) << 1) | ((lds_row & 16) >> 2) | (lds_row & 32);
    }
    __device__ __forceinline__ void init(const void* first, int ld_bytes, int reduction,
                                         int c0, int nc, int wave, int lane) {
        base = static_cast<const char*>(first) + (int64_t)c0 * 2;
        ld2 = ld_bytes;
        nr = reduction;
        skip2 = c0 * 2;
        const int row = wave * kRowsPerLoad + lane / kRowChunks;
        const int c = (lane & (kRowChunks - 1)) ^ swizzle(row);
        voff = c0 + c * 8 < nc ? (uint32_t)(stage_row(row) * ld2) + c * 16 : kOutside;
    }
    // k0: unsigned, as a stage past 2^31 - 1 rows starts past 2^31.
    __device__ __forceinline__ void load(lds_char* lds, uint32_t k0, int wave) const {
        const uint32_t v = k0 < (uint32_t)nr ? voff : kOutside;
        const __amdgpu_buffer_rsrc_t rs =
            make_rsrc(base + (int64_t)k0 * ld2, min((int)((uint32_t)nr - k0), BK) * ld2 - skip2);
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rs, (lds_void*)(lds + (j * NW + wave) * 1024), 16,
                (int)(v + stage_row(j * kStep) * ld2), 0, 0, 0);
    }
    // Where a lane reads: columns from `first`, in steps of 16.  The permutation
    // moves 16 columns within their 128.
    struct At {
        int at[8];
        __device__ __forceinline__ void init(int first, int lane) {
            const int low = ((lane >> 4) << 2) | ((lane >> 2) & 3);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int col = first + 16 * x;
                const int c = (col / 8 + ((lane >> 1) & 1)) ^ swizzle(low);
                at[x] = opaque(low * B * 2 + c * 16 + (lane & 1) * 8);
            }
        }
            // `off` columns further (a constant)
        __device__ __forceinline__ s16x8 frag(const lds_char* lds, int off, int kk) const {
            s16x8 v;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int rest = (16 * h + 32 * kk) * B * 2 + (off & ~127) * 2;
                const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s16x4*)(lds + at[off / 16 & 7] + rest));
                v[4 * h] = t[0];
                v[4 * h + 1] = t[1];
                v[4 * h + 2] = t[2];
                v[4 * h + 3] = t[3];
            }
            return v;
        }
    };
};

// Waves of a tile: WP x WQ.  Wave (wp, wq) has the P blocks of 16 at
//   p = (i / (TP / 2)) * BP / 2 + wp * BP / 2 / WP + (i % (TP / 2)) * 16
// (its share of both halves of the tile) and the Q blocks at
//   q = j * 16 * WQ + wq * 16
// (dealt out in turn, so that a tile with few rows keeps every wave equally
// busy and leaves out whole blocks).
template <int BP, int WP>
__device__ __forceinline__ constexpr int p_step(int i) {
    constexpr int TP = BP / WP / 16;
    return (i / (TP / 2)) * (BP / 2) + (i % (TP / 2)) * 16;
}
template <int BP, int WP>
__device__ __forceinline__ int p_block(int wp, int i) {
    return wp * (BP / 2 / WP) + p_step<BP, WP>(i);
}
template <int WQ>
__device__ __forceinline__ int q_block(int wq, int j) {
    return j * 16 * WQ + wq * 16;
}

// A tile by 4 waves that takes at most half of a CU's LDS and registers: two
// workgroups share a CU, and one multiplies while the other waits at its
// barrier or stores its tile.  Three LDS buffers of 32 reduction values rotate:
// while stage s is multiplied, s + 1 is arriving and s + 2 is asked for.  Best
// where both operands are across r (weight gradients of 64 experts of 512 rows,
// 4096 x 7168: 2220 us; 2614, against 2930 as 256 x 256 tiles of 8 waves, before
// the odd stages went first); an operand along
// r would be fetched in half lines, which costs the forward product 20%.
template <typename S, int BP, int BQ, int WP, int WQ, int NQ, typename LP, typename LQ>
struct SharedCuLoop {
    static constexpr int TP = BP / WP / 16, TQ = BQ / WQ / 16;
    static constexpr int kBK = 32, kBuffers = 3;
    static constexpr int kStageLoads = LP::kLoads + LQ::kLoads;
    typename LP::At ap;
    typename LQ::At aq;

    __device__ __forceinline__ SharedCuLoop(int wp, int wq, int lane) {
        ap.init(wp * (BP / 2 / WP), lane);
        aq.init(wq * 16, lane);
    }
    __device__ __forceinline__ void load(const LP& gp, const LQ& gq, lds_char* lp, lds_char* lq,
                                         int it, int wave) const {
        gp.load(lp, (uint32_t)it * kBK, wave);
        gq.load(lq, (uint32_t)it * kBK, wave);
    }
    // Waits until only the last stage's loads are in flight and meets the other
    // waves.  The wait is the compiler's own instruction, so that it knows which
    // buffers have arrived and adds no wait before their reads.
    static __device__ __forceinline__ void arrive() {
        static_assert(kStageLoads < 16, "the wait's count has 4 bits here");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(kStageLoads | 0x70);  // vmcnt, no expcnt, lgkmcnt 0
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
    // Multiplies stage `it` (in lp, lq) and loads stage it + 2 into np, nq, which
    // every wave has read.  Past the reduction's end a load leaves zeros.
    __device__ __forceinline__ void stage(const LP& gp, const LQ& gq, const lds_char* lp,
                                          const lds_char* lq, lds_char* np, lds_char* nq, int it,
                                          int wave, f32x4 (&acc)[TP][TQ]) const {
        s16x8 p[TP], q[NQ];
        load(gp, gq, np, nq, it + 2, wave);
#pragma unroll
        for (int j = 0; j < NQ; ++j) q[j] = aq.frag(lq, j * 16 * WQ, 0);
#pragma unroll
        for (int i = 0; i < TP; ++i) p[i] = ap.frag(lp, p_step<BP, WP>(i), 0);
#pragma unroll
        for (int i = 0; i < TP; ++i)
#pragma unroll
            for (int j = 0; j < NQ; ++j) acc[i][j] = Mfma<S>::mul(p[i], q[j], acc[i][j]);
        // The Q reads and two of P first, then a read and a load per P block.
        __builtin_amdgcn_sched_group_barrier(0x100, LQ::kFragReads * NQ + 2 * LP::kFragReads, 0);
#pragma unroll
        for (int i = 0; i < TP; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, NQ, 0);
            if (i < kStageLoads) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
            if (i + 2 < TP) __builtin_amdgcn_sched_group_barrier(0x100, LP::kFragReads, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        // The next stage has arrived (only this stage's loads may be in flight),
        // and this wave's reads are done: their products have been issued.
        arrive();
    }
    __device__ __forceinline__ void run(const LP& gp, const LQ& gq, lds_char* lp0, lds_char* lq0,
                                        lds_char* lp1, lds_char* lq1, lds_char* lp2, lds_char* lq2,
                                        int nk, int wave, f32x4 (&acc)[TP][TQ]) const {
        if (nk <= 0) return;
        // The stages past a multiple of three go first, in the last buffers, so
        // that the loop always starts at buffer 0.
        // The waits count loads, so stage 1's stay behind stage 0's.
        const int odd = nk % kBuffers;
        if (odd == 0) {
            load(gp, gq, lp0, lq0, 0, wave);
            __builtin_amdgcn_sched_barrier(0);
            load(gp, gq, lp1, lq1, 1, wave);
        } else if (odd == 1) {
            load(gp, gq, lp2, lq2, 0, wave);
            __builtin_amdgcn_sched_barrier(0);
            load(gp, gq, lp0, lq0, 1, wave);
        } else {
            load(gp, gq, lp1, lq1, 0, wave);
            __builtin_amdgcn_sched_barrier(0);
            load(gp, gq, lp2, lq2, 1, wave);
        }
        arrive();
        int it = 0;
        if (odd == 2) {
            stage(gp, gq, lp1, lq1, lp0, lq0, it, wave, acc);
            ++it;
        }
        if (odd != 0) {
            stage(gp, gq, lp2, lq2, lp1, lq1, it, wave, acc);
            ++it;
        }
        while (it < nk) {
            stage(gp, gq, lp0, lq0, lp2, lq2, it, wave, acc);
            stage(gp, gq, lp1, lq1, lp0, lq0, it + 1, wave, acc);
            stage(gp, gq, lp2, lq2, lp1, lq1, it + 2, wave, acc);
            it += kBuffers;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS is left in flight
    }
};

// A tile whose operands' stages of 64 reduction values go around rings of LDS
// buffers, kP of them for P and kQ for Q.  A stage is multiplied in two halves
// of 32: while the first half's products run, the second half is read; past the
// barrier the stages kP and kQ further start loading into the buffers just
// read, and the next stage's first half is read under the second half's
// products.
//
// `stage` is told (restrict) that the buffers it reads are not the ones it
// loads into: the compiler then puts no wait of its own before an LDS read, and
// the one before the barrier is exact.  kPartQ: only the rows of Q that the
// tile has are loaded (64 experts of 128 rows, 7168 -> 4096: 735 us with all of
// them, 690 us without; no gain where P is read across r).
template <typename S, int BP, int BQ, int WP, int WQ, int NQ, int kP, int kQ, bool kPartQ,
          typename LP, typename LQ>
struct RingLoop {
    static constexpr int TP = BP / WP / 16, TQ = BQ / WQ / 16;
    static constexpr int kBK = 64;
    static constexpr int kPBytes = BP * kBK * 2, kQBytes = BQ * kBK * 2;
    static constexpr int kQLoads = kPartQ ? NQ : LQ::kLoads;
    static_assert(LQ::kLoadRows * WP * WQ == 16 * WQ, "a load of all waves is a block per wave");
    static_assert(kP >= kQ && kQ >= 2, "P is loaded at least as far ahead as Q");
    typename LP::At ap;
    typename LQ::At aq;
    int shift, stages;

    // Stages are taken from `first_stage` on, around the reduction.
    __device__ __forceinline__ RingLoop(int wp, int wq, int lane, int first_stage, int nk)
        : shift(first_stage), stages(nk) {
        ap.init(wp * (BP / 2 / WP), lane);
        aq.init(wq * 16, lane);
    }
    __device__ __forceinline__ int place(int it) const {
        const int s = it + shift;
        return (s - (s >= stages ? stages : 0)) * kBK;
    }
    __device__ __forceinline__ void frags(const lds_char* lp, const lds_char* lq, int kk,
                                          s16x8 (&p)[TP], s16x8 (&q)[TQ]) const {
#pragma unroll
        for (int i = 0; i < TP; ++i) p[i] = ap.frag(lp, p_step<BP, WP>(i), kk);
#pragma unroll
        for (int j = 0; j < NQ; ++j) q[j] = aq.frag(lq, j * 16 * WQ, kk);
    }
    static __device__ __forceinline__ void products(const s16x8 (&p)[TP], const s16x8 (&q)[TQ],
                                                    f32x4 (&acc)[TP][TQ]) {
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int i = 0; i < TP; ++i) acc[i][j] = Mfma<S>::mul(p[i], q[j], acc[i][j]);
    }
    // The first half's products (operands in p0, q0) while the second half is
    // read from rp, rq.
    __device__ __forceinline__ void first(const lds_char* rp, const lds_char* rq,
                                          const s16x8 (&p0)[TP], const s16x8 (&q0)[TQ],
                                          s16x8 (&p1)[TP], s16x8 (&q1)[TQ],
                                          f32x4 (&acc)[TP][TQ]) const {
        frags(rp, rq, 1, p1, q1);
        products(p0, q0, acc);
        interleave<false>();
        __builtin_amdgcn_sched_barrier(0);
    }
    // The second half's products while the next stage's first half is read from
    // rp, rq and further stages load into wp, wq.  Past the last stage what is
    // fetched and read goes unused.
    __device__ __forceinline__ void second(const LP& gp, const LQ& gq,
                                           const lds_char* __restrict rp,
                                           const lds_char* __restrict rq,
                                           lds_char* __restrict wp, lds_char* __restrict wq, int it,
                                           int wave, s16x8 (&p0)[TP], s16x8 (&q0)[TQ],
                                           const s16x8 (&p1)[TP], const s16x8 (&q1)[TQ],
                                           f32x4 (&acc)[TP][TQ]) const {
        frags(rp, rq, 0, p0, q0);
        gq.template load<kQLoads>(wq, place(it + kQ), wave);
        // The waits count loads in this order: no load may pass here.
        __builtin_amdgcn_sched_barrier(0x38e);
        gp.load(wp, place(it + kP), wave);
        products(p1, q1, acc);
        interleave<true>();
        __builtin_amdgcn_sched_barrier(0);
    }
    // Spreads a half's LDS reads (and a stage's loads) among its products: both
    // waves of a SIMD leave the barrier together, and what they issue before
    // their first product is time the matrix unit stands still.
    template <bool kLoads>
    static __device__ __forceinline__ void interleave() {
        constexpr int kReads = LP::kFragReads * TP + LQ::kFragReads * NQ;
        constexpr int kMem = kReads + (kLoads ? LP::kLoads + kQLoads : 0);
        constexpr int kPer = TP * NQ / kMem > 0 ? TP * NQ / kMem : 1;
        __builtin_amdgcn_sched_group_barrier(0x002, 12, 0);  // addresses
#pragma unroll
        for (int i = 0; i < kReads; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);     // LDS read
            __builtin_amdgcn_sched_group_barrier(0x008, kPer, 0);  // products
        }
        if constexpr (kLoads) {
#pragma unroll
            for (int i = 0; i < LP::kLoads + kQLoads; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);  // load
                __builtin_amdgcn_sched_group_barrier(0x008, kPer, 0);
            }
        }
    }
    template <int kInFlight>
    static __device__ __forceinline__ void barrier() {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kInFlight) : "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void run(const LP& gp, const LQ& gq, lds_char* lp, lds_char* lq,
                                        int wave, f32x4 (&acc)[TP][TQ]) const {
        if (stages <= 0) return;
        // in the order in which they are needed
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            if (i < kQ) gq.template load<kQLoads>(lq + i * kQBytes, place(i), wave);
            __builtin_amdgcn_sched_barrier(0);
            gp.load(lp + i * kPBytes, place(i), wave);
            __builtin_amdgcn_sched_barrier(0);
        }
        // At a barrier only a P stage that is needed later may be in flight.
        constexpr int kAhead = kP > kQ ? LP::kLoads : 0;
        barrier<(kP - 1) * LP::kLoads + (kQ - 1) * kQLoads>();
        s16x8 p0[TP], q0[TQ], p1[TP], q1[TQ];
        frags(lp, lq, 0, p0, q0);
        int pb = 0, qb = 0;
        for (int it = 0; it < stages; ++it) {
            lds_char* const rp = lp + pb * kPBytes;
            lds_char* const rq = lq + qb * kQBytes;
            pb = pb + 1 == kP ? 0 : pb + 1;
            qb = qb + 1 == kQ ? 0 : qb + 1;
            first(rp, rq, p0, q0, p1, q1, acc);
            barrier<kAhead>();
            second(gp, gq, lp + pb * kPBytes, lq + qb * kQBytes, rp, rq, it, wave, p0, q0, p1, q1,
                   acc);
        }
        barrier<0>();  // no load into LDS is left in flight
    }
};

}  // namespace moedx
