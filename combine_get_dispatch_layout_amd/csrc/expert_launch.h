// Internal launchers of the router, expert-order and expert-product kernels
// (host functions; not exported).  Shapes have been validated by the C-ABI
// layer.  As in launch.h, a launcher enqueues on L.stream and returns the HIP
// status; L.start / L.stop are stamped by its first and last kernel.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_plan.h"
#include "launch.h"

namespace moedx {

// ---- router -------------------------------------------------------------------

struct GateArgs {
    const void* logits;  // [T, E]
    int dtype;           // MOEDX_BF16 / F16 / F32
    int T, E, K;
    int score;           // MOEDX_GATE_SOFTMAX / SIGMOID
    int groups, groups_kept;
    int renormalize;
    float scale;
    const float* bias;   // [E] or null; selection only
    FastDiv per_div;     // by the experts of a group
};

hipError_t launch_gate_topk(const GateArgs& a, int64_t* topk_idx, float* topk_weights,
                            const Launch& L);
hipError_t launch_gate_topk_backward(const GateArgs& a, const int64_t* topk_idx,
                                     const float* d_topk_weights, void* d_logits,
                                     const Launch& L);

// ---- rows in expert order -----------------------------------------------------

// Pairs (token, slot) are counted and ranked in tiles of kOrderTile * iters,
// at most kOrderMaxTiles of them: every ranking workgroup reads all counts.
constexpr int kOrderTile = 1024;
constexpr int kOrderMaxTiles = 128;

struct OrderArgs {
    const int64_t* topk_idx;  // [T, K]
    int T, K, E;
    // ids local to the bucket of their receive row (null: ids are global)
    const int32_t* rank_prefix_matrix;  // [R] inclusive
    int R, P;
    int32_t* expert_offsets;  // [E + 1]
    int32_t* row_of_slot;     // [T, K]
    int32_t* slot_of_row;     // [T * K]
    int32_t* tile_counts;     // workspace [tiles, E]
    int tiles, iters;
};

inline int order_iters(int64_t pairs) {
    const int64_t per = (int64_t)kOrderTile * kOrderMaxTiles;
    return pairs > per ? (int)((pairs + per - 1) / per) : 1;
}
inline int order_tiles(int64_t pairs) {
    const int64_t tile = (int64_t)kOrderTile * order_iters(pairs);
    return (int)((pairs + tile - 1) / tile);
}

hipError_t launch_expert_order(const OrderArgs& a, const Launch& L);

// row_bytes: a multiple of 16.
hipError_t launch_expert_sort(const void* x, int T, int K, int64_t row_bytes,
                              const int32_t* row_of_slot, void* rows, const Launch& L);
hipError_t launch_expert_unsort(const void* rows, int dtype, int T, int K, int H,
                                const int32_t* row_of_slot, const float* weights, void* out,
                                const Launch& L);
hipError_t launch_expert_unsort_backward(const void* d_out, const void* rows, int dtype, int T,
                                         int K, int H, const int32_t* row_of_slot,
                                         const int32_t* slot_of_row, const float* weights,
                                         void* d_rows, float* d_weights, const Launch& L);

// ---- the experts' products ----------------------------------------------------

// y [rows, N] = x [rows, K] w[e]^T, w [E, N, K]; with swiglu w is [E, 2N, K]
// (gate rows, then up rows), y = silu(gate) * up and pre (or null) receives
// [rows, 2N].  dtype: MOEDX_BF16 / F16.
hipError_t launch_expert_linear(const void* x, const void* w, int dtype, const ExpertRows& er,
                                int K, int N, bool swiglu, void* y, void* pre, const Launch& L);
// d_x [rows, K] = d_y [rows, N] w[e]
hipError_t launch_expert_dgrad(const void* d_y, const void* w, int dtype, const ExpertRows& er,
                               int K, int N, void* d_x, const Launch& L);
// d_w [E, N, K] = d_y_e^T x_e; f32_out: d_w is fp32 (else of dtype)
hipError_t launch_expert_wgrad(const void* d_y, const void* x, int dtype, const ExpertRows& er,
                               int K, int N, void* d_w, bool f32_out, const Launch& L);
// d_pre [rows, 2N] from d_h [rows, N] and pre [rows, 2N]
hipError_t launch_swiglu_backward(const void* d_h, const void* pre, int dtype,
                                  const ExpertRows& er, int N, void* d_pre, const Launch& L);

// ---- rows in int8 ---------------------------------------------------------------

// block: 0 (a scale per row) or 128 (one per 128 values).  With neither offsets
// nor counts every row counts.
hipError_t launch_expert_quantize(const void* x, int dtype, const ExpertRows& er, int H, int block,
                                  int8_t* codes, float* scales, const Launch& L);
hipError_t launch_expert_sort_int8(const void* x, int dtype, int T, int K, int H,
                                   const int32_t* row_of_slot, int8_t* codes, float* scales,
                                   const Launch& L);
hipError_t launch_expert_dequantize(const int8_t* codes, const float* scales, const ExpertRows& er,
                                    int H, int block, void* x, int dtype, const Launch& L);
// y [rows, N] of `dtype` from codes x [rows, K] and w [E, N or 2N, K]
hipError_t launch_expert_linear_int8(const int8_t* x, const float* x_scales, const int8_t* w,
                                     const float* w_scales, const ExpertRows& er, int K, int N,
                                     bool swiglu, void* y, int dtype, const Launch& L);
// d_w [E, N, K] from d_y [rows, N] of `dtype` and codes x [rows, K]
hipError_t launch_expert_wgrad_int8(const void* d_y, const int8_t* x, const float* x_scales,
                                    int block, int dtype, const ExpertRows& er, int K, int N,
                                    void* d_w, bool f32_out, const Launch& L);
// d_pre [rows, 2N] and h [rows, N] (or null) from d_h and codes of pre [rows, 2N]
hipError_t launch_swiglu_backward_int8(const void* d_h, const int8_t* codes, const float* scales,
                                       int block, int dtype, const ExpertRows& er, int N,
                                       void* d_pre, void* h, const Launch& L);

}  // namespace moedx
