// Router kernels for gfx950: top-k expert choice with gate weights, and its
// gradient.
//
// For token logits l [E]: score p = softmax(l), or sigmoid(l); key = score +
// bias.  With groups (contiguous, E / G experts), a group's score is the sum
// of its two best keys and only the groups_kept best groups keep their
// experts.  The K best keys are chosen, ties to the lower index.  An expert
// whose logit is -inf or NaN is never chosen and has p = 0.
//
// The chosen set must not depend on how exp rounds: two keys that differ by
// less than an fp32 rounding are common among 10^6 scores.  So keys are fp64
// wherever they go through exp, and the logits themselves (exact, and in the
// same order) when there is neither bias nor group.  The weights are fp32.
//
// One wavefront per token: lane l holds experts l, l + 64, ...; the K rounds
// are wave-wide maxima.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "expert_launch.h"
#include "moedx.h"
#include "numeric.h"

namespace moedx {

namespace {

constexpr int kGateWaves = 4;
constexpr int kGateThreads = kGateWaves * 64;

constexpr float kNegInf = -INFINITY;

// log sigmoid(l), without overflow
__device__ __forceinline__ float log_sigmoid(float l) {
    return fminf(l, 0.0f) - log1pf(expf(-fabsf(l)));
}
__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// Wave-wide best (largest key, then lowest index).
template <typename Key>
__device__ __forceinline__ void wave_best(Key& key, int& idx) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const Key k = __shfl_xor(key, d, 64);
        const int i = __shfl_xor(idx, d, 64);
        if (k > key || (k == key && i < idx)) {
            key = k;
            idx = i;
        }
    }
}

// The token's logits, l[j] of expert lane + 64 j; NaN counts as -inf.
template <typename S, int NV>
__device__ __forceinline__ void load_logits(const S* logits, int E, int t, int lane,
                                            float (&l)[NV]) {
    const S* row = logits + (int64_t)t * E;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = lane + 64 * j;
        const float v = e < E ? (float)row[e] : kNegInf;
        l[j] = v >= kNegInf ? v : kNegInf;
    }
}

template <int NV>
__device__ __forceinline__ float row_max(const float (&l)[NV]) {
    float m = l[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) m = fmaxf(m, l[j]);
    return wave_max(m);
}

template <int NV>
__device__ __forceinline__ float exp_sum(const float (&l)[NV], float m) {
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) z += l[j] > kNegInf ? expf(l[j] - m) : 0.0f;
    return wave_sum(z);
}

// Key: float (the logits are the keys) or double.
template <typename S, int NV, typename Key>
__global__ __launch_bounds__(kGateThreads) void gate_topk_kernel(GateArgs a,
                                                                 int64_t* __restrict__ topk_idx,
                                                                 float* __restrict__ topk_weights) {
    constexpr bool kExact = sizeof(Key) == 8;
    __shared__ Key staged[kExact ? kGateWaves * NV * 64 : 1];
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int t = blockIdx.x * kGateWaves + wave;
    if (t >= a.T) return;
    float l[NV];
    load_logits<S, NV>(static_cast<const S*>(a.logits), a.E, t, lane, l);
    const bool softmax = a.score == MOEDX_GATE_SOFTMAX;
    const float m = row_max(l);
    const float z = softmax ? exp_sum(l, m) : 1.0f;

    const Key none = (Key)kNegInf;
    Key key[NV];
    if constexpr (!kExact) {
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = l[j];
    } else {
        double zd = 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            key[j] = softmax ? exp((double)l[j] - (double)m) : 1.0 / (1.0 + exp(-(double)l[j]));
            if (!(l[j] > kNegInf)) key[j] = 0.0;
            zd += key[j];
        }
        if (softmax) {
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) zd += __shfl_xor(zd, d, 64);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = lane + 64 * j;
            if (softmax) key[j] /= zd;
            if (a.bias && e < a.E) key[j] += (double)a.bias[e];
            if (!(l[j] > kNegInf) || !(key[j] > none)) key[j] = none;
        }
        if (a.groups > 1) {
            Key* mine = staged + wave * NV * 64;
#pragma unroll
            for (int j = 0; j < NV; ++j) mine[lane + 64 * j] = key[j];
            __builtin_amdgcn_wave_barrier();
            // lane g < groups: the sum of the group's two best keys
            const int per = a.E / a.groups;
            Key one = none, two = none;
            if (lane < a.groups) {
                for (int i = 0; i < per; ++i) {
                    const Key v = mine[lane * per + i];
                    two = fmax(two, fmin(one, v));
                    one = fmax(one, v);
                }
            }
            const Key gs = one > none ? one + (two > none ? two : 0.0) : none;
            int better = 0;
            for (int g = 0; g < a.groups; ++g) {
                const Key o = __shfl(gs, g, 64);
                better += (o > gs || (o == gs && g < lane)) ? 1 : 0;
            }
            const uint64_t keep = __ballot(lane < a.groups && better < a.groups_kept);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int e = lane + 64 * j;
                if (e < a.E && !((keep >> (e / per)) & 1)) key[j] = none;
            }
        }
    }

    // K rounds; lane k keeps the k-th choice and its logit.
    int mine_idx = -1;
    float mine_l = kNegInf;
    for (int k = 0; k < a.K; ++k) {
        Key best = none;
        int at = 1 << 30;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (key[j] > best) {
                best = key[j];
                at = lane + 64 * j;
            }
        wave_best(best, at);
        if (!(best > none)) break;
        float lv = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (at == lane + 64 * j) {
                key[j] = none;
                lv = l[j];
            }
        }
        lv = __shfl(lv, at & 63, 64);
        if (lane == k) {
            mine_idx = at;
            mine_l = lv;
        }
    }
    const bool have = mine_idx >= 0;
    float w = 0.0f;
    if (a.renormalize) {
        // a softmax over the chosen (log) scores: never 0 / 0
        const float s = !have ? kNegInf : softmax ? mine_l : log_sigmoid(mine_l);
        const float top = wave_max(s);
        const float x = have ? expf(s - top) : 0.0f;
        const float total = wave_sum(x);
        w = have ? x / total : 0.0f;
    } else if (have) {
        w = softmax ? expf(mine_l - m) / z : sigmoid(mine_l);
    }
    if (lane < a.K) {
        topk_idx[(int64_t)t * a.K + lane] = mine_idx;
        topk_weights[(int64_t)t * a.K + lane] = have ? a.scale * w : 0.0f;
    }
}

template <typename S, int NV>
__global__ __launch_bounds__(kGateThreads) void gate_topk_backward_kernel(
    GateArgs a, const int64_t* __restrict__ topk_idx, const float* __restrict__ d_topk_weights,
    S* __restrict__ d_logits) {
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * kGateWaves + (threadIdx.x >> 6);
    if (t >= a.T) return;
    const S* logits = static_cast<const S*>(a.logits);
    float l[NV];
    load_logits<S, NV>(logits, a.E, t, lane, l);
    const bool softmax = a.score == MOEDX_GATE_SOFTMAX;

    // lane k: the k-th choice, its logit and its incoming gradient
    int idx = -1;
    float g = 0.0f, lk = kNegInf;
    if (lane < a.K) {
        const int64_t i = topk_idx[(int64_t)t * a.K + lane];
        if (i >= 0 && i < a.E) {
            idx = (int)i;
            g = d_topk_weights[(int64_t)t * a.K + lane];
            const float v = (float)logits[(int64_t)t * a.E + idx];
            lk = v >= kNegInf ? v : kNegInf;
        }
    }
    const bool have = idx >= 0 && lk > kNegInf;
    float own = 0.0f;    // gradient added at the chosen expert
    float dot = 0.0f;    // softmax over all experts: p_j * scale * (g_j - dot)
    float m = 0.0f, z = 1.0f;
    const bool dense = softmax && !a.renormalize;
    if (a.renormalize) {
        const float s = !have ? kNegInf : softmax ? lk : log_sigmoid(lk);
        const float top = wave_max(s);
        const float x = have ? expf(s - top) : 0.0f;
        const float total = wave_sum(x);
        const float v = have ? x / total : 0.0f;
        const float gv = wave_sum(have ? g * v : 0.0f);
        own = have ? a.scale * v * (g - gv) : 0.0f;
        if (!softmax) own *= sigmoid(-lk);
        if (!have) own = 0.0f;
    } else if (softmax) {
        m = row_max(l);
        z = exp_sum(l, m);
        const float p = have ? expf(lk - m) / z : 0.0f;
        dot = wave_sum(have ? g * p : 0.0f);
        own = have ? g : 0.0f;
    } else {
        own = have ? a.scale * g * sigmoid(lk) * sigmoid(-lk) : 0.0f;
    }
    float d[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) d[j] = 0.0f;
    for (int k = 0; k < a.K; ++k) {
        const int e = __builtin_amdgcn_readlane(idx, k);
        const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(own), k));
#pragma unroll
        for (int j = 0; j < NV; ++j) d[j] += e == lane + 64 * j ? v : 0.0f;
    }
    S* out = d_logits + (int64_t)t * a.E;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = lane + 64 * j;
        if (e >= a.E) continue;
        float v = d[j];
        if (dense) v = l[j] > kNegInf ? a.scale * (expf(l[j] - m) / z) * (v - dot) : 0.0f;
        out[e] = (S)v;
    }
}

template <typename S, int NV>
hipError_t launch_gate_nv(const GateArgs& a, int64_t* idx, float* w, const Launch& L) {
    const dim3 grid((a.T + kGateWaves - 1) / kGateWaves), block(kGateThreads);
    if (a.bias == nullptr && a.groups <= 1)
        return launch_kernel(gate_topk_kernel<S, NV, float>, grid, block, L, a, idx, w);
    return launch_kernel(gate_topk_kernel<S, NV, double>, grid, block, L, a, idx, w);
}

template <typename S, int NV>
hipError_t launch_gate_bwd_nv(const GateArgs& a, const int64_t* idx, const float* dw, void* dl,
                              const Launch& L) {
    const dim3 grid((a.T + kGateWaves - 1) / kGateWaves), block(kGateThreads);
    return launch_kernel(gate_topk_backward_kernel<S, NV>, grid, block, L, a, idx, dw,
                         static_cast<S*>(dl));
}

template <typename F>
hipError_t by_width(int E, F&& f) {
    const int nv = (E + 63) / 64;
    if (nv <= 1) return f(std::integral_constant<int, 1>{});
    if (nv <= 2) return f(std::integral_constant<int, 2>{});
    if (nv <= 4) return f(std::integral_constant<int, 4>{});
    if (nv <= 8) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_gate_topk(const GateArgs& a, int64_t* idx, float* w, const Launch& L) {
    return by_width(a.E, [&](auto nv) {
        if (a.dtype == MOEDX_F32) return launch_gate_nv<float, nv()>(a, idx, w, L);
        if (a.dtype == MOEDX_F16) return launch_gate_nv<_Float16, nv()>(a, idx, w, L);
        return launch_gate_nv<__bf16, nv()>(a, idx, w, L);
    });
}

hipError_t launch_gate_topk_backward(const GateArgs& a, const int64_t* idx, const float* dw,
                                     void* dl, const Launch& L) {
    return by_width(a.E, [&](auto nv) {
        if (a.dtype == MOEDX_F32) return launch_gate_bwd_nv<float, nv()>(a, idx, dw, dl, L);
        if (a.dtype == MOEDX_F16) return launch_gate_bwd_nv<_Float16, nv()>(a, idx, dw, dl, L);
        return launch_gate_bwd_nv<__bf16, nv()>(a, idx, dw, dl, L);
    });
}

}  // namespace moedx
