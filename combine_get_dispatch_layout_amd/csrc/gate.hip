// Router kernels for gfx950: top-k expert choice with gate weights, and its
// gradient.
//
// For token logits l [E]: score p = softmax(l), or sigmoid(l); key = score +
// bias.  With groups (contiguous, E / G experts), a group's score is the sum
// of its two best keys and only the groups_kept best groups keep their
// experts.  The K best keys are chosen, ties to the lower index.  An expert
// whose logit is -inf or NaN is never chosen and has p = 0.  A logit of +inf
// makes a softmax's weights NaN; the choice is that of the limit, where the
// experts with +inf share p = 1.
//
// The chosen set must not depend on how exp rounds: two keys that differ by
// less than an fp32 rounding are common among 10^6 scores.  So keys are fp64
// wherever they go through exp, and the logits themselves (exact, and in the
// same order) when there is neither bias nor group.  The weights are fp32.
//
// Where scores are the keys, one wavefront takes a token: lane l holds experts
// l NV .. l NV + NV - 1 in registers (one vector load where E allows it).  A
// round takes the wave-wide maximum of the keys, then the first lane that holds
// it.  Where the logits are, and in the gradient, a row of 16 lanes takes a token
// (up to 256 experts): a key is the ordered logit with the expert's number below
// it, so keys differ, a maximum names its expert, ties go to the lower one by
// themselves, and a round is the maximum below the last one.
//
// What bounds these kernels is the instructions of the rounds and exps, not the
// logits' bytes: 16384 tokens of 256 bf16 logits, top-8, softmax: 7.1 us, and
// 7.9 for the gradient (16.6 and 14.7 with a wave per token).  128 tokens with
// bias, 8 groups and renormalised sigmoids, one wave's latency: 7.2 us, of which
// 3.6 are the launch, the loads and the scores, 2 the rounds.
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

// Unsigned integers in the order of the values; +0 and -0 are alike.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
    return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}

// The token's logits, l[j] of expert lane * NV + j; NaN counts as -inf, and
// past the last expert there is -inf.  `vec`: E is a multiple of NV and rows
// are aligned to NV values.
template <typename S, int NV>
__device__ __forceinline__ void load_logits(const S* logits, int E, int t, int lane, bool vec,
                                            float (&l)[NV]) {
    const S* row = logits + (int64_t)t * E;
    const int e0 = lane * NV;
    if (vec) {
        typedef S vals __attribute__((ext_vector_type(NV)));
        vals v{};
        if (e0 < E) v = *reinterpret_cast<const vals*>(row + e0);
#pragma unroll
        for (int j = 0; j < NV; ++j) l[j] = e0 < E ? (float)v[j] : kNegInf;
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) l[j] = e0 + j < E ? (float)row[e0 + j] : kNegInf;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) l[j] = fmaxf(l[j], kNegInf);  // the number, of a NaN and one
}

// The bias of the lane's experts, asked for together with the logits.
template <int NV>
__device__ __forceinline__ void load_bias(const GateArgs& a, int lane, float (&b)[NV]) {
    typedef float vals __attribute__((ext_vector_type(NV), aligned(4)));
    const int e0 = lane * NV;
#pragma unroll
    for (int j = 0; j < NV; ++j) b[j] = 0.0f;
    if (!a.bias) return;
    if (e0 + NV <= a.E) {
        const vals v = *reinterpret_cast<const vals*>(a.bias + e0);
#pragma unroll
        for (int j = 0; j < NV; ++j) b[j] = v[j];
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (e0 + j < a.E) b[j] = a.bias[e0 + j];
    }
}

template <int NV>
__device__ __forceinline__ float token_max(const float (&l)[NV]) {
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

// The renormalised weight (before scale) of a row's lane that holds a chosen
// logit l: a softmax over the chosen (log) scores, never 0 / 0.
__device__ __forceinline__ float row_share(bool have, bool softmax, float l) {
    const float s = !have ? kNegInf : softmax ? l : log_sigmoid(l);
    const float top = row_max(s);  // by every lane of the row
    const float x = have ? expf(s - top) : 0.0f;
    const float total = row_sum(x);
    return have ? x / total : 0.0f;
}

// The sum of the two best of (one, two), each -inf when there is none.
__device__ __forceinline__ double pair_score(double one, double two) {
    return one > -INFINITY ? one + (two > -INFINITY ? two : 0.0) : -INFINITY;
}

// Drops the keys outside the groups_kept best groups.  staged: 64 * NV values
// of this wave in LDS.
template <int NV>
__device__ __forceinline__ void keep_groups(const GateArgs& a, int lane, double* staged,
                                            double (&key)[NV]) {
    const int per = a.E / a.groups;
    const int span = per / NV;  // lanes of a group, when it fills whole lanes
    double gs = -INFINITY;      // lane g < groups: the group's score
    if (per % NV == 0 && (span & (span - 1)) == 0 && span <= 64) {
        double one = key[0], two = -INFINITY;
#pragma unroll
        for (int j = 1; j < NV; ++j) {
            two = fmax(two, fmin(one, key[j]));
            one = fmax(one, key[j]);
        }
        // the other half's pair: of 2, 4, 8 and 16 lanes by lane-shifted reads,
        // of 32 and 64 through LDS
        const auto join = [&](double o1, double o2) {
            two = fmax(fmin(one, o1), fmax(two, o2));
            one = fmax(one, o1);
        };
        if (span > 1) join(lane_swap<0xb1>(one), lane_swap<0xb1>(two));
        if (span > 2) join(lane_swap<0x4e>(one), lane_swap<0x4e>(two));
        if (span > 4) join(lane_swap<0x141>(one), lane_swap<0x141>(two));
        if (span > 8) join(lane_swap<0x140>(one), lane_swap<0x140>(two));
        for (int d = 16; d < span; d <<= 1)
            join(__shfl_xor(one, d, 64), __shfl_xor(two, d, 64));
        const double score = pair_score(one, two);
        gs = __shfl(score, lane * span & 63, 64);
        if (lane >= a.groups) gs = -INFINITY;
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) staged[lane * NV + j] = key[j];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        double one = -INFINITY, two = -INFINITY;
        if (lane < a.groups) {
            for (int i = 0; i < per; ++i) {
                const double v = staged[lane * per + i];
                two = fmax(two, fmin(one, v));
                one = fmax(one, v);
            }
            gs = pair_score(one, two);
        }
    }
    const uint64_t mine = ordered(gs);
    int better = 0;
    for (int g = 0; g < a.groups; ++g) {
        const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)mine, g);
        const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(mine >> 32), g);
        const uint64_t o = ((uint64_t)hi << 32) | lo;
        better += (o > mine || (o == mine && g < lane)) ? 1 : 0;
    }
    const uint64_t keep = __ballot(lane < a.groups && better < a.groups_kept);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int g = (int)a.per_div.div((uint32_t)(lane * NV + j));
        if (g >= 64 || !((keep >> g) & 1)) key[j] = -INFINITY;
    }
}

// Key: uint32_t where the logits are the keys, double where scores are.
template <typename S, int NV, typename Key>
__global__ __launch_bounds__(kGateThreads) void gate_topk_kernel(GateArgs a, bool vec,
                                                                 int64_t* __restrict__ topk_idx,
                                                                 float* __restrict__ topk_weights) {
    constexpr bool kScores = sizeof(Key) == 8;
    constexpr Key kNone = kScores ? (Key)-INFINITY : (Key)0;  // cannot be chosen
    __shared__ double staged[kScores ? kGateWaves * NV * 64 : 1];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.x * kGateWaves + wave;
    if (t >= a.T) return;
    float l[NV], bias[kScores ? NV : 1];
    if constexpr (kScores) load_bias<NV>(a, lane, bias);
    load_logits<S, NV>(static_cast<const S*>(a.logits), a.E, t, lane, vec, l);
    const bool softmax = a.score == MOEDX_GATE_SOFTMAX;

    float m = 0.0f;
    Key key[NV];
    if constexpr (!kScores) {
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = l[j] > kNegInf ? ordered(l[j]) : 0u;
        if (softmax && !a.renormalize) m = token_max(l);
    } else {
        double s[NV];
        if (softmax) {
            m = token_max(l);
            double z = 0.0;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                // 1 at the maximum, also where it is +inf: the others are 0 then
                s[j] = !(l[j] > kNegInf) ? 0.0
                       : l[j] == m       ? 1.0
                                         : exp((double)l[j] - (double)m);
                z += s[j];
            }
            z = wave_sum(z);
#pragma unroll
            for (int j = 0; j < NV; ++j) s[j] /= z;
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) s[j] = 1.0 / (1.0 + exp(-(double)l[j]));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            s[j] += (double)bias[j];
            if (!(l[j] > kNegInf) || !(s[j] > -INFINITY)) s[j] = -INFINITY;
        }
        if (a.groups > 1) keep_groups<NV>(a, lane, staged + wave * NV * 64, s);
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = s[j];
    }

    // K rounds; lane k keeps the k-th choice.
    int mine_idx = -1;
    for (int k = 0; k < a.K; ++k) {
        Key best = key[0];
        int at = 0;
#pragma unroll
        for (int j = 1; j < NV; ++j)
            if (key[j] > best) {
                best = key[j];
                at = j;
            }
        const Key top = wave_max(best);
        if (top == kNone) break;
        const int from = __builtin_ctzll(__ballot(best == top));
        const int j0 = __builtin_amdgcn_readlane(at, from);
        const int gone = lane == from ? at : NV;
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = j == gone ? kNone : key[j];
        if (lane == k) mine_idx = from * NV + j0;
    }
    // its logit, from the lane that holds it
    float mine_l = kNegInf;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const float v = __shfl(l[j], max(mine_idx, 0) / NV, 64);
        if (mine_idx >= 0 && mine_idx % NV == j) mine_l = v;
    }
    const bool have = mine_idx >= 0;
    float w = 0.0f;
    if (a.renormalize) {
        w = row_share(have, softmax, mine_l);  // the choices are in the first row
        if (m == INFINITY) w = NAN;  // a softmax with +inf, whether that was chosen or not
    } else if (softmax) {
        const float z = exp_sum(l, m);
        w = have ? expf(mine_l - m) / z : 0.0f;
    } else if (have) {
        w = sigmoid(mine_l);
    }
    if (lane < a.K) {
        topk_idx[(int64_t)t * a.K + lane] = mine_idx;
        topk_weights[(int64_t)t * a.K + lane] = have ? a.scale * w : 0.0f;
    }
}

template <typename S, int NV>
__global__ __launch_bounds__(kGateThreads) void gate_topk_backward_kernel(
    GateArgs a, bool vec, const int64_t* __restrict__ topk_idx, const float* __restrict__ d_topk_weights,
    S* __restrict__ d_logits) {
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * kGateWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.T) return;
    const S* logits = static_cast<const S*>(a.logits);
    float l[NV];
    load_logits<S, NV>(logits, a.E, t, lane, vec, l);
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
        m = token_max(l);
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
        for (int j = 0; j < NV; ++j) d[j] += e == lane * NV + j ? v : 0.0f;
    }
    if (dense) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            d[j] = l[j] > kNegInf ? a.scale * (expf(l[j] - m) / z) * (d[j] - dot) : 0.0f;
    }
    S* out = d_logits + (int64_t)t * a.E + lane * NV;
    if (vec) {
        typedef S vals __attribute__((ext_vector_type(NV)));
        vals v;
#pragma unroll
        for (int j = 0; j < NV; ++j) v[j] = (S)d[j];
        if (lane * NV < a.E) *reinterpret_cast<vals*>(out) = v;
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (lane * NV + j < a.E) out[j] = (S)d[j];
    }
}

// ---- a token per row of 16 lanes ------------------------------------------------

constexpr int kRowTokens = kGateThreads / 16;  // tokens of a workgroup

// A logit's key: ordered, and below it ~expert, so that keys differ.  Keys up to
// kNone, those of -inf among them, cannot be chosen.
template <typename S>
struct LogitKey {  // bf16 and fp16 leave the low 13 bits of their fp32 form clear
    typedef uint32_t type;
    static constexpr type kNone = 0x007fffffu;  // the order of -inf
    static __device__ __forceinline__ type make(float l, int e) {
        return (ordered(l) & ~0xffu) | (~e & 0xff);
    }
    static __device__ __forceinline__ int expert(type k) { return (int)(~k & 0xff); }
    static __device__ __forceinline__ float logit(type k) {
        return __uint_as_float((k >> 31) ? (k & ~0xffu) ^ 0x80000000u : ~(k | 0xffu));
    }
};
template <>
struct LogitKey<float> {
    typedef uint64_t type;
    static constexpr type kNone = 0x007fffffffffffffull;
    static __device__ __forceinline__ type make(float l, int e) {
        return ((uint64_t)ordered(l) << 32) | (uint32_t)~e;
    }
    static __device__ __forceinline__ int expert(type k) { return (int)~(uint32_t)k; }
    static __device__ __forceinline__ float logit(type k) {
        const uint32_t o = (uint32_t)(k >> 32);
        return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
    }
};

template <int NV>
__device__ __forceinline__ float row_exp_sum(const float (&l)[NV], float m) {
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) z += exp_neg(l[j] - m);  // 0 for -inf, whatever m is
    return row_sum(z);
}

template <typename S, int NV>
__global__ __launch_bounds__(kGateThreads) void gate_rows_kernel(GateArgs a, bool vec,
                                                                 int64_t* __restrict__ topk_idx,
                                                                 float* __restrict__ topk_weights) {
    typedef LogitKey<S> Key;
    const int lane = threadIdx.x & 15;
    const int t = blockIdx.x * kRowTokens + (threadIdx.x >> 4);
    float l[NV];
    load_logits<S, NV>(static_cast<const S*>(a.logits), a.E, min(t, a.T - 1), lane, vec, l);
    typedef typename Key::type key_t;
    key_t key[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) key[j] = Key::make(l[j], lane * NV + j);
    const bool softmax = a.score == MOEDX_GATE_SOFTMAX;
    // lane k keeps the k-th choice and its logit
    int mine = -1;
    float mine_l = kNegInf, m = 0.0f;
    key_t top = 0;
    for (int k = 0; k < a.K; ++k) {
        // The largest key below the last: of the differences to it, taken modulo
        // the type's range, those of smaller keys are the largest.
        key_t d = key[0] - top;
#pragma unroll
        for (int j = 1; j < NV; ++j) {
            const key_t o = key[j] - top;
            d = o > d ? o : d;
        }
        d = row_max(d);
        const key_t next = d + top;
        top = k == 0 || next < top ? next : 0;  // or there is none
        if (lane == k && top > Key::kNone) {
            mine = Key::expert(top);
            mine_l = Key::logit(top);
        }
        if (k == 0 && top > Key::kNone) m = Key::logit(top);
    }
    const bool have = mine >= 0;
    float w;
    if (a.renormalize)
        w = row_share(have, softmax, mine_l);
    else if (softmax)
        w = expf(mine_l - m) / row_exp_sum(l, m);
    else
        w = sigmoid(mine_l);
    if (lane < a.K && t < a.T) {
        topk_idx[(int64_t)t * a.K + lane] = mine;
        topk_weights[(int64_t)t * a.K + lane] = have ? a.scale * w : 0.0f;
    }
}

template <typename S, int NV>
__global__ __launch_bounds__(kGateThreads) void gate_rows_backward_kernel(
    GateArgs a, bool vec, const int64_t* __restrict__ topk_idx,
    const float* __restrict__ d_topk_weights, S* __restrict__ d_logits) {
    __shared__ __align__(16) float spread[kRowTokens][16 * NV];
    const int lane = threadIdx.x & 15, slot = threadIdx.x >> 4;
    const int t = min((int)blockIdx.x * kRowTokens + slot, a.T - 1);
    const S* logits = static_cast<const S*>(a.logits);
    const bool softmax = a.score == MOEDX_GATE_SOFTMAX;
    const bool dense = softmax && !a.renormalize;
    float l[NV];
    if (dense) load_logits<S, NV>(logits, a.E, t, lane, vec, l);
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
#pragma unroll
    for (int j = 0; j < NV; ++j) spread[slot][lane * NV + j] = 0.0f;
    const bool have = idx >= 0 && lk > kNegInf;
    float own = 0.0f;            // gradient added at the chosen expert
    float m = 0.0f, z = 1.0f, dot = 0.0f;
    if (a.renormalize) {
        const float v = row_share(have, softmax, lk);
        const float gv = row_sum(have ? g * v : 0.0f);
        own = a.scale * v * (g - gv);
        if (!softmax) own *= sigmoid(-lk);
    } else if (softmax) {  // p_j * scale * (g_j - dot) for every expert j
        m = l[0];
#pragma unroll
        for (int j = 1; j < NV; ++j) m = fmaxf(m, l[j]);
        m = row_max(m);
        z = row_exp_sum(l, m);
        dot = row_sum(have ? g * (expf(lk - m) / z) : 0.0f);
        own = g;
    } else {
        own = a.scale * g * sigmoid(lk) * sigmoid(-lk);
    }
    // the row's lanes are of one wave, whose LDS accesses keep their order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (have) atomicAdd(&spread[slot][idx], own);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const float per_z = a.scale / z;
    float d[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        d[j] = spread[slot][lane * NV + j];
    if (dense) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const float v = exp_neg(l[j] - m) * per_z * (d[j] - dot);
            d[j] = l[j] > kNegInf ? v : 0.0f;
        }
    }
    if ((int)blockIdx.x * kRowTokens + slot >= a.T) return;
    S* out = d_logits + (int64_t)t * a.E + lane * NV;
    if (vec) {
        typedef S vals __attribute__((ext_vector_type(NV)));
        vals v;
#pragma unroll
        for (int j = 0; j < NV; ++j) v[j] = (S)d[j];
        if (lane * NV < a.E) *reinterpret_cast<vals*>(out) = v;
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (lane * NV + j < a.E) out[j] = (S)d[j];
    }
}

// Whether rows can be moved NV values at a time (16 bytes at most).
template <typename S, int NV>
bool vector_rows(const GateArgs& a, const void* other) {
    constexpr uintptr_t kBytes = sizeof(S) * NV < 16 ? sizeof(S) * NV : 16;
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(other);
    return a.E % NV == 0 && (p | (a.E * sizeof(S))) % kBytes == 0;
}

// Calls f with NV, a power of two, such that `lanes` lanes of NV hold E experts.
template <int kLeast = 1, typename F>
hipError_t by_width(int E, int lanes, F&& f) {
    const int nv = (E + lanes - 1) / lanes;
    if constexpr (kLeast <= 1)
        if (nv <= 1) return f(std::integral_constant<int, 1>{});
    if constexpr (kLeast <= 2)
        if (nv <= 2) return f(std::integral_constant<int, 2>{});
    if constexpr (kLeast <= 4)
        if (nv <= 4) return f(std::integral_constant<int, 4>{});
    if (nv <= 8) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 16>{});
}

constexpr int kRowExperts = 256;  // a row of 16 lanes holds them

template <typename S>
hipError_t gate_as(const GateArgs& a, int64_t* idx, float* w, const Launch& L) {
    const dim3 waves((a.T + kGateWaves - 1) / kGateWaves), block(kGateThreads);
    if (a.bias != nullptr || a.groups > 1)
        return by_width(a.E, 64, [&](auto nv) {
            return launch_kernel(gate_topk_kernel<S, nv(), double>, waves, block, L, a,
                                 vector_rows<S, nv()>(a, nullptr), idx, w);
        });
    if (a.E > kRowExperts)
        return by_width<8>(a.E, 64, [&](auto nv) {
            return launch_kernel(gate_topk_kernel<S, nv(), uint32_t>, waves, block, L, a,
                                 vector_rows<S, nv()>(a, nullptr), idx, w);
        });
    return by_width(a.E, 16, [&](auto nv) {
        return launch_kernel(gate_rows_kernel<S, nv()>, dim3((a.T + kRowTokens - 1) / kRowTokens),
                             block, L, a, vector_rows<S, nv()>(a, nullptr), idx, w);
    });
}

template <typename S>
hipError_t gate_backward_as(const GateArgs& a, const int64_t* idx, const float* dw, void* dl,
                            const Launch& L) {
    const dim3 waves((a.T + kGateWaves - 1) / kGateWaves), block(kGateThreads);
    S* out = static_cast<S*>(dl);
    if (a.E > kRowExperts)
        return by_width<8>(a.E, 64, [&](auto nv) {
            return launch_kernel(gate_topk_backward_kernel<S, nv()>, waves, block, L, a,
                                 vector_rows<S, nv()>(a, dl), idx, dw, out);
        });
    return by_width(a.E, 16, [&](auto nv) {
        return launch_kernel(gate_rows_backward_kernel<S, nv()>,
                             dim3((a.T + kRowTokens - 1) / kRowTokens), block, L, a,
                             vector_rows<S, nv()>(a, dl), idx, dw, out);
    });
}

}  // namespace

hipError_t launch_gate_topk(const GateArgs& a, int64_t* idx, float* w, const Launch& L) {
    if (a.dtype == MOEDX_F32) return gate_as<float>(a, idx, w, L);
    if (a.dtype == MOEDX_F16) return gate_as<_Float16>(a, idx, w, L);
    return gate_as<__bf16>(a, idx, w, L);
}

hipError_t launch_gate_topk_backward(const GateArgs& a, const int64_t* idx, const float* dw,
                                     void* dl, const Launch& L) {
    if (a.dtype == MOEDX_F32) return gate_backward_as<float>(a, idx, dw, dl, L);
    if (a.dtype == MOEDX_F16) return gate_backward_as<_Float16>(a, idx, dw, dl, L);
    return gate_backward_as<__bf16>(a, idx, dw, dl, L);
}

}  // namespace moedx
