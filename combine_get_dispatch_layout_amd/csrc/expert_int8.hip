// The experts' rows in int8 for gfx950: quantised (in place of order, or moved
// into expert order), restored, and the gated activation's gradient from saved
// (gate, up) values.
//
// A group (a row, or 128 values of it) with largest magnitude a:
//   m = max(a, 2^-100), scale = m / 127, code = nearest even of x (127 / m),
// every operation one fp32 rounding, so |code| <= 127 without a clamp (x (127 /
// m) is at most 127 (1 + 2^-23)^2) and codes are the same on any machine.
// Restored, a value is code * scale: off by at most half a scale and 2^-22 of
// itself (but fp32's largest finite value comes back as inf).  The floor keeps
// 127 / m finite; values below 2^-108 become 0.  Magnitudes are compared as bit
// patterns, NaN above inf: a group that holds one gets a scale of inf or NaN and
// is NaN when it is restored.
//
// All of it is bound by memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_launch.h"
#include "expert_tile.h"
#include "moedx.h"
#include "numeric.h"

namespace moedx {

namespace {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int64_t kGrid = 1 << 20;  // workgroups at most: they go on through the rows

// Cache policy of loads (the intrinsics' bits) and stores that pass the caches
// by: rows that are read once, and what the next call is not likely to read.
constexpr int kStream = 2;
template <typename V>
__device__ __forceinline__ void stream(V* at, V v) {
    __builtin_nontemporal_store(v, at);
}

// Eight values of type S: what a lane takes of a row at a time.  fp32 needs two
// loads that share cache lines, so these stay in the caches (49152 rows of 4096
// bf16 values 104 us for 112, half as many fp32 ones 94 for 105 the other way).
template <typename S>
struct Unit {
    static constexpr int kChunks = (int)sizeof(S) / 2;
    static constexpr int kPolicy = kChunks == 1 ? kStream : 0;
    u32x4_t c[kChunks];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            c[i] = __builtin_bit_cast(
                u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, (int)(off + i * 16), 0,
                                                                kPolicy));
    }
    __device__ __forceinline__ void values(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            float part[Chunk<S>::kN];
            chunk_to_f32<S>(c[i], part);
#pragma unroll
            for (int j = 0; j < Chunk<S>::kN; ++j) f[i * Chunk<S>::kN + j] = part[j];
        }
    }
    // Adds its magnitudes to `top`: bit patterns, two of 16 bits or one of 32.
    __device__ __forceinline__ uint32_t magnitude(uint32_t top) const {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(S) == 2)
                    top = __builtin_bit_cast(
                        uint32_t,
                        __builtin_elementwise_max(__builtin_bit_cast(u16x2, top),
                                                  __builtin_bit_cast(u16x2, c[i][j] & 0x7fff7fffu)));
                else
                    top = max(top, c[i][j] & 0x7fffffffu);
            }
        return top;
    }
};
// One bit pattern of what magnitude() gave, and its value.
template <typename S>
__device__ __forceinline__ uint32_t one_magnitude(uint32_t top) {
    return sizeof(S) == 2 ? max(top >> 16, top & 0xffffu) : top;
}
template <typename S>
__device__ __forceinline__ float magnitude_value(uint32_t bits) {
    if constexpr (sizeof(S) == 2) return (float)__builtin_bit_cast(S, (uint16_t)bits);
    else return __builtin_bit_cast(float, bits);
}

struct Scale {
    float scale, factor;
    __device__ __forceinline__ explicit Scale(float a) {
        const float m = a < 0x1p-100f ? 0x1p-100f : a;  // NaN stays
        scale = m / 127.0f;
        factor = 127.0f / m;
    }
};

// Adding 1.5 * 2^23 leaves the nearest integer in the low bits.
__device__ __forceinline__ uint32_t code_bits(float x, float factor) {
    return __builtin_bit_cast(uint32_t, x * factor + 12582912.0f);
}
template <typename S>
__device__ __forceinline__ u32x2_t codes_of(const Unit<S>& v, float factor) {
    float f[8];
    v.values(f);
    u32x2_t o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t a = code_bits(f[4 * i], factor), b = code_bits(f[4 * i + 1], factor);
        const uint32_t c = code_bits(f[4 * i + 2], factor), d = code_bits(f[4 * i + 3], factor);
        o[i] = __builtin_amdgcn_perm(b, a, 0x0c0c0400u) | __builtin_amdgcn_perm(d, c, 0x04000c0cu);
    }
    return o;
}

// The eight values of a lane's codes.
__device__ __forceinline__ void restored(u32x2_t c, float scale, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = in_fp32((float)(int8_t)(c[i >> 2] >> (8 * (i & 3))) * scale);
}

// The rows of the buffer that are an expert's (with neither array, all), in
// groups of up to `per`.  Slots are taken place by place through the experts:
// expert by expert, the live ones (the first of each expert's) would fall to
// workgroups a multiple of 8 apart and so to a few of the XCDs (64 experts of 12 live
// rows in 128 slots, 4096 bf16 values, the kernel alone: from memory 10.8 us, this way
// 5.0; with the rows in the caches 7.9 and 3.8).
struct LiveRows {
    ExpertRows er;
    FastDiv experts;  // by er.E
    int64_t groups;
    int per;

    // Calls f(first, n) for groups i, i + step, ... that have live rows.  i does
    // not depend on the lane.
    template <typename F>
    __device__ __forceinline__ void each(int64_t i, int64_t step, F&& f) const {
        if (er.counts) {
            for (; i < groups; i += step) {
                const int j = (int)experts.div((uint32_t)i), e = (int)(i - (int64_t)j * er.E);
                const int slot = j * per;
                const int n = min(min(er.counts[e], er.cap) - slot, per);
                if (n > 0) f((int64_t)e * er.cap + slot, n);
            }
            return;
        }
        int64_t lo = 0, hi = er.rows;
        if (er.offsets) {
            lo = max(lo, (int64_t)er.offsets[0]);
            hi = min(hi, (int64_t)er.offsets[er.E]);
        }
        for (; i < groups; i += step) {
            const int64_t first = max(i * per, lo), end = min(i * per + per, hi);
            if (first < end) f(first, (int)(end - first));
        }
    }
};

// A row by one wave, held in registers between its largest magnitude and its
// codes: NU units a lane; longer rows (kLong) are read twice.  49146 rows of 4096
// bf16 values, a scale each: 105 us (5.8 TB/s).  `to` gives the
// codes and the scale their places.
template <typename S, int NU, bool kLong, typename F>
__device__ __forceinline__ void quantize_row(const S* x, int H, int lane, F&& to) {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(x, H * (int)sizeof(S));
    constexpr int kSpan = 64 * 8 * NU;  // values of one batch of loads
    Unit<S> v[NU];
    uint32_t top = 0;
    const auto fetch = [&](int at) {
#pragma unroll
        for (int u = 0; u < NU; ++u)
            v[u].load(rs, (uint32_t)(at + (u * 64 + lane) * 8) * (uint32_t)sizeof(S));
    };
    for (int at = 0; at < (kLong ? H : 1); at += kSpan) {
        fetch(at);
#pragma unroll
        for (int u = 0; u < NU; ++u) top = v[u].magnitude(top);
    }
    const Scale s(magnitude_value<S>(wave_max(one_magnitude<S>(top))));
    for (int at = 0; at < (kLong ? H : 1); at += kSpan) {
        if (kLong) fetch(at);
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int k = at + (u * 64 + lane) * 8;
            const u32x2_t c = codes_of(v[u], s.factor);
            if (k < H) to.codes(k, c);
        }
    }
    if (lane == 0) to.scale(s.scale);
}

template <typename S, int NU, bool kLong>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const S* x, LiveRows live, int H,
                                                                 int8_t* codes, float* scales) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    live.each((int64_t)blockIdx.x * kWaves + wave, (int64_t)gridDim.x * kWaves,
              [&](int64_t row, int) {
                  struct {
                      int8_t* c;
                      float* s;
                      __device__ __forceinline__ void codes(int k, u32x2_t v) const {
                          *reinterpret_cast<u32x2_t*>(c + k) = v;
                      }
                      __device__ __forceinline__ void scale(float v) const { *s = v; }
                  } to{codes + row * H, scales + row};
                  quantize_row<S, NU, kLong>(x + row * H, H, lane, to);
              });
}

// A token's row, quantised once, at the rows of its filled slots.
template <typename S, int NU, bool kLong>
__global__ __launch_bounds__(kThreads) void sort_int8_kernel(const S* x, int T, int K, int H,
                                                             int64_t rows,
                                                             const int32_t* row_of_slot,
                                                             int8_t* codes, float* scales) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < T; t += (int64_t)gridDim.x * kWaves) {
        int row = -1;
        if (lane < K) row = row_of_slot[t * K + lane];
        uint64_t filled = __ballot(row >= 0 && row < rows);
        if (!filled) continue;
        struct {
            int8_t* c;
            float* s;
            uint64_t filled;
            int row, H;
            __device__ __forceinline__ void codes(int k, u32x2_t v) const {
                for (uint64_t f = filled; f; f &= f - 1) {
                    const int64_t r = __builtin_amdgcn_readlane(row, __builtin_ctzll(f));
                    *reinterpret_cast<u32x2_t*>(c + r * H + k) = v;
                }
            }
            __device__ __forceinline__ void scale(float v) const {
                for (uint64_t f = filled; f; f &= f - 1)
                    s[__builtin_amdgcn_readlane(row, __builtin_ctzll(f))] = v;
            }
        } to{codes, scales, filled, row, H};
        quantize_row<S, NU, kLong>(x + t * H, H, lane, to);
    }
}

constexpr int kBlock = 128, kBlockLanes = kBlock / 8;  // a lane has 8 values

// What a lane (or 16) takes of a row at a time: so many to a row.
struct RowItems {
    int n;
    FastDiv div;  // by n
};

// 16 lanes to a block of 128 values.  49146 rows of 4096 bf16 values: 98 us (6.1
// TB/s).
template <typename S>
__global__ __launch_bounds__(kThreads) void quantize_blocks_kernel(const S* x, LiveRows live, int H,
                                                                   RowItems items, int8_t* codes,
                                                                   float* scales) {
    constexpr int U = 4, kSlots = kThreads / kBlockLanes;
    const int in = threadIdx.x % kBlockLanes, slot = threadIdx.x / kBlockLanes;
    const auto some = [&](int64_t row0, int rows) {
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(x + row0 * H, rows * H * (int)sizeof(S));
        int8_t* const c0 = codes + row0 * H;
        float* const s0 = scales + row0 * items.n;
        for (int i0 = slot; i0 < rows * items.n; i0 += U * kSlots) {
            Unit<S> v[U];
            int at[U];
            bool here[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * kSlots;
                const int r = (int)items.div.div((uint32_t)i), k = (i - r * items.n) * kBlock + in * 8;
                here[u] = i < rows * items.n && k < H;
                at[u] = r * H + k;
                v[u].load(rs, here[u] ? (uint32_t)at[u] * (uint32_t)sizeof(S) : kOutside);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Scale s(magnitude_value<S>(row_max(one_magnitude<S>(v[u].magnitude(0)))));
                const u32x2_t c = codes_of(v[u], s.factor);
                if (!here[u]) continue;
                stream(reinterpret_cast<u32x2_t*>(c0 + at[u]), c);
                if (in == 0) s0[i0 + u * kSlots] = s.scale;
            }
        }
    };
    live.each(blockIdx.x, gridDim.x, some);
}

template <typename S>
__device__ __forceinline__ void store_unit(S* at, const float (&f)[8]) {
    constexpr int N = Chunk<S>::kN;
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) {
        float part[N];
#pragma unroll
        for (int j = 0; j < N; ++j) part[j] = f[i * N + j];
        stream(reinterpret_cast<u32x4_t*>(at + i * N), chunk_from_f32<S>(part));
    }
}

__device__ __forceinline__ u32x2_t load_codes(__amdgpu_buffer_rsrc_t rs, int at) {
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(rs, at, 0, kStream));
}
__device__ __forceinline__ float load_scale(__amdgpu_buffer_rsrc_t rs, int at) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, at * 4, 0, 0));
}

// groups: scales of a row, 0 = one for all of it (here and below).  49146 rows of
// 4096: 98 us (6.1 TB/s; 120 where each item asked whether its row is live, a
// load ahead of its own).
template <typename S>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const int8_t* codes,
                                                              const float* scales, LiveRows live,
                                                              int H, int groups, RowItems items,
                                                              S* x) {
    constexpr int U = 4;
    const int per_row = groups ? groups : 1;
    const auto some = [&](int64_t row0, int rows) {
        const __amdgpu_buffer_rsrc_t rc = make_rsrc(codes + row0 * H, rows * H);
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(scales + row0 * per_row, rows * per_row * 4);
        S* const out = x + row0 * H;
        for (int i0 = threadIdx.x; i0 < rows * items.n; i0 += U * kThreads) {
            u32x2_t c[U];
            float s[U];
            int at[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // past the last item loads give zeros: rows' offsets end the range
                const int i = i0 + u * kThreads;
                const int r = (int)items.div.div((uint32_t)i), k = (i - r * items.n) * 8;
                at[u] = r * H + k;
                c[u] = load_codes(rc, at[u]);
                s[u] = load_scale(rs, r * per_row + (groups ? k / kBlock : 0));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[8];
                restored(c[u], s[u], f);
                if (i0 + u * kThreads < rows * items.n) store_unit<S>(out + at[u], f);
            }
        }
    };
    live.each(blockIdx.x, gridDim.x, some);
}

// Two items' loads at a time: 49146 rows of 2 x 2048, h with it, bf16: 165 us (6.1
// TB/s; one item 167, four 171; through the caches 176).
template <typename S>
__global__ __launch_bounds__(kThreads) void swiglu_backward_int8_kernel(
    const S* d_h, const int8_t* codes, const float* scales, LiveRows live, int N, int groups,
    RowItems items, S* d_pre, S* h) {
    constexpr int U = 2;
    const int per_row = groups ? groups : 1;
    const auto some = [&](int64_t row0, int rows) {
        const __amdgpu_buffer_rsrc_t rc = make_rsrc(codes + row0 * 2 * N, rows * 2 * N);
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(scales + row0 * per_row, rows * per_row * 4);
        const __amdgpu_buffer_rsrc_t rd = make_rsrc(d_h + row0 * N, rows * N * 2);
        for (int i0 = threadIdx.x; i0 < rows * items.n; i0 += U * kThreads) {
            Unit<S> dv[U];
            u32x2_t gc[U], uc[U];
            float sg[U], su[U];
            int r[U], k[U];
#pragma unroll
            for (int v = 0; v < U; ++v) {
                const int i = i0 + v * kThreads;
                r[v] = (int)items.div.div((uint32_t)i);
                k[v] = (i - r[v] * items.n) * 8;
                dv[v].load(rd, (uint32_t)(r[v] * N + k[v]) * 2);
                gc[v] = load_codes(rc, r[v] * 2 * N + k[v]);
                uc[v] = load_codes(rc, r[v] * 2 * N + N + k[v]);
                sg[v] = load_scale(rs, r[v] * per_row + (groups ? k[v] / kBlock : 0));
                su[v] = load_scale(rs, r[v] * per_row + (groups ? (N + k[v]) / kBlock : 0));
            }
#pragma unroll
            for (int v = 0; v < U; ++v) {
                float d[8], g[8], u[8], out[8];
                dv[v].values(d);
                restored(gc[v], sg[v], g);
                restored(uc[v], su[v], u);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float s = 1.0f / (1.0f + expf(-g[j]));
                    const float gs = g[j] * s;
                    out[j] = gs * u[j];
                    const float du = d[j] * gs;
                    g[j] = d[j] * u[j] * s * (1.0f + g[j] * (1.0f - s));
                    u[j] = du;
                }
                if (i0 + v * kThreads >= rows * items.n) break;
                const int64_t row = row0 + r[v];
                store_unit<S>(d_pre + row * 2 * N + k[v], g);
                store_unit<S>(d_pre + row * 2 * N + N + k[v], u);
                if (h) store_unit<S>(h + row * N + k[v], out);
            }
        }
    };
    live.each(blockIdx.x, gridDim.x, some);
}

RowItems row_items(int of_row) { return RowItems{of_row, make_fastdiv((uint32_t)of_row)}; }
// Rows to a workgroup: about `n` items, a row at least, so that narrow rows fill
// it too.
int rows_per(const RowItems& items, int n) { return n > items.n ? n / items.n : 1; }

LiveRows live_rows(const ExpertRows& er, int per) {
    const int64_t groups = er.counts ? er.E * tiles_of(er.cap, per) : tiles_of(er.rows, per);
    return LiveRows{er, make_fastdiv((uint32_t)er.E), groups, per};
}
dim3 grid_of(int64_t workgroups) {
    return dim3((unsigned)(workgroups < kGrid ? workgroups : kGrid));
}

// Calls f with the number of units per lane that hold a row, and whether it is
// longer than any.
template <typename F>
hipError_t with_units(int H, F&& f) {
    const int units = (H + 511) / 512;
    if (units <= 1) return f(std::integral_constant<int, 1>{}, std::false_type{});
    if (units <= 2) return f(std::integral_constant<int, 2>{}, std::false_type{});
    if (units <= 4) return f(std::integral_constant<int, 4>{}, std::false_type{});
    if (units <= 8) return f(std::integral_constant<int, 8>{}, std::false_type{});
    if (units <= 16) return f(std::integral_constant<int, 16>{}, std::false_type{});
    return f(std::integral_constant<int, 8>{}, std::true_type{});
}

template <typename S>
hipError_t quantize_as(const void* x, const ExpertRows& er, int H, int block, int8_t* codes,
                       float* scales, const Launch& L) {
    const S* xs = static_cast<const S*>(x);
    if (block) {
        const RowItems items = row_items((H + kBlock - 1) / kBlock);
        const LiveRows live = live_rows(er, rows_per(items, 64));
        return launch_kernel(quantize_blocks_kernel<S>, grid_of(live.groups), dim3(kThreads), L, xs,
                             live, H, items, codes, scales);
    }
    return with_units(H, [&](auto nu, auto longer) {
        const LiveRows live = live_rows(er, 1);
        return launch_kernel(quantize_rows_kernel<S, decltype(nu)::value, decltype(longer)::value>,
                             grid_of(tiles_of(live.groups, kWaves)), dim3(kThreads), L, xs, live, H,
                             codes, scales);
    });
}

template <typename S>
hipError_t sort_int8_as(const void* x, int T, int K, int H, const int32_t* row_of_slot,
                        int8_t* codes, float* scales, const Launch& L) {
    return with_units(H, [&](auto nu, auto longer) {
        return launch_kernel(sort_int8_kernel<S, decltype(nu)::value, decltype(longer)::value>,
                             grid_of(tiles_of(T, kWaves)), dim3(kThreads), L,
                             static_cast<const S*>(x), T, K, H, (int64_t)T * K, row_of_slot, codes,
                             scales);
    });
}

template <typename S>
hipError_t dequantize_as(const int8_t* codes, const float* scales, const ExpertRows& er, int H,
                         int block, void* x, const Launch& L) {
    const RowItems items = row_items(H / 8);
    const LiveRows live = live_rows(er, rows_per(items, 4 * kThreads));
    return launch_kernel(dequantize_kernel<S>, grid_of(live.groups), dim3(kThreads), L, codes,
                         scales, live, H, block ? (H + kBlock - 1) / kBlock : 0, items,
                         static_cast<S*>(x));
}

template <typename S>
hipError_t swiglu_backward_int8_as(const void* d_h, const int8_t* codes, const float* scales,
                                   const ExpertRows& er, int N, int block, void* d_pre, void* h,
                                   const Launch& L) {
    const RowItems items = row_items(N / 8);
    const LiveRows live = live_rows(er, rows_per(items, 2 * kThreads));
    return launch_kernel(swiglu_backward_int8_kernel<S>, grid_of(live.groups), dim3(kThreads), L,
                         static_cast<const S*>(d_h), codes, scales, live, N,
                         block ? (2 * N + kBlock - 1) / kBlock : 0, items, static_cast<S*>(d_pre),
                         static_cast<S*>(h));
}

}  // namespace

hipError_t launch_expert_quantize(const void* x, int dtype, const ExpertRows& er, int H, int block,
                                  int8_t* codes, float* scales, const Launch& L) {
    const auto as = dtype == MOEDX_F32   ? quantize_as<float>
                    : dtype == MOEDX_F16 ? quantize_as<_Float16>
                                         : quantize_as<__bf16>;
    return as(x, er, H, block, codes, scales, L);
}

hipError_t launch_expert_sort_int8(const void* x, int dtype, int T, int K, int H,
                                   const int32_t* row_of_slot, int8_t* codes, float* scales,
                                   const Launch& L) {
    const auto as = dtype == MOEDX_F32   ? sort_int8_as<float>
                    : dtype == MOEDX_F16 ? sort_int8_as<_Float16>
                                         : sort_int8_as<__bf16>;
    return as(x, T, K, H, row_of_slot, codes, scales, L);
}

hipError_t launch_expert_dequantize(const int8_t* codes, const float* scales, const ExpertRows& er,
                                    int H, int block, void* x, int dtype, const Launch& L) {
    const auto as = dtype == MOEDX_F32   ? dequantize_as<float>
                    : dtype == MOEDX_F16 ? dequantize_as<_Float16>
                                         : dequantize_as<__bf16>;
    return as(codes, scales, er, H, block, x, L);
}

hipError_t launch_swiglu_backward_int8(const void* d_h, const int8_t* codes, const float* scales,
                                       int block, int dtype, const ExpertRows& er, int N,
                                       void* d_pre, void* h, const Launch& L) {
    const auto as =
        dtype == MOEDX_F16 ? swiglu_backward_int8_as<_Float16> : swiglu_backward_int8_as<__bf16>;
    return as(d_h, codes, scales, er, N, block, d_pre, h, L);
}

}  // namespace moedx
