// Which expert a row tile belongs to (device code).  Tiles of BM rows are
// numbered expert by expert, an expert with c rows having ceil(c / BM) of
// them, so a launch needs no count on the host: its grid covers the most
// tiles that the buffer's rows can make, and workgroups past the last exit.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_launch.h"

namespace moedx {

struct RowSpan {
    int begin, end;
};

// Clamped to the buffer, whatever the arrays hold.
__device__ __forceinline__ RowSpan expert_span(const ExpertRows& er, int e) {
    if (er.offsets) {
        const int rows = (int)er.rows;
        const int b = min(max(er.offsets[e], 0), rows);
        return RowSpan{b, min(max(er.offsets[e + 1], b), rows)};
    }
    const int b = e * er.cap;
    return RowSpan{b, b + min(max(er.counts[e], 0), er.cap)};
}

struct RowTile {
    int e;           // expert, or -1 past the last tile
    int begin, end;  // the tile's rows
    int col;         // its column tile
};

// Tile `i` (wave-uniform; every lane of the wave takes part) where each expert
// has ceil(c / BM) x cols tiles: up to kGroup row tiles go through the columns
// together, so that tiles close in number share both operands.
template <int BM, int kGroup>
__device__ __forceinline__ RowTile find_block(const ExpertRows& er, int i, int cols) {
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int e0 = 0; e0 < er.E; e0 += 64) {
        const int e = e0 + lane;
        RowSpan s{0, 0};
        if (e < er.E) s = expert_span(er, e);
        const int t = row_tiles<BM>(s.end - s.begin);
        int incl = t;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(incl, d, 64);
            if (lane >= d) incl += v;
        }
        const uint64_t past = __ballot((int64_t)(base + incl) * cols > i);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int begin = __builtin_amdgcn_readlane(s.begin, l);
            const int end = __builtin_amdgcn_readlane(s.end, l);
            const int mine = __builtin_amdgcn_readlane(t, l);
            const int first = base + __builtin_amdgcn_readlane(incl - t, l);
            int local = i - first * cols;
            const int grp = local / (kGroup * cols);
            local -= grp * kGroup * cols;
            const int in_grp = min(kGroup, mine - grp * kGroup);
            const int col = local / in_grp;
            const int step = row_step<BM>(end - begin, mine);
            const int b = begin + (grp * kGroup + local - col * in_grp) * step;
            return RowTile{e0 + l, b, b + min(step, end - b), col};
        }
        base += __builtin_amdgcn_readlane(incl, 63);
    }
    return RowTile{-1, 0, 0, 0};
}

}  // namespace moedx
