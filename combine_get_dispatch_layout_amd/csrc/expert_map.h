// Which expert a row tile belongs to (device code).  Tiles of BM rows are
// numbered expert by expert, an expert with c rows having ceil(c / BM) of
// them, so a launch needs no count on the host: its grid covers the most
// tiles that the buffer's rows can make, and workgroups past the last exit.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_launch.h"
#include "numeric.h"

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

// Tile `local` of expert e, whose rows begin .. end have `mine` row tiles.
template <int BM, int kGroup>
__device__ __forceinline__ RowTile tile_of(int e, int begin, int end, int mine, int local, int cols) {
    const int grp = local / (kGroup * cols);
    local -= grp * kGroup * cols;
    const int in_grp = min(kGroup, mine - grp * kGroup);
    const int col = local / in_grp;
    const int step = row_step<BM>(end - begin, mine);
    const int b = begin + (grp * kGroup + local - col * in_grp) * step;
    return RowTile{e, b, b + min(step, end - b), col};
}

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
            return tile_of<BM, kGroup>(e0 + l, __builtin_amdgcn_readlane(s.begin, l),
                                       __builtin_amdgcn_readlane(s.end, l),
                                       __builtin_amdgcn_readlane(t, l),
                                       i - (base + __builtin_amdgcn_readlane(incl - t, l)) * cols,
                                       cols);
        }
        base += __builtin_amdgcn_readlane(incl, 63);
    }
    return RowTile{-1, 0, 0, 0};
}

// find_block for growing tile numbers: the rows of the 64 experts that the last
// tile was found among may be asked for ahead.
struct TileSearch {
    const int32_t* rows;  // offsets or counts
    int last;             // their last entry
    int e0 = 0, base = 0;  // the first of 64 experts, tiles before them
    struct Entries {
        int a, b;
    };

    __device__ __forceinline__ explicit TileSearch(const ExpertRows& er)
        : rows(er.offsets ? er.offsets : er.counts), last(er.offsets ? er.E : er.E - 1) {}
    __device__ __forceinline__ Entries ask(int lane) const {
        return Entries{rows[min(e0 + lane, last)], rows[min(e0 + lane + 1, last)]};
    }
    template <int BM, int kGroup>
    __device__ __forceinline__ RowTile find(const ExpertRows& er, Entries n, int lane, int i,
                                            int cols) {
        for (;;) {
            const int all = (int)er.rows, first = er.offsets ? n.a : min(e0 + lane, er.E) * er.cap;
            const int begin = min(max(first, 0), all);
            const int end = er.offsets ? min(max(n.b, begin), all)
                            : e0 + lane < er.E ? begin + min(max(n.a, 0), er.cap)
                                               : begin;
            const int t = row_tiles<BM>(end - begin);
            const int incl = wave_scan(t);
            const uint64_t past = __ballot((int64_t)(base + incl) * cols > i);
            if (past) {
                const int l = __builtin_ctzll(past);
                return tile_of<BM, kGroup>(e0 + l, __builtin_amdgcn_readlane(begin, l),
                                           __builtin_amdgcn_readlane(end, l),
                                           __builtin_amdgcn_readlane(t, l),
                                           i - (base + __builtin_amdgcn_readlane(incl - t, l)) * cols,
                                           cols);
            }
            if (e0 + 64 >= er.E) return RowTile{-1, 0, 0, 0};
            base += __builtin_amdgcn_readlane(incl, 63);
            e0 += 64;
            n = ask(lane);
        }
    }
};

}  // namespace moedx
