// Checks the tile choice of the int8 products (expert_plan.h) on the host: over
// the documented range a choice's grid can be launched (HIP counts a grid's
// threads in 32 bits), nothing is refused that 256 x 256 tiles can do, the rules'
// examples are taken, and an expert's rows are all in its tiles.
#include <cmath>
#include <cstdio>
#include <random>

#include "expert_plan.h"

using namespace moedx;

static ExpertRows with_counts(int E, int64_t cap) {
    static const int32_t any = 0;
    return ExpertRows{nullptr, &any, (int)cap, E, (int64_t)E * cap};
}
static ExpertRows with_offsets(int E, int64_t rows) {
    static const int32_t any = 0;
    return ExpertRows{&any, nullptr, 0, E, rows};
}

static int64_t threads(const ExpertRows& er, int64_t bm, int64_t outs_per_tile, int threads_per, int outs) {
    int64_t tiles = 0;
    if (er.offsets) {
        tiles = er.rows / bm + er.E;
        if (tiles > er.rows) tiles = er.rows;
    } else {
        tiles = (int64_t)er.E * ((er.cap + bm - 1) / bm);
    }
    return tiles * ((outs + outs_per_tile - 1) / outs_per_tile) * threads_per;
}

static bool check(const ExpertRows& er, int outs) {
    const int64_t limit = (int64_t)1 << 32;
    const Int8Tiles got = int8_tiles(er, outs);
    int64_t n = 0;
    switch (got) {
        case Int8Tiles::kNarrow: n = threads(er, 32, 64, 256, outs); break;
        case Int8Tiles::kOnce:
        case Int8Tiles::kDeepOnce:
        case Int8Tiles::kDeep: n = threads(er, 128, 128, 256, outs); break;
        case Int8Tiles::kWide: n = threads(er, 256, 256, 512, outs); break;
        case Int8Tiles::kNone: n = 0; break;
    }
    const bool refused = got == Int8Tiles::kNone;
    if (n < limit && (!refused || threads(er, 256, 256, 512, outs) >= limit)) return true;
    std::printf("FAIL %s E=%d cap=%d rows=%lld outs=%d: choice %d\n", er.offsets ? "offsets" : "counts",
                er.E, er.cap, (long long)er.rows, outs, (int)got);
    return false;
}

template <int BM>
static bool split(int64_t count) {
    const int64_t tiles = row_tiles<BM>((int)count), step = row_step<BM>((int)count, (int)tiles);
    return tiles == (count + BM - 1) / BM && step > 0 && step <= BM && (tiles - 1) * step < count &&
           tiles * step >= count;
}

static bool check_split(int64_t count) {
    return split<32>(count) && split<128>(count) && split<256>(count);
}

int main() {
    const struct {
        ExpertRows er;
        int outs;
        Int8Tiles want;
    } examples[] = {
        {with_offsets(64, 8), 4096, Int8Tiles::kNarrow},      // one token's experts
        {with_offsets(64, 256), 4096, Int8Tiles::kOnce},      // a few rows in each
        {with_offsets(64, 256), 1408, Int8Tiles::kDeepOnce},  // about a tile per workgroup
        {with_offsets(64, 4096), 4096, Int8Tiles::kOnce},
        {with_offsets(64, 32768), 4096, Int8Tiles::kWide},
        {with_offsets(8, 512), 4096, Int8Tiles::kDeepOnce},   // too few wide tiles
        {with_offsets(8, 1024), 4096, Int8Tiles::kDeepOnce},
        {with_offsets(8, 2048), 2048, Int8Tiles::kDeep},
        {with_offsets(1, 256), 8192, Int8Tiles::kDeep},
        {with_offsets(1, 32), 8192, Int8Tiles::kNarrow},
        {with_counts(64, 128), 4096, Int8Tiles::kOnce},       // a decode batch's slots
        {with_counts(64, 32), 4096, Int8Tiles::kDeepOnce},    // a few tokens'
        {with_counts(64, 1), 4096, Int8Tiles::kNarrow},
        {with_counts(1024, 128), 1024, Int8Tiles::kDeepOnce},
        {with_counts(64, 4096), 4096, Int8Tiles::kWide},
        {with_counts(1024, 1 << 20), 16384, Int8Tiles::kNone},
        {with_offsets(1, INT32_MAX), 8, Int8Tiles::kNone},
        {with_offsets(1, ((int64_t)1 << 31) - 513), 8, Int8Tiles::kWide},
    };
    int n = 0;
    for (const auto& x : examples) {
        const Int8Tiles got = int8_tiles(x.er, x.outs);
        if (got != x.want) {
            std::printf("FAIL example %d: %d, expected %d\n", n, (int)got, (int)x.want);
            return 1;
        }
        ++n;
    }
    std::mt19937_64 rng(1);
    const auto log_uniform = [&](double top) {
        return (int64_t)std::exp2(std::uniform_real_distribution<double>(0.0, std::log2(top))(rng));
    };
    for (int i = 0; i < 2000000; ++i) {
        const int E = (int)log_uniform(1025.0);
        const int64_t rows = log_uniform(2147483648.0);
        const int outs = (int)(8 * log_uniform(262145.0));
        if (!check(with_offsets(E, rows), outs) || !check(with_counts(E, rows / E), outs)) return 1;
    }
    for (int64_t count = 1; count < 100000; ++count)
        if (!check_split(count) || !check_split(INT32_MAX - count + 1)) {
            std::printf("FAIL %lld rows\n", (long long)count);
            return 1;
        }
    std::printf("ok %d\n", n);
    return 0;
}
