// Checks the tile choice of the experts' products (expert_plan.h) on the host:
// over the documented range a choice's grid can be launched (HIP counts a
// grid's threads in 32 bits) and covers every row and column, the preferred
// tiles are taken where they can be, and nothing is refused that 256 x 256
// tiles can do.  And an expert's rows, up to 2^31 - 1, are all in its tiles.
#include <cmath>
#include <cstdio>
#include <random>

#include "expert_plan.h"

using namespace moedx;

static int64_t threads(const ExpertRows& er, const TileShape& t, int outs) {
    int64_t tiles = 0;
    if (er.offsets) {
        tiles = er.rows / t.rows + er.E;
        if (tiles > er.rows) tiles = er.rows;
    } else {
        tiles = (int64_t)er.E * (((int64_t)er.cap + t.rows - 1) / t.rows);
    }
    return tiles * (((int64_t)outs + t.outs - 1) / t.outs) * t.threads;
}

static const char* name(Tiles t) {
    static const char* const names[] = {"few", "small", "wide", "none"};
    return names[(int)t];
}

static bool check(const ExpertRows& er, int outs) {
    const int64_t limit = (int64_t)1 << 32;
    const int64_t few = threads(er, kFewTile, outs), small = threads(er, kSmallTile, outs),
                  wide = threads(er, kWideTile, outs);
    const int64_t likely = er.offsets ? er.rows / er.E : er.E > 8 ? (int64_t)er.cap * 8 / er.E : er.cap;
    const int64_t wide_tiles = ((likely + 255) / 256) * er.E * (((int64_t)outs + 255) / 256);
    const auto row_tiles_of = [&](const TileShape& t) { return threads(er, t, t.outs) / t.threads; };
    const int64_t t32 = row_tiles_of(kFewTile), t128 = row_tiles_of(kSmallTile),
                  t256 = row_tiles_of(kWideTile);
    Tiles want = Tiles::kWide;
    if (wide_tiles < 256 || (likely <= 48 && (er.offsets || t128 <= 512 || t128 == t256)))
        want = Tiles::kSmall;
    if (likely <= 8 && (er.offsets ? t32 : t32 * ((er.E + 63) / 64)) <= 256) want = Tiles::kFew;
    Tiles back = wide_tiles < 256 ? Tiles::kSmall : Tiles::kWide;
    if (want == Tiles::kFew && few >= limit) want = Tiles::kSmall;
    if (want == Tiles::kSmall && small >= limit) want = Tiles::kWide;
    if (want == Tiles::kWide && wide >= limit) want = Tiles::kNone;
    if (back == Tiles::kSmall && small >= limit) back = Tiles::kWide;
    if (back == Tiles::kWide && wide >= limit) back = Tiles::kNone;
    const Tiles got = forward_tiles(er, outs), got_back = input_gradient_tiles(er, outs);
    if (got == want && got_back == back) return true;
    std::printf("FAIL %s E=%d cap=%d rows=%lld outs=%d: %s, expected %s; back %s, expected %s\n",
                er.offsets ? "offsets" : "counts", er.E, er.cap, (long long)er.rows, outs, name(got),
                name(want), name(got_back), name(back));
    return false;
}

static ExpertRows with_counts(int E, int cap) {
    static const int32_t any = 0;
    return ExpertRows{nullptr, &any, cap, E, (int64_t)E * cap};
}
static ExpertRows with_offsets(int E, int64_t rows) {
    static const int32_t any = 0;
    return ExpertRows{&any, nullptr, 0, E, rows};
}

// The tiles of an expert's rows are not empty, at most BM rows each, and cover
// all of them.
template <int BM>
static bool check_split(int64_t count) {
    const int64_t tiles = row_tiles<BM>((int)count), step = row_step<BM>((int)count, (int)tiles);
    if (tiles == (count + BM - 1) / BM && step > 0 && step <= BM && (tiles - 1) * step < count &&
        tiles * step >= count)
        return true;
    std::printf("FAIL %lld rows in tiles of %d: %lld of %lld\n", (long long)count, BM,
                (long long)tiles, (long long)step);
    return false;
}

int main() {
    // slots of 1024 experts whose likely rows are few: 32-row tiles of the
    // capacity would be 2^24 workgroups of 256 threads
    if (grid_fits(workgroups(with_counts(1024, 1024), kFewTile, 16384), kFewTile.threads) ||
        forward_tiles(with_counts(1024, 1024), 16384) != Tiles::kWide) {
        std::printf("FAIL slots of 1024 experts\n");
        return 1;
    }
    // a decode batch's slots, many experts, and rows that may all be of a few
    if (forward_tiles(with_counts(64, 71), 4096) != Tiles::kFew ||
        forward_tiles(with_counts(128, 64), 4096) != Tiles::kSmall ||
        forward_tiles(with_counts(256, 128), 4096) != Tiles::kSmall ||
        forward_tiles(with_counts(1024, 512), 4096) != Tiles::kWide ||
        forward_tiles(with_offsets(64, 512), 4096) != Tiles::kFew ||
        forward_tiles(with_offsets(256, 2048), 4096) != Tiles::kSmall ||
        forward_tiles(with_offsets(1024, 8192), 4096) != Tiles::kSmall ||
        forward_tiles(with_offsets(1024, 8), 4096) != Tiles::kFew) {
        std::printf("FAIL many experts\n");
        return 1;
    }
    if (forward_tiles(with_offsets(1, INT32_MAX), 8) != Tiles::kNone ||
        forward_tiles(with_offsets(1, ((int64_t)1 << 31) - 513), 8) != Tiles::kWide) {
        std::printf("FAIL the largest buffers\n");
        return 1;
    }
    if (max_tiles(with_counts(1, INT32_MAX), 256) != (1 << 23)) {
        std::printf("FAIL tiles of the largest capacity\n");
        return 1;
    }
    std::mt19937_64 rng(1);
    const auto log_uniform = [&](double top) {
        return (int64_t)std::exp2(std::uniform_real_distribution<double>(0.0, std::log2(top))(rng));
    };
    int n = 0;
    for (; n < 2000000; ++n) {
        const int E = (int)log_uniform(1025.0);
        const int64_t rows = log_uniform(2147483648.0);
        const int outs = (int)(8 * log_uniform(262145.0));
        if (!check(with_offsets(E, rows), outs) || !check(with_counts(E, (int)(rows / E)), outs))
            return 1;
    }
    const auto splits = [&](int64_t count) {
        return check_split<32>(count) && check_split<128>(count) && check_split<256>(count);
    };
    for (int64_t count = 1; count < 100000; ++count)
        if (!splits(count) || !splits(INT32_MAX - count + 1)) return 1;
    for (int i = 0; i < 1000000; ++i)
        if (!splits(1 + (int64_t)(rng() % INT32_MAX)) || !splits(log_uniform(2147483648.0))) return 1;
    std::printf("ok %d\n", 2 * n);
    return 0;
}
