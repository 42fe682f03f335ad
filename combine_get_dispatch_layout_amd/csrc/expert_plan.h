// Which tiles an experts' product takes, from what the host knows (no device
// code and no HIP: the rules are checked on a machine without a GPU).
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define MOEDX_PLAN_HD __host__ __device__
#else
#define MOEDX_PLAN_HD
#endif

namespace moedx {

// Which rows belong to an expert: [offsets[e], offsets[e + 1]), or, with
// offsets null, the first counts[e] of the cap rows from e * cap.
struct ExpertRows {
    const int32_t* offsets;
    const int32_t* counts;
    int cap;
    int E;
    int64_t rows;  // rows of the buffers; nothing at or past it is touched
};

// A workgroup's share of an output: so many rows and columns (of a gated
// product's weight rows, gate and up together), by so many threads.
struct TileShape {
    int rows, outs, threads;
};
constexpr TileShape kFewTile{32, 32, 256}, kSmallTile{128, 128, 256}, kWideTile{256, 256, 512};
// Of a weight gradient: weight rows (N) and columns (K).
constexpr TileShape kWeightTile{128, 256, 256};

// An expert's rows (up to 2^31 - 1) are dealt evenly to its ceil(count / BM)
// tiles, in steps of 64 rows (16 for small tiles): two full tiles and one of 20
// rows would take longer than three of 192.  All but the last get row_step, at
// most BM; unsigned, because the sums pass 2^31.
template <int BM>
MOEDX_PLAN_HD inline int row_tiles(int count) {
    return (int)(((uint32_t)count + (BM - 1)) / BM);
}
template <int BM>
MOEDX_PLAN_HD inline int row_step(int count, int tiles) {
    constexpr uint32_t kUnit = BM < 64 ? 16 : 64;  // divides BM, so a step is at most BM
    const uint32_t unit = kUnit * (uint32_t)tiles;
    return (int)(((uint32_t)count + unit - 1) / unit * kUnit);
}

constexpr int64_t tiles_of(int64_t n, int b) { return (n + b - 1) / b; }

// The most tiles of `bm` rows that the buffer's rows can make.
inline int64_t max_tiles(const ExpertRows& er, int bm) {
    if (!er.offsets) return er.E * tiles_of(er.cap, bm);
    const int64_t n = er.rows / bm + er.E;
    return n < er.rows ? n : er.rows;
}

inline int64_t workgroups(const ExpertRows& er, const TileShape& t, int outs) {
    return max_tiles(er, t.rows) * tiles_of(outs, t.outs);
}
inline int64_t weight_workgroups(const ExpertRows& er, int K, int N) {
    return er.E * tiles_of(N, kWeightTile.rows) * tiles_of(K, kWeightTile.outs);
}

// HIP counts a grid's threads in 32 bits.
constexpr bool grid_fits(int64_t workgroups, int threads) {
    return workgroups <= (int64_t)UINT32_MAX / threads;
}

// Rows an expert is likely to have, from what the host knows.  A capacity
// buffer holds at most cap tokens, each with a few experts: 8 are taken, the
// top-k of the wide routings (more only moves where the kernels change).
inline int64_t expected_rows(const ExpertRows& er) {
    if (er.offsets) return er.rows / er.E;
    return er.E > 8 ? (int64_t)er.cap * 8 / er.E : er.cap;
}

// Whether 256 x 256 tiles would leave compute units without one: then 128 x 128
// serve better (8 experts of 256 rows, 4096 -> 2048, 64 wide tiles: 54 and 83
// us; of 512 rows, 4096 -> 4096, 256 wide tiles: 157 and 128).
inline bool few_wide_tiles(const ExpertRows& er, int64_t likely, int outs) {
    return tiles_of(likely, kWideTile.rows) * er.E * tiles_of(outs, kWideTile.outs) < 256;
}

// A few rows, or a few experts' rows: weights straight into registers.  8 of 64
// experts with one row each, 7168 -> 4096: 79 us, 128 x 128 tiles 113.  Rows in
// all 64, few-row kernel and 128 x 128:
//   rows each                1           4           8           9          16
//   7168 -> 4096        594  606    626  636    644  638    648  640    719  642
//   4096 -> 2 x 2048    359  400    361  401    370  403    374  404    409  403
//   2048 -> 1408         64   79     67   79     72   79     74   80     83   80
//   1024 -> 1024         25   23     28   23     29   23
constexpr int64_t kFewLikely = 8;

// But every workgroup, also one past the last tile, looks through the experts'
// rows for its own, so small tiles of a buffer that may hold many rows cost more
// than they save: the few-row kernel stays below so many 32-row tiles, of slots,
// which may be nearly all empty, below so many looks at 64 experts; 128 x 128 of
// slots stays below so many 128-row tiles unless 256-row tiles are as many.
// 4096 -> 2048, us, few-row kernel and 128 x 128:
//   offsets, 256 experts, 256 and 320 tiles   704  741    715  728
//   the same, 1024 -> 1024                    106  104    124  105
//   2048 rows of 2 of 256 experts (7168 -> 2048)          441   79
//   slots: every expert has 1 to 4 rows; one token's 8 experts have one
//   64 experts, 64 tiles (32 slots)           180  183     28   37
//   128 experts, 128 tiles (32)               347  360     36   37
//   128 experts, 256 tiles (64)               353  361     48   37
//   256 experts, 1024 tiles (128)             797  717    176   39
//   1024 experts, 4096 tiles (128)           4350 2814   2174  226
// and 128 x 128 and 256 x 256 (1 to 8 rows; one token):
//   256 experts, 512 tiles (256 slots)        738  745     53   70
//   512 experts, 1024 tiles (256)            1482 1468    130  108
//   1024 experts, 1024 tiles (128)           2814 2911    226  259
//   1024 experts, 4096 tiles (512)           3475 3148    830  465
constexpr int64_t kFewTiles = 256, kFewSlotLooks = 256, kSmallSlotTiles = 512;

inline bool few_serves(const ExpertRows& er) {
    const int64_t tiles = max_tiles(er, kFewTile.rows);
    return er.offsets ? tiles <= kFewTiles : tiles * tiles_of(er.E, 64) <= kFewSlotLooks;
}
inline bool small_serves(const ExpertRows& er) {
    const int64_t tiles = max_tiles(er, kSmallTile.rows);
    return er.offsets || tiles <= kSmallSlotTiles || tiles == max_tiles(er, kWideTile.rows);
}

// Up to so many rows per expert the forward product takes 128 x 128 tiles: the
// weights' bytes count, and two workgroups per CU keep them coming (64 experts,
// 4096 -> 4096, 128 x 128 and 256 x 256: 364 and 375 us at 12 rows, 373 and 383
// at 30; 7168 -> 4096: 635 both at 45, 648 and 643 at 64, 717 and 670 at about
// 100).  The input gradient is better off with 256 x 256 at any number (4096 ->
// 4096: 363 and 330 us at 12 rows, 417 and 378 at 100).
constexpr int64_t kSmallRows = 48;

enum class Tiles { kFew, kSmall, kWide, kNone };

// `best`, or the next larger tiles whose grid can be launched: the rules go by
// the likely rows, the grid covers all that the buffer can hold.
inline Tiles launchable(Tiles best, const ExpertRows& er, int outs) {
    if (best == Tiles::kFew && grid_fits(workgroups(er, kFewTile, outs), kFewTile.threads))
        return Tiles::kFew;
    if (best != Tiles::kWide && grid_fits(workgroups(er, kSmallTile, outs), kSmallTile.threads))
        return Tiles::kSmall;
    if (grid_fits(workgroups(er, kWideTile, outs), kWideTile.threads)) return Tiles::kWide;
    return Tiles::kNone;
}

// `outs`: outputs per row, gate and up counted both.
inline Tiles forward_tiles(const ExpertRows& er, int outs) {
    const int64_t likely = expected_rows(er);
    Tiles best = Tiles::kWide;
    if (likely <= kFewLikely && few_serves(er))
        best = Tiles::kFew;
    else if (few_wide_tiles(er, likely, outs) || (likely <= kSmallRows && small_serves(er)))
        best = Tiles::kSmall;
    return launchable(best, er, outs);
}
inline Tiles input_gradient_tiles(const ExpertRows& er, int outs) {
    return launchable(few_wide_tiles(er, expected_rows(er), outs) ? Tiles::kSmall : Tiles::kWide, er,
                      outs);
}

// Whether workgroups start at scattered places of the reduction (`scattered`).
// 64 experts, 4096 outputs, from the start and scattered:
//   rows each           8          12          30          64         120
//   2048            192  191    248  194    257  199    261  213    285  231
//   4096            374  368    451  380    464  386    466  412    504  445
//   6144            565  560    595  558    632  572    642  591    662  660
//   8192            752  721    752  743    761  758    807  815    878  891
// of about 180 rows (4096), 517 and 517, but of skewed numbers about 180, 317
// and 356.
inline bool rotates(int64_t likely, int reduction) {
    return likely <= 120 && reduction % 2048 == 0;
}

}  // namespace moedx
