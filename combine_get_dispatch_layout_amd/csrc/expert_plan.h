// Which tiles an experts' product takes, from what the host knows (no device
// code and no HIP: the rules are checked on a machine without a GPU).
#pragma once

#include <stdint.h>

#include "xcd.h"

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
// Of an int8 product of few rows and very few workgroups.
constexpr TileShape kNarrowTile{32, 64, 256};
// Of a weight gradient: weight rows (N) and columns (K).
constexpr TileShape kWeightTile{128, 256, 256};
// The same from rows saved in int8.
constexpr TileShape kSavedTile{256, 128, 256};

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
inline int64_t weight_workgroups(const ExpertRows& er, int K, int N,
                                 const TileShape& t = kWeightTile) {
    return er.E * tiles_of(N, t.rows) * tiles_of(K, t.outs);
}

constexpr int kRunLog2 = 5;  // an XCD takes runs of 32 tiles: one per CU, sharing operands in its L2

// Workgroups of a kernel that goes through `total` tiles: one of 512 threads to a
// compute unit, two of 256.  Workgroup b takes the tiles xcd_run_block(v) for v =
// b, b + workgroups, ...  Their numbers have to grow: it searches the experts' rows
// forwards only and ends at the first tile that is not there.  They do among the
// numbers of one XCD, b % 8, which a multiple of 8 keeps.
constexpr int64_t kUnits = 256;
static_assert(kUnits % kXcds == 0, "a workgroup's tiles are those of one XCD");
inline int64_t workgroups_through(const TileShape& t, int64_t total) {
    const int64_t most = kUnits * (t.threads == 512 ? 1 : 2);
    return total < most ? total : most;
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

// The int8 product's tiles.  kNarrow: 32 x 64; kOnce: 128 x 128 with the weights
// past the caches; kDeep, kDeepOnce: 128 x 128 with three stages of the weights,
// through the caches and past them; kWide: 256 x 256.  64 experts with the same
// number of rows each, us, the weights from memory (other ones in between):
//   rows each                    1    8   16   32   64   96  128
//   7168 -> 4096   kNarrow     267  276  287  322
//                  kOnce       270  276  277  280  299  324  357
//                  kDeepOnce   269  274  275  276  293  336  358
//                  kWide       307  310  313  313  321  330  340
//   4096 -> 4096   kNarrow     163  164  170  186
//                  kOnce       166  162  163  164  169  184  249
//                  kDeepOnce   163  163  163  165  170  190  233
//                  kWide       182  180  181  183  189  196  260
//   2048 -> 1408   kNarrow      36   35   36   39
//                  kOnce        40   38   37   37   39   42   46
//                  kDeepOnce    35   33   33   33   36   39   44
//                  kWide        47   44   44   44   46   49   51
// and with rows that vary, as uniform and as skewed routing of top-8 gives them
// (on average 8, 12, 16, 32, 64, 80, 96 and 128):
//   4096 -> 4096
//   kOnce       163 157  163 162  164 164  166 195  172 222  181 264  189 279  334 311
//   kDeepOnce   163 159  164 164  165 166  166 188  174 229  185 262  196 278  336 307
//   kWide       180 176  181 182  183 185  184 193  191 234  195 248  198 250  260 266
//   7168 -> 4096
//   kOnce                                           302 367  318 437  331 436  552 525
//   kDeepOnce                                       302 377  325 430  342 438  554 533
//   kWide                                           322 380  326 384  331 395  348 413
//   4096 -> 2048
//   kOnce                                            90 119   94 133   99 148  167 170
//   kDeepOnce                                        89 114   94 136   98 148  167 156
//   kWide                                           101 135  102 139  106 143  138 147
//   2048 -> 1408
//   kOnce                                            43  43   42  45   43  46   64  61
//   kDeepOnce                                        39  43   39  46   41  47   62  57
//   kWide                                            50  48   49  48   49  48   52  55
//   256 experts, 7168 -> 4096
//   kOnce                                         1265 1601         1387 1923 2287 2247
//   kDeepOnce                                     1287 1609         1437 1938 2293 2288
//   kWide                                         1281 1439         1308 1602 1399 1753
//   256 experts, 2048 -> 1408
//   kOnce                                          140  168          147  198  226  229
//   kDeepOnce                                      138  167          148  196  231  225
//   kWide                                          150  169          156  193  168  199
// At 128 the experts past 128 rows take a second 128-row tile, and kWide wins
// whatever the reduction (with just 128 rows in each, which no routing gives,
// kDeepOnce: 44 and 51, 233 and 260).  Between 80 and 128 neither does: at 96 kWide
// takes 20% more than kDeepOnce for 2048 -> 1408 of uniform numbers, 8% for 4096 ->
// 2048, and up to 17% less for skewed ones.  The rule knows neither the skew nor the
// reduction.
//
// A decode batch's slots (64 x 128, 12 live each, 4096 -> 2 x 2048, gated): 172 by
// kOnce, 177 by kDeepOnce.  Of 256 experts (128 tokens, top-8, 7168 -> 2 x 2048, gated):
// 1060 by kDeepOnce, 1075 by kOnce, 1193 by kWide.
//
// One or a few tokens ask for the weights of as many experts: up to two
// workgroups of 128 x 128 per compute unit, 32 x 64 keep more in flight (rows in
// 1, 8 and 16 experts, 7168 -> 2048: 14 21 38, by kDeepOnce 27 31 38; one expert of 32
// rows, 8192 -> 8192: 23 and 33).  Where 256 x 256 leave compute units without a
// tile (8 experts, 7168 -> 4096, 48, 96, 128, 256 and 512 rows):
//   kOnce           56   58   61   81  148
//   kDeepOnce       39   43   47   82  153
//   kDeep           44   48   52   77  133
//   kWide           60   65   68   95  102 (256 tiles)
// (Weights that the 256 MB memory-side cache holds from the call before, as a
// small model's may be, are better read through the caches: 8 of 48 rows, 4096 ->
// 2048: 19 by kDeep, 20 by kDeepOnce; from memory 22 and 20.)
//
// Slots may be nearly all empty (4096 -> 1024; every expert has 4 rows, and 8 have
// one):
//                              kNarrow      kOnce   kDeepOnce      kWide
//    64 experts, 128 slots     47   11     43  29     43  19     50  32
//   128 experts, 64 slots      86   14     83  29     83  19     94  33
//   256 experts, 128 slots    201   65    162  30    162  20    182  33
//   1024 experts, 128 slots  1234  808    629  33    626  22    701  36
// kNarrow has a workgroup to each tile, and each looks at 64 experts at a time.
//
// The others launch 512 workgroups at most, but are held to the tiles of a grid
// with a workgroup to each all the same: the limit is the 16-bit product's, and
// tile numbers (and what workgroups add to them) stay far below 2^31.
constexpr int64_t kNarrowLikely = 32, kOnceLikely = 80, kDeepOnceLikely = 128;
constexpr int64_t kNarrowLooks = 512, kOnceLikelySlots = 8;

enum class Int8Tiles { kNarrow, kOnce, kDeepOnce, kDeep, kWide, kNone };

inline Int8Tiles int8_tiles(const ExpertRows& er, int outs) {
    const int64_t likely = expected_rows(er);
    const int64_t rows = er.offsets ? er.rows : 8 * (int64_t)er.cap;
    const int64_t active = rows < er.E ? rows : er.E;  // experts with rows, at most
    const int64_t tiles = active * tiles_of(outs, kSmallTile.outs);
    const int64_t looks = er.offsets ? 0 : max_tiles(er, kNarrowTile.rows) * tiles_of(er.E, 64);
    const auto fits = [&](const TileShape& t) { return grid_fits(workgroups(er, t, outs), t.threads); };
    if (likely <= kNarrowLikely && tiles <= 512 && looks <= kNarrowLooks && fits(kNarrowTile))
        return Int8Tiles::kNarrow;
    if (likely <= kOnceLikely && fits(kSmallTile))
        return tiles >= 1024 && (er.offsets || likely >= kOnceLikelySlots) ? Int8Tiles::kOnce
                                                                           : Int8Tiles::kDeepOnce;
    if (few_wide_tiles(er, likely, outs) && fits(kSmallTile))
        return likely <= kDeepOnceLikely ? Int8Tiles::kDeepOnce : Int8Tiles::kDeep;
    return fits(kWideTile) ? Int8Tiles::kWide : Int8Tiles::kNone;
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
