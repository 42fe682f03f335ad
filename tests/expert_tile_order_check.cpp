// Checks the order in which workgroups go through tiles (expert_plan.h, xcd.h) on
// the host: every tile is taken once, and a workgroup's tile numbers grow.
#include <cstdio>
#include <vector>

#include "expert_plan.h"

using namespace moedx;

static bool check(const TileShape& t, int total) {
    const int step = (int)workgroups_through(t, total);
    std::vector<char> seen(total, 0);
    for (int b = 0; b < step; ++b) {
        int last = -1;
        for (int v = b; v < total; v += step) {
            const int tile = xcd_run_block<kRunLog2>(v, total);
            if (tile <= last || tile >= total || seen[tile]++) {
                std::printf("FAIL %d tiles, workgroup %d: tile %d after %d\n", total, b, tile, last);
                return false;
            }
            last = tile;
        }
    }
    for (int i = 0; i < total; ++i)
        if (!seen[i]) {
            std::printf("FAIL %d tiles: %d is left out\n", total, i);
            return false;
        }
    return true;
}

int main() {
    std::vector<int> totals;
    for (int n = 1; n <= 3100; ++n) totals.push_back(n);
    for (int n : {4095, 4096, 4097, 65535, 65536, 100003, (1 << 23) - 1, (1 << 24) - 1})
        totals.push_back(n);
    for (const int n : totals)
        if (!check(kWideTile, n) || !check(kSmallTile, n)) return 1;
    std::printf("ok %d\n", (int)totals.size());
    return 0;
}
