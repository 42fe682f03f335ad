// Prints the tiles that expert_plan.h chooses for an int8 product, one line for each
// argument triple after the layout: "offsets" or "counts", experts, rows (or a
// slot's capacity) and outputs per row.
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "expert_plan.h"

using namespace moedx;

int main(int argc, char** argv) {
    static const int32_t any = 0;
    static const char* const names[] = {"kNarrow", "kOnce", "kDeepOnce", "kDeep", "kWide", "kNone"};
    for (int i = 1; i + 3 < argc; i += 4) {
        const int E = std::atoi(argv[i + 1]), outs = std::atoi(argv[i + 3]);
        const int64_t n = std::atoll(argv[i + 2]);
        const ExpertRows er = std::strcmp(argv[i], "offsets") == 0
                                  ? ExpertRows{&any, nullptr, 0, E, n}
                                  : ExpertRows{nullptr, &any, (int)n, E, E * n};
        std::printf("%s\n", names[(int)int8_tiles(er, outs)]);
    }
    return 0;
}
