"""Cases of expert_linear_int8 by the kernel that each takes, whose workgroups go
through several tiles.  test_expert_int8_tiles.py asks the library's own rule
which tiles a case takes (no GPU needed); test_gpu_expert_int8_tiles.py runs
them.  A rule that moves a case to another kernel fails the first."""

import random

# kind -> (rows, outputs) of a tile, and the workgroups at most
TILES = {"kOnce": (128, 128, 512), "kDeepOnce": (128, 128, 512), "kDeep": (128, 128, 512),
         "kWide": (256, 256, 256)}


def mixed(E, top, seed):
    """0 to `top` rows in each expert; the first, one in the middle and the last
    have none, one and the most."""
    rng = random.Random(seed)
    counts = [rng.randint(0, top) for _ in range(E)]
    counts[0], counts[E // 2], counts[-1] = 0, 1, top
    return counts


class Case:
    """counts: rows of each expert; cap: of slots (0: expert order); outs: outputs
    per row, gate and up counted both."""

    def __init__(self, kind, counts, cap, K, outs):
        self.kind, self.counts, self.cap, self.K, self.outs = kind, counts, cap, K, outs
        self.E = len(counts)
        # expert order: rows behind the last expert's
        self.rows = self.E * cap if cap else sum(counts) + 5

    def __repr__(self):
        where = f"slots{self.cap}" if self.cap else f"{sum(self.counts)}r"
        return f"{self.kind}-{self.E}e-{where}-{self.K}-{self.outs}"

    def live_tiles(self):
        rows, outs, _ = TILES[self.kind]
        return sum(-(-c // rows) for c in self.counts) * -(-self.outs // outs)


CASES = [Case("kOnce", mixed(64, 65, 1), 0, k, 2064) for k in (16, 272, 400, 4096, 8192)]
CASES += [Case("kOnce", mixed(64, 60, 2), 128, k, 2064) for k in (272, 4096)]
CASES += [Case("kOnce", mixed(256, 65, 3), 0, k, 1040) for k in (400, 4096)]
CASES += [Case("kDeepOnce", mixed(64, 65, 4), 0, k, 1168) for k in (272, 400, 4096)]
CASES += [Case("kDeepOnce", mixed(256, 9, 5), 128, k, 1040) for k in (272, 4096)]
CASES += [Case("kDeep", [1024, 0, 3000, 1, 700, 65, 2400, 1002], 0, k, 1776) for k in (272, 400, 4096)]
CASES += [Case("kWide", mixed(256, 256, 6), 0, k, 1040) for k in (272, 4096)]

# (kind, cap, outs, M rows in the buffer of 8 or 64 experts, rows of each expert in
# turn): what a captured call finds in its offsets or counts.
CHANGING = [
    ("kOnce", 0, 2064, 2560, [mixed(64, 65, 11), mixed(64, 30, 12), [0] * 64, [2560] + [0] * 63,
                              [40] * 64]),
    ("kOnce", 128, 2064, 64 * 128, [mixed(64, 128, 13), [0] * 64, [1] * 64, [128] * 64,
                                    [0] * 63 + [128]]),
    ("kDeepOnce", 0, 1168, 2560, [mixed(64, 65, 14), [0] * 64, [0] * 63 + [2560], [40] * 64]),
    ("kDeep", 0, 1776, 8192, [[1024] * 8, [0, 3000, 1, 700, 65, 0, 4000, 300], [0] * 8,
                              [8192] + [0] * 7]),
    ("kWide", 0, 4112, 8192, [[1024] * 8, [0, 3000, 1, 700, 65, 0, 4000, 300], [0] * 8,
                              [0] * 7 + [8192]]),
]
