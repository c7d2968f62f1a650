"""Sizes that reach every kernel, tile and split of the e4m3 and grouped products, with the plan each takes.

test_fp8_plans.py holds the plans to csrc/fp8_layout.h on the host; the GPU tests
run the sizes. A plan is (streaming kernel, tile, whole tiles, tiles cut along k,
parts of each), tiles by TILES' index.
"""

TILES = ("32x64", "64x128", "128x128", "256x128", "256x256")

# (m, n, k, fast sums, plan)
DENSE = [
    (5, 2069, 1936, False, (1, 0, 0, 0, 1)),
    (17, 100, 1936, False, (1, 0, 0, 0, 1)),
    (17, 2069, 1936, False, (1, 0, 0, 0, 1)),
    (17, 12053, 1392, False, (0, 0, 189, 0, 1)),
    (17, 3438, 4880, False, (0, 0, 0, 54, 4)),
    (33, 16435, 928, False, (0, 1, 129, 0, 1)),
    (33, 2346, 4768, False, (0, 1, 0, 19, 9)),
    (65, 16644, 912, False, (0, 2, 131, 0, 1)),
    (65, 10949, 1936, False, (0, 2, 0, 86, 2)),
    (65, 33025, 912, False, (0, 2, 256, 3, 2)),
    (129, 16694, 912, False, (0, 3, 131, 0, 1)),
    (129, 5394, 4368, False, (0, 3, 0, 43, 5)),
    (129, 32937, 928, False, (0, 3, 256, 2, 2)),
    (515, 14946, 1936, False, (0, 3, 256, 95, 2)),
    (17, 3438, 4880, True, (0, 0, 0, 54, 4)),
    (33, 2346, 4768, True, (0, 1, 0, 19, 9)),
    (65, 16644, 912, True, (0, 2, 131, 0, 1)),
    (65, 10949, 1936, True, (0, 2, 0, 86, 2)),
    (65, 33025, 912, True, (0, 2, 256, 3, 2)),
    (129, 16694, 912, True, (0, 3, 131, 0, 1)),
    (132, 5391, 5680, True, (0, 3, 0, 43, 5)),
    (262, 16433, 3344, True, (0, 3, 256, 2, 6)),
    (257, 16415, 912, True, (0, 4, 130, 0, 1)),
    (129, 16814, 5728, True, (0, 4, 0, 66, 3)),
    (258, 33324, 912, True, (0, 4, 256, 6, 2)),
]

LEAD, SPARE = 3, 5   # rows before the first run and behind the last

# name -> runs of rows: empty, of one row, ending in a tile's first rows, in its first half, at its end, one behind it
RUNS = {
    "few": [5, 0, 40, 0, 0, 1, 2],
    "short": [1, 64, 0, 65, 63, 128, 17, 33, 60, 48] * 4,
    "long": [1, 256, 0, 257, 64, 63, 65, 128, 129, 200] * 4,
    "longer": [2, 512, 0, 300, 63, 64, 385, 128, 129, 360] * 4,
}

# (runs, n, k, tile of e4m3, of e4m3 with fast sums, of bf16)
GROUPED = [
    ("few", 100, 400, 0, 0, 0),
    ("few", 100, 1040, 0, 0, 0),
    ("short", 781, 144, 1, 1, 1),
    ("short", 781, 1040, 1, 1, 1),
    ("longer", 209, 1040, 1, 2, 2),
    ("longer", 209, 400, 1, 2, 2),
    ("long", 649, 144, 3, 4, 4),
    ("long", 649, 528, 3, 4, 4),
    ("long", 649, 1040, 3, 4, 0),
]


def rows_of(runs):
    return LEAD + sum(RUNS[runs]) + SPARE
