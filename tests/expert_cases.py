"""Cases of test_gpu_expert_forms.py, each meant for one kernel form;
test_expert_forms.py holds them to it on the CPU."""

# form: (M, N, K). K with short last blocks, even and odd block counts (the
# forms that take two blocks a step), N a multiple of eight and not.
F8 = {
    "rows1": [(5, 100, 160), (200, 130, 416)],
    "rows2": [(40, 1500, 288), (300, 301, 160)],
    "rows3": [(40, 4096, 160), (70, 1501, 416), (48, 4096, 1184)],
    "rows4": [(64, 4096, 288), (100, 1502, 1056)],
    "quarter": [(1, 8200, 288), (140, 3900, 416), (130, 2002, 160), (64, 14336, 1184)],
    "half": [(70, 14400, 288), (100, 14402, 416), (66, 8200, 1120)],
    "small": [(520, 4096, 160), (221, 8201, 288), (700, 4100, 1312)],
    "wide": [(1000, 4104, 416), (300, 14401, 160)],
    "large": [(3900, 4096, 288), (975, 8201, 416)],
}

# form: (counts of the groups, N, K, share, extra rows in no group).
F8_GROUPED = {
    "rows1": [([5, 0, 9, 1], 100, 160, 1, 2)],
    "rows2": [([30, 0, 3, 17], 300, 288, 2, 1)],
    "rows4": [([70, 1, 0, 40], 300, 416, 3, 0), ([0, 90, 3, 1], 515, 160, 1, 3)],
    "quarter": [([100, 0, 29, 1], 3900, 416, 2, 3), ([40, 33, 0, 64], 500, 288, 1, 0)],
    "half": [([64, 1, 0, 96], 4100, 288, 3, 0), ([0, 200, 65, 35], 8200, 160, 1, 4)],
    "small": [([300, 0, 129, 271], 4100, 288, 2, 5), ([222, 0], 8200, 416, 1, 0)],
    "wide": [([130, 0, 1, 389], 8200, 160, 2, 1), ([1, 1, 0, 2], 14400, 288, 1, 0)],
    "large": [([257, 0, 1, 720], 8201, 288, 2, 2)],
}

# Grouped products over Q4_0 and Q8_0 in the GEMM's tiles: several column tiles,
# last tiles of 1 to 32, 33 to 64 and more rows, empty groups, an order, a
# share, rows in no group; K of one pair of blocks and of two (shorter than the
# rings), of a whole number of rings and of 2 pairs more (K = 128 mod 256).
TILES = [
    ([300, 0, 220], 3300, 384, 1, 2),
    ([129, 1, 0, 400, 30], 3400, 1152, 2, 0),
    ([600, 40], 3300, 64, 1, 0),
    ([160, 480], 3300, 128, 4, 0),
    ([148, 306, 185], 3300, 320, 3, 1),
    ([40, 60, 500], 3300, 640, 1, 0),
    ([0, 0, 128, 0, 512, 0], 3300, 512, 2, 0),
]

# (activation rows T, experts, top_k, N, K) of the streams and captured tests.
TILE_LAYERS = [(300, 6, 2, 3300, 384), (330, 4, 2, 3300, 640)]

# fmt: form: (counts, N, K, share, extra).
FEW = {
    "q4": {
        "few1x1": [([20, 0, 17], 300, 320, 2, 1)],
        "few4x1": [([16, 0, 20, 3], 16400, 128, 1, 0)],
        "few4x2": [([64, 3, 40, 0], 16400, 192, 2, 2)],
    },
    "q8": {
        "few1x1": [([20, 0, 17], 300, 320, 2, 1)],
        "few2x1": [([16, 0, 20, 3], 8200, 128, 1, 0)],
        "few2x2": [([64, 3, 40, 0], 8200, 192, 2, 2)],
    },
}
