"""Cases of products with adapters that reach every way through the kernels (test_grouped_ways.py checks that they do).

(rows of each request, each one's adapter, N, K, rank)
"""
from tests.test_gpu_grouped import ADAPTERS

# ranks that are no multiple of 16, of 32 or of 64
PADDED = [
    ([1], [1], 4104, 4096, 8),
    ([9], [2], 520, 1032, 24),
    ([5], [2], 1032, 520, 40),
    ([1, 2, 1], [0, 1, 2], 256, 264, 8),
    ([4352], [1], 4104, 2056, 40),
    ([2100, 900, 1500], [1, 0, 3], 4104, 1032, 56),
    ([2100, 900, 1500], [1, 0, 3], 4104, 1032, 8),
    ([2100, 900, 1500], [1, 0, 3], 4104, 1032, 32),
]

MORE = [
    ([3, 22], [0, 1], 8, 15600, 40),                                          # projections in parts, tiles of 64 x 64 in parts
    ([1392, 80, 46], [2, -1, 3], 392, 7560, 56),                              # projections in parts before large tiles
    ([26, 1391, 59], [1, 0, 3], 1352, 72, 16),                                # large tiles, whole
    ([14, 2], [3, 1], 24, 16848, 120),                                        # 16 x 16 in parts, then dot products
    ([144, 1, 230, 12, 37], [0, 1, 2, -1, 3], 2360, 1168, 48),                # sums in one part for the tiles behind them
    ([38, 5, 3, 373, 33], [1, 2, 3, 0, -1], 4248, 2504, 8),                   # tiles of 128 x 128 in parts
    ([1, 1, 333, 1, 64, 1, 900, 17, 1, 1, 128, 1, 1, 250, 33], [b % 5 - 1 for b in range(15)], 2056, 1000, 24),   # and whole
    ([3, 3, 2, 18, 15, 2, 6, 22] * 18, [b % 5 - 1 for b in range(144)], 16, 16, 96),   # projections of 64 x 128
    ([5, 8, 40, 1] * 31, [b % 5 - 1 for b in range(124)], 24, 168, 112),      # tiles of 16 x 16
    ([174, 1, 6, 382, 2, 29, 98, 285], [0, 1, -1, 2, 3, 0, 1, 2], 88, 8608, 128),   # tiles of 64 x 128 in parts
    ([1, 22, 12, 10, 4, 8, 77], [3, 2, 1, 0, 3, -1, 1], 6208, 8, 24),         # and whole
]

EVERY_WAY = ADAPTERS + PADDED + MORE
