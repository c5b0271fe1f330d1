"""Sizes of the FP8 product that take each tile kernel, and how each runs: (tile
rows / 64, tile columns / 64, parts of the contraction, blocks of 128 per part).

Sizes are cut on both axes; where the variant allows it a part has more than 16
blocks (a second chunk of staged scales) and the last part another, odd count.
The host test pins each plan, so that a change of the planner's times cannot take
these sizes, and with them the GPU tests, to another kernel unnoticed."""

TILES = [
    # m, n, k, result, plan
    (1300, 1500, 2310, "bf16", (1, 1, 1, 19)),
    (1300, 1500, 2310, "f32", (1, 1, 1, 19)),
    (2001, 1999, 2310, "bf16", (2, 2, 1, 19)),
    (2001, 1999, 2310, "f32", (2, 2, 1, 19)),
    (2047, 6143, 2310, "bf16", (4, 3, 1, 19)),
    (2047, 6143, 2310, "f32", (4, 3, 1, 19)),
    (6143, 2047, 2310, "bf16", (3, 4, 1, 19)),
    (6143, 2047, 2310, "f32", (3, 4, 1, 19)),
    (4000, 4004, 2310, "bf16", (4, 4, 1, 19)),
    (4000, 4004, 2310, "f32", (4, 4, 1, 19)),
    (401, 700, 9000, "bf16", (1, 1, 6, 12)),
    (300, 3000, 16300, "f32", (1, 1, 2, 64)),
    (65, 6143, 9000, "bf16", (2, 2, 9, 8)),
    (1000, 1001, 16300, "f32", (2, 2, 4, 32)),
    (3000, 777, 16300, "bf16", (4, 3, 4, 32)),
    (777, 3000, 16300, "f32", (4, 3, 4, 32)),
    (777, 3000, 16300, "bf16", (3, 4, 4, 32)),
    (6144, 200, 16300, "f32", (3, 4, 8, 16)),
    (201, 8191, 29900, "bf16", (4, 4, 8, 32)),
    (1200, 1201, 65000, "f32", (4, 4, 8, 64)),
]

# Sizes of other tests that are meant for one kind of kernel: narrow kernels
# (0, 0), with the operands straight in registers or through LDS, or tiles.
OTHERS = [
    # m, n, k, result, (tile rows / 64, tile columns / 64, split, straight to registers)
    (300, 300, 384, "bf16", (0, 0, False, True)),
    (300, 300, 384, "f32", (0, 0, False, True)),
    (300, 301, 5000, "bf16", (0, 0, False, False)),
    (60, 2000, 9000, "f32", (0, 0, False, False)),
    (600, 600, 640, "bf16", (1, 1, False, False)),
    (600, 600, 640, "f32", (1, 1, False, False)),
    (700, 1025, 257, "bf16", (1, 1, False, False)),
    (1030, 520, 300, "f32", (1, 1, False, False)),
    (8190, 8001, 640, "bf16", (2, 2, False, False)),
    (401, 700, 9000, "f32", (1, 1, True, False)),
    (1501, 1300, 16200, "f32", (1, 1, False, False)),
]
