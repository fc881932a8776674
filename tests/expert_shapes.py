"""Sizes that take each of the grouped products' tile shapes, with groups that
end inside the tiles at every height a last tile can have.  The choice is
pinned on the CPU (test_expert_host.py), the results are checked on the GPU
(test_gpu_expert.py), so that a change of the rule cannot leave a shape untested.

Each entry: operation, rows of the experts, R, C, and the shape (rows, columns,
summed axis of a stage, stages) at 256 CUs, with and without AROUND more rows
that belong to no expert."""

AROUND = 3

FORWARD = [
    # the last launch round in halves: those of 64, 130 and 200 rows here, none there
    ("forward", [4928, 2944, 64, 130, 200], 8008, 72, (256, 256, 64, 2)),
    ("forward", [7000, 1000, 64, 130, 200], 8200, 136, (256, 256, 64, 2)),
    ("forward", [5000, 61, 131, 3000], 2056, 136, (128, 192, 64, 2)),
    ("forward", [64, 70, 0, 129] * 12, 1416, 72, (128, 192, 64, 2)),          # 48 to 96 rows on average
    ("forward", [90, 200, 1, 129] * 16, 1544, 72, (128, 128, 64, 2)),         # 96 to 192
    ("forward", [120, 130, 100, 129] * 16, 1288, 136, (128, 128, 64, 2)),
    ("forward", [50, 48, 0, 129] * 12, 2056, 72, (128, 128, 64, 2)),          # by the rounds of workgroups
    ("forward", [2000, 129, 65], 1032, 72, (64, 128, 64, 2)),
    ("forward", [64, 130, 20] * 3, 1032, 264, (64, 128, 64, 3)),
    ("forward", [2, 0, 1, 66], 328, 2104, (64, 64, 64, 5)),
    ("forward", [2, 0, 1, 70], 520, 328, (64, 64, 64, 4)),
]
DX = [
    # every tile in halves; the last 32 of 288, of groups of 64 to 250 rows; none
    ("dx", [64, 128, 192, 256, 2000, 1], 4160, 2096, (256, 256, 32, 4)),
    ("dx", [3968, 2880, 256, 64, 128, 192, 250], 4104, 2056, (256, 256, 32, 4)),
    ("dx", [64, 130, 200, 256, 2500, 257], 4160, 2056, (256, 256, 32, 4)),
    ("dx", [5000, 61, 131, 3000], 136, 2056, (128, 192, 64, 2)),
    ("dx", [1, 0, 2, 0, 1] * 12, 72, 1160, (128, 192, 64, 2)),
    ("dx", [200, 130] * 8, 200, 2056, (128, 192, 64, 2)),
    ("dx", [200, 330] * 16, 200, 1160, (128, 128, 64, 2)),
    ("dx", [2000, 129, 65], 72, 1032, (64, 128, 64, 2)),
    ("dx", [64, 130, 20] * 3, 264, 1032, (64, 128, 64, 3)),
    ("dx", [2, 0, 1, 70], 328, 520, (64, 64, 64, 4)),
]
# the weight gradient's rows whole cache lines in fp32 and bf16, in fp32 alone, in neither
DW = [
    ("dw", [300, 0, 65, 1], 1096, 2112, (128, 256, 32, 3)), ("dw", [300, 0, 65, 1], 1096, 2080, (128, 256, 32, 3)),
    ("dw", [300, 0, 65, 1], 1096, 2056, (128, 256, 32, 3)), ("dw", [0, 129, 40], 1352, 2144, (128, 256, 32, 3)),
    ("dw", [33, 31, 97, 0], 1096, 1088, (128, 128, 64, 2)), ("dw", [33, 31, 97, 0], 1096, 1056, (128, 128, 64, 2)),
    ("dw", [33, 31, 97, 0], 1096, 1032, (128, 128, 64, 2)),
    ("dw", [70, 0, 129], 328, 320, (64, 64, 64, 4)), ("dw", [70, 0, 129], 328, 288, (64, 64, 64, 4)),
    ("dw", [70, 0, 129], 328, 264, (64, 64, 64, 4)),
]
CASES = FORWARD + DX + DW
SHAPES = {
    "forward": {(256, 256, 64, 2), (128, 192, 64, 2), (128, 128, 64, 2), (64, 128, 64, 2), (64, 128, 64, 3),
                (64, 64, 64, 5), (64, 64, 64, 4)},
    "dx": {(256, 256, 32, 4), (128, 192, 64, 2), (128, 128, 64, 2), (64, 128, 64, 2), (64, 128, 64, 3), (64, 64, 64, 4)},
    "dw": {(128, 256, 32, 3), (128, 128, 64, 2), (64, 64, 64, 4)},
}


def halved(op, counts, R, C, shape, cus=256):
    """Whether the last round of the 256 x 256 tiles is cut in halves, by the rule in the kernel's comment."""
    last = sum(-(-n // shape[0]) for n in counts) * -(-(R if op == "forward" else C) // shape[1]) % cus
    return 0 < 2 * last <= cus
