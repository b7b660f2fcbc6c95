"""Sizes of the grouped linear layer's products for every kind of tile and row layout.  That they
take these is asserted on the CPU (test_grouped_tiles.py), what they compute on the GPU
(test_gpu_grouped_kernels.py)."""

# product, tile, whether the weights' gradient is in chunks of rows, rows, groups, K, M.  "dw" and
# "dx" are gradients asked for alone, "both" is one launch for the two.
HALF = [
    ("forward", 32, False, 70, 3, 264, 136), ("forward", 64, False, 300, 3, 264, 136),
    ("forward", 128, False, 1500, 41, 264, 1544), ("forward", 256, False, 9001, 12, 264, 4104),
    ("dx", 32, False, 70, 3, 136, 264), ("dx", 64, False, 300, 3, 136, 264),
    ("dx", 128, False, 1500, 41, 1544, 264), ("dx", 256, False, 9001, 12, 4104, 264),
    ("dw", 64, True, 300, 3, 136, 136), ("dw", 128, True, 9000, 3, 264, 520),
    ("dw", 128, False, 700, 7, 264, 3080), ("dw", 256, False, 5000, 41, 328, 3080),
    ("both", 64, True, 300, 3, 136, 264), ("both", 128, True, 9000, 3, 264, 520),
    ("both", 128, False, 700, 7, 3080, 264), ("both", 256, False, 5000, 41, 3080, 328),
]
FULL = [
    ("forward", 32, False, 70, 3, 264, 136), ("forward", 64, False, 300, 3, 264, 136),
    ("forward", 128, False, 7000, 41, 264, 328),
    ("dx", 32, False, 70, 3, 136, 264), ("dx", 64, False, 300, 3, 136, 264),
    ("dx", 128, False, 7000, 41, 328, 264),
    ("dw", 64, True, 300, 3, 136, 136), ("dw", 128, True, 9000, 3, 264, 520),
    ("dw", 128, False, 700, 7, 264, 3080),
    ("both", 64, True, 300, 3, 136, 264), ("both", 128, True, 9000, 3, 264, 520),
    ("both", 128, False, 700, 7, 3080, 264),
]
# What is added to K and M: rows of whole 16-byte chunks, of words, and of 2-byte values at any place
CHUNKS, WORDS, ODD = 2, 1, 0
SHIFTS = {"half": {CHUNKS: (0, 0), WORDS: (2, -2), ODD: (1, -1)}, "full": {CHUNKS: (0, 0), WORDS: (1, -1)}}


def cases():
    """(product, tile, chunked, layout, rows, groups, K, M, type)"""
    for dtype in ("bf16", "fp16", "fp32"):
        size = "full" if dtype == "fp32" else "half"
        for product, tile, chunked, rows, groups, K, M in FULL if dtype == "fp32" else HALF:
            for layout, (dk, dm) in SHIFTS[size].items():
                yield product, tile, chunked, layout, rows, groups, K + dk, M + dm, dtype


def name(c):
    return "-".join([c[0], str(c[1]), "chunked" if c[2] else "whole", ("odd", "words", "chunks")[c[3]], c[8]])
