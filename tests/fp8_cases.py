"""Sizes that reach each kernel of the FP8 products, with its name (debug_fp8_kernel), so that a test can see that a
changed rule of choice leaves none untested. Pure data; no device."""

# (kernel, rows of every expert (a number: one matrix without offsets), columns K, rows of the matrix N (SwiGLU: inter),
# rows before the first expert's, rows behind the last's). Counts hold empty experts, full tiles and tiles that end after
# every kind of fragment; K ends inside a block, after one and after several; N ends inside a tile.
_MIXED = [5, 0, 31, 64, 65, 1, 16, 33, 17, 32, 128, 130, 0, 257]
CASES = [
    ("few_rows_4", [1, 0, 2, 1], 16, 5, 0, 1), ("few_rows_4", [1, 0, 2, 1], 144, 100, 0, 0), ("few_rows_4", [3], 512, 48, 1, 0),
    ("few_rows_4", [0, 1, 15, 16, 17, 0] + [0] * 10, 1024, 272, 0, 3), ("few_rows_4", 1, 2048, 33, 0, 0), ("few_rows_4", 5, 4624, 131, 0, 0),
    ("few_rows_4", [2, 1, 0, 4, 1, 8], 6144, 129, 1, 1), ("", [0, 0, 0], 128, 16, 2, 2),
    ("lines_128", _MIXED, 16, 33, 0, 0), ("lines_128", _MIXED, 128, 256, 3, 3), ("lines_128", _MIXED, 144, 300, 0, 1),
    ("lines_128", _MIXED, 256, 128, 0, 0), ("lines_128", _MIXED, 384, 129, 2, 0), ("lines_128", _MIXED, 512, 520, 0, 2),
    ("lines_128", _MIXED, 1040, 257, 1, 0), ("lines_128", 100, 640, 70, 0, 0), ("lines_128", 300, 2048, 1500, 0, 0),
    ("lines_128", [40] * 70, 896, 384, 0, 0), ("lines_128", [9] * 300, 272, 48, 5, 5),
    ("lines_256", 1300, 16, 300, 0, 0), ("lines_256", [900, 0, 1000, 613, 257], 128, 256, 1, 2), ("lines_256", 1025, 272, 513, 0, 0),
    ("lines_256", [512, 700], 512, 129, 0, 0), ("lines_256", 700, 1152, 640, 0, 0), ("lines_256", [1000, 300, 2000], 656, 200, 2, 1),
]
