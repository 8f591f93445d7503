"""Sizes that reach each kernel of the FP8 products, with its name (debug_fp8_kernel) for 16-bit and for 32-bit
results, so that a test can see that a changed rule of choice leaves none untested. Pure data; no device."""

_MIXED = [5, 0, 31, 64, 65, 1, 16, 33, 17, 32, 128, 130, 0, 257]
_MANY = [200, 0, 129, 300, 64, 513, 256, 1, 128, 400, 255, 130]
_FULL = [900, 0, 1300, 613, 257, 1024, 512, 1]

# (kernel, that of 32-bit results, rows of every expert (a number: one matrix without offsets), columns K, rows of the
# matrix N (SwiGLU: inter), rows before the first expert's, rows behind the last's). Counts hold empty experts, full tiles
# and tiles that end after every kind of fragment; K ends inside a block, after one and after several; N ends inside a tile.
CASES = [
    ("few_rows_16", "few_rows_16", [1, 0, 2, 1], 16, 5, 0, 1), ("few_rows_16", "few_rows_16", [1, 0, 2, 1], 144, 100, 0, 0),
    ("few_rows_16", "few_rows_16", [3], 512, 48, 1, 0), ("few_rows_16", "few_rows_16", [0, 1, 15, 16, 17, 0], 1024, 272, 0, 3),
    ("few_rows_16", "few_rows_16", 1, 2048, 33, 0, 0), ("few_rows_16", "few_rows_16", 37, 4624, 131, 0, 0),
    ("few_rows_32", "few_rows_32", [2, 1, 0, 4, 1, 8], 6144, 929, 1, 1), ("few_rows_32", "few_rows_32", 9, 272, 4100, 0, 0),
    ("few_rows_32", "few_rows_32", _MIXED, 512, 520, 0, 2), ("few_rows_32", "few_rows_32", 100, 1040, 1500, 0, 0),
    ("few_rows_32", "few_rows_32", [9] * 300, 272, 48, 5, 5),
    ("few_rows_16", "few_rows_16", [0, 0, 0], 128, 16, 2, 2),
    ("lines_128", "lines_128", _MANY * 4, 16, 161, 0, 0), ("lines_128", "lines_128", _MANY * 4, 128, 256, 3, 3),
    ("lines_128", "lines_128", _MANY * 4, 144, 300, 0, 1), ("lines_128", "lines_128", _MANY * 5, 256, 128, 0, 0),
    ("lines_128", "lines_128", _MANY * 4, 384, 129, 2, 0), ("lines_128", "lines_128", _MANY * 2, 512, 520, 0, 2),
    ("lines_128", "lines_128", _MANY, 1040, 1025, 1, 0), ("lines_128", "few_rows_32", 700, 640, 1500, 0, 0),
    ("lines_128", "few_rows_32", [16, 17, 40, 0, 3] * 30, 896, 768, 0, 0), ("lines_128", "few_rows_32", [20] * 260, 272, 512, 5, 5),
    ("lines_256", "lines_128", 9000, 16, 1300, 0, 0), ("lines_256", "lines_128", _FULL * 3, 128, 2056, 1, 2),
    ("lines_256", "lines_128", 8200, 272, 1313, 0, 0), ("lines_256", "lines_128", [2300, 0, 3700], 512, 2049, 0, 0),
    ("lines_256", "lines_128", 4500, 1152, 2060, 0, 0), ("lines_256", "lines_128", [2000, 3001, 1000], 656, 2040, 2, 1),
    # several groups of scales (four blocks each) a unit
    ("lines_128", "lines_128", _MANY, 1024, 640, 1, 0), ("lines_128", "lines_128", _MANY * 2, 1536, 300, 0, 2),
    ("lines_128", "few_rows_32", [70] * 40, 2560, 264, 0, 0), ("lines_128", "lines_128", 1500, 2048, 1100, 0, 0),
    ("lines_128", "lines_128", _FULL * 2, 1024, 2056, 1, 1), ("lines_256", "lines_128", 9000, 1536, 1300, 0, 0),
    ("lines_256", "lines_128", [2300, 0, 3700], 2048, 2049, 0, 0), ("lines_256", "lines_128", [256] * 40, 2560, 520, 0, 0),
]

# SwiGLU into FP8 rows, by how the sums are formed: (form, rows of every expert, K, inter, rows before and behind). "exact":
# fewer than 2^20 values, whose tiles take exact products; "parts": columns in parts, with a workspace, whose sums the FP8
# rows are formed from. K ends inside a block and after one, with one group of scales, several, and a short last one.
FP8_ROWS = [
    ("exact tiles", _MANY * 4, 16, 48, 0, 0), ("exact tiles", _FULL, 128, 160, 1, 0), ("exact tiles", _MANY * 2, 144, 144, 0, 0),
    ("exact tiles", 9000, 384, 112, 0, 0), ("exact tiles", _MANY, 512, 400, 0, 1), ("exact tiles", _MANY * 4, 1040, 80, 2, 3),
    ("exact tiles", _MANY * 2, 1536, 144, 0, 0), ("exact tiles", [70] * 40, 2576, 272, 0, 0),
    ("exact parts", 150, 5136, 2064, 0, 0), ("exact parts", [130, 0, 123, 1], 8192, 2064, 3, 4),
    ("parts", 256, 5136, 4096, 0, 0), ("parts", 256, 8208, 4112, 0, 0), ("parts", 300, 8192, 4112, 0, 0),
    ("parts", [300, 0, 250], 8192, 2048, 1, 2),
]
