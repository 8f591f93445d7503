"""Sizes that reach each kernel of the FP8 products, with its name (debug_fp8_kernel), so that a test can see that a
changed rule of choice leaves none untested. Pure data; no device."""

# (kernel, rows of every expert (a number: one matrix without offsets), columns K, rows of the matrix N (SwiGLU: inter),
# rows before the first expert's, rows behind the last's). Counts hold empty experts, full tiles and tiles that end after
# every kind of fragment; K ends inside a block, after one and after several; N ends inside a tile.
CASES = [
    ("few_rows_4", [1, 0, 2, 1], 16, 5, 0, 1), ("few_rows_4", [1, 0, 2, 1], 144, 100, 0, 0), ("few_rows_4", [3], 512, 48, 2, 0),
    ("few_rows_4", [0, 1, 15, 16, 17, 0], 1024, 272, 0, 3), ("few_rows_4", 1, 2048, 33, 0, 0), ("few_rows_4", 5, 4624, 131, 0, 0),
    ("few_rows_4", [2, 1, 0, 4, 1, 8], 6144, 129, 1, 1), ("few_rows_4", [0, 0, 0], 128, 16, 2, 2),
]
