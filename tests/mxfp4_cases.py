"""Sizes that reach each kernel of the MXFP4 products, with its name (debug_mxfp4_kernel), so that a test can
see that a changed rule of choice leaves none untested. Pure data and the question; no device."""

# (kernel, rows of every expert (a number: one matrix without offsets), columns K, scales on 16-byte boundaries, rows
# behind the last); N and inter are chosen per kernel below. Counts hold empty experts, full tiles and tiles that end
# after every kind of fragment; K ends in every kind of partial chunk.
_TILES64 = [5, 0, 31, 64, 65, 1, 16, 33, 17, 32] * 8
_TILES128 = [33, 129, 0, 64, 65, 128, 70, 200] * 5
_SHORT = [9, 0, 130, 1, 64, 65, 128] * 10
CASES = [
    ("few_rows_2", [1, 0, 2, 1], 96, False, 1), ("few_rows_2", [1, 0, 2, 1], 1536, True, 1), ("few_rows_2", 40, 1120, False, 0),
    ("few_rows_4", [1, 0, 2, 1], 4128, False, 1), ("few_rows_4", [1, 0, 2, 1], 4608, True, 1),
    ("tiles_short", _SHORT, 32, False, 0), ("tiles_short", _SHORT, 96, True, 3), ("tiles_short", _SHORT, 224, False, 0),
    ("tiles_short", _SHORT, 256, True, 1), ("tiles_short", _SHORT, 288, False, 0), ("tiles_short", _SHORT, 480, False, 5),
    ("tiles_short", 2100, 160, False, 0), ("tiles_short", 2100, 352, True, 0),
    ("tiles_64", _TILES64, 512, True, 0), ("tiles_64", _TILES64, 544, False, 2), ("tiles_64", _TILES64, 1024, False, 0),
    ("tiles_64", _TILES64, 1120, True, 0), ("tiles_64", _TILES64, 1504, False, 1), ("tiles_64", _TILES64, 2880, False, 0),
    ("tiles_128", _TILES128, 512, False, 0), ("tiles_128", _TILES128, 544, True, 4), ("tiles_128", _TILES128, 736, False, 0),
    ("tiles_128", _TILES128, 1024, False, 1), ("tiles_128", _TILES128, 1120, False, 0), ("tiles_128", 2100, 608, True, 0),
    ("lines_128", _TILES64, 1024, True, 2), ("lines_128", _TILES128, 1536, True, 0), ("lines_128", [3, 4] * 40, 1024, True, 1),
    ("lines_256", [2600, 0, 1300], 1024, True, 3), ("lines_256", 2700, 1536, True, 0),
]


def matrix_rows(kernel, counts, swiglu):
    """N of the product (odd, so that rows of the output end anywhere), or inter: enough tiles of 256 rows for the
    kernel, the last one partial."""
    if kernel.startswith("few"):
        return 96 if swiglu else 131
    if kernel == "lines_256" or isinstance(counts, int):
        wide = {"lines_256": 3712 if not isinstance(counts, int) else 6304}.get(kernel, 2112)
        return wide // 2 // 32 * 32 if swiglu else wide - 11
    return 480 if swiglu else 903


def rows_of(counts, spare):
    """(rows, matrices, grouped)."""
    return (counts, 1, False) if isinstance(counts, int) else (sum(counts) + spare, len(counts), True)


def chosen(coli, counts, spare, K, N, aligned):
    rows, E, grouped = rows_of(counts, spare)
    return coli.debug_mxfp4_kernel(rows, K, E, N, grouped, aligned)


# a layer of random experts: (tokens, experts, slots, hidden, inter, kernel of the gate/up and of the down product)
LAYERS = [(5, 16, 4, 4128, 544, "few_rows_4", "few_rows_2"), (200, 64, 4, 2400, 480, "tiles_64", "tiles_short"),
          (200, 32, 4, 2080, 1056, "tiles_64", "tiles_64"), (400, 32, 4, 2080, 1056, "tiles_128", "tiles_128"),
          (300, 32, 4, 2048, 1024, "lines_128", "lines_128"), (4100, 2, 1, 4096, 2048, "lines_256", "lines_256")]
