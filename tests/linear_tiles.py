"""Products that between them use every kernel of the dense products: each tile size, alone,
cut along k and walked persistently (more tiles than run at once), forwards, for dX and for dW. All
have ragged ends in every axis. tests/test_linear_plan.py holds them to the plans named here,
tests/test_gpu_linear_tiles.py to the oracle's values."""

# (product, M, columns N' of P, K): tile, cut along k, walked
TILES = {
    ("fwd", 36, 8, 1453): (64, True, False),
    ("fwd", 792, 4959, 197): (64, False, True),
    ("fwd", 16459, 394, 18): (128, False, True),
    ("fwd", 9001, 130, 2305): (128, True, False),
    ("fwd", 12662, 902, 268): (256, False, False),
    ("fwd", 17785, 1588, 259): (256, False, True),
    ("fwd", 16934, 142, 2214): (256, True, False),
    ("dX", 34, 1418, 17): (64, True, False),
    ("dX", 1156, 200, 3208): (64, False, True),
    ("dX", 17539, 8, 394): (128, False, True),
    ("dX", 5516, 3302, 17): (128, True, False),
    ("dX", 9139, 260, 1305): (256, False, False),
    ("dX", 17090, 262, 1729): (256, False, True),
    ("dX", 16527, 2192, 131): (256, True, False),
    ("dW", 1440, 8, 17): (64, True, False),
    ("dW", 205, 524, 6539): (64, False, True),
    ("dW", 34, 5892, 1319): (128, False, True),
    ("dW", 3198, 5466, 17): (128, True, False),
    ("dW", 257, 1422, 8199): (256, False, False),
    ("dW", 261, 4100, 7202): (256, False, True),
    ("dW", 8973, 140, 6708): (256, True, False),
}


def axes(form, M, R, K):
    """(rows, columns, length of the sums) of the product."""
    return {"fwd": (M, R, K), "dX": (M, K, R), "dW": (R, K, M)}[form]
