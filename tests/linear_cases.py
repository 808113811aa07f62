"""Sizes that reach each kind of tile of the 16-bit linear, with a reduction of
more than eight stages of 32 (the longest ring of stage buffers) and no whole
last stage, and what the library says that a size is launched as."""

import ctypes

import w4a4_rank_assisted_amd as hsq

# M, K, N, product, its tiles
DEEP = [
    (5, 333, 328, "fwd", "skinny"),
    (17, 328, 333, "fwd", "skinny"),
    (33, 328, 328, "fwd", "skinny"),
    (16, 1160, 328, "fwd", "skinny split"),
    (17, 1001, 333, "fwd", "skinny split"),
    (48, 1160, 333, "fwd", "skinny split"),
    (70, 328, 328, "fwd", "quarters"),
    (70, 1160, 328, "fwd", "split"),
    (70, 328, 333, "fwd", "ragged quarters"),
    (70, 1001, 328, "fwd", "ragged split"),
    (333, 328, 12300, "fwd", "halves"),
    (521, 328, 12300, "fwd", "whole"),
    (5001, 328, 4104, "fwd", "whole + halves"),
    (2049, 328, 8200, "fwd", "whole + quarters"),
    (17, 328, 328, "dX", "quarters"),
    (17, 328, 1160, "dX", "split"),
    (17, 328, 333, "dX", "ragged quarters"),
    (17, 328, 1001, "dX", "ragged split"),
    (521, 328, 328, "dX", "halves"),
    (2049, 4100, 328, "dX", "whole"),
    (1033, 1001, 360, "dX", "whole"),
    (5001, 4104, 328, "dX", "whole + halves"),
    (4097, 4104, 328, "dX", "whole + quarters"),
    (333, 328, 328, "dW", "quarters"),
    (1033, 328, 328, "dW", "split"),
    (333, 333, 328, "dW", "ragged quarters"),
    (1033, 333, 333, "dW", "ragged split"),
    (333, 328, 520, "dW", "halves"),
    (333, 1160, 1001, "dW", "whole"),
    (333, 2056, 12300, "dW", "whole + halves"),
    (333, 4104, 4104, "dW", "whole + quarters"),
]


def units(M, K, N, product):
    """(tiles, units) of one product: the forward one, or dX or dW of a call for
    both."""
    f = hsq._load().hsq_internal_linear_units
    f.restype = None
    v = (ctypes.c_int * 12)()
    f(M, K, N, int(product != "fwd"), v)
    skinny, splits, ragged, full, cut, parts = v[6:] if product == "dW" else v[:6]
    if skinny:
        return "skinny split" if splits > 1 else "skinny", 1
    if splits > 1 or ragged:
        return ("ragged " if ragged else "") + ("split" if splits > 1 else "quarters"), parts
    names = (["whole"] if full else []) + ([{2: "halves", 4: "quarters"}[cut]] if parts else [])
    return " + ".join(names), full + parts
