"""Sizes of products that take every instance of the product kernels: each kind
of product, tile, way of summing and of scaling, whole and cut along the
contraction. Sizes are ragged on every side; the large ones have more tiles than
run at once and several whole steps of the contraction before a partial one."""
from __future__ import annotations

import numpy as np

from tests import linear_plan as P

# m, n, k, experts (0: no offsets)
FP8 = [
    (3, 136, 8208, 0), (3, 264, 4112, 0), (7, 77, 400, 0), (20, 136, 8208, 0), (24, 264, 2064, 0),
    (232, 130, 720, 0), (67, 144, 1840, 0), (8219, 1908, 864, 0), (652, 140, 7648, 0), (2772, 130, 4064, 0), (5096, 3078, 720, 0),
    (8723, 1848, 704, 0), (2747, 680, 9744, 0), (6662, 1169, 720, 0), (4128, 481, 6032, 0), (5477, 4444, 720, 0),
    (8414, 420, 8224, 0), (4851, 793, 8432, 0),
    (3, 136, 8208, 4), (9, 136, 4112, 2), (7, 77, 400, 3), (40, 136, 4112, 3), (29, 77, 656, 2),
    (237, 129, 720, 3), (107, 132, 1744, 3), (738, 8861, 1888, 8), (3913, 3952, 720, 3), (1127, 140, 3680, 8), (4269, 3086, 704, 8),
    (444, 129, 11600, 8), (1453, 6652, 720, 8), (432, 2844, 8880, 3), (8411, 933, 704, 8), (4037, 436, 6624, 3),
    (3226, 6824, 720, 5), (8045, 393, 8640, 5)]
FWD = [
    (3, 136, 4104, 1), (5, 72, 328, 3), (40, 136, 4104, 3), (29, 72, 328, 2), (3, 136, 8200, 4), (2, 520, 2056, 1),
    (221, 136, 456, 1), (104, 152, 848, 3), (780, 8840, 928, 8), (1294, 152, 1896, 3), (5902, 2568, 424, 3), (3545, 272, 6536, 5),
    (2062, 4200, 408, 8), (6913, 264, 7312, 5), (8762, 2744, 408, 3), (5730, 4400, 408, 1)]
BWD = [  # for dx
    (200, 456, 136, 1), (79, 872, 136, 3), (651, 936, 8912, 8), (1294, 1888, 136, 3), (6122, 408, 2360, 8), (1751, 12768, 264, 3),
    (1391, 408, 6640, 5), (7074, 7504, 264, 3), (8527, 408, 2744, 8), (6373, 408, 3856, 1),
    # for dw
    (719, 72, 144, 3), (3517, 4320, 264, 8), (3354, 72, 8232, 8), (3239, 416, 6232, 8), (414, 3848, 4104, 1), (412, 2144, 7184, 1),
    (402, 5272, 4632, 1)]


def offsets(m, groups):
    """Uneven experts, one of them (of three and more) without rows, rows of no expert before the first and after the last."""
    g = np.random.default_rng([61, m, groups])
    lo, hi = (2, m - 3) if m > 20 else (0, m)
    cuts = np.sort(g.integers(lo, hi + 1, groups - 1))
    off = np.concatenate([[lo], cuts, [hi]])
    if groups > 2:
        off[2] = off[1]
    return [int(v) for v in off]


def _key(p):
    return p[:-1] + ("sliced" if p[-1] > 1 else "whole",)


def instances():
    """{(kind, exact, row scales, kernel and tile, sliced or whole): a case that takes it}."""
    out = {}
    for m, n, k, e in FP8:
        for exact in (0, 1):
            for rows in (1, 128) if not e else (128,):
                out.setdefault((P.FP8, exact, rows, *_key(P.plan(P.FP8, exact, m, n, k, max(e, 1)))), []).append((m, n, k, e))
    for m, n, k, e in FWD:
        out.setdefault((P.FWD, 0, 0, *_key(P.plan(P.FWD, 0, m, n, k, e))), []).append((m, n, k, e))
    for m, n, k, e in BWD:
        out.setdefault((P.DX, 0, 0, *_key(P.plan(P.DX, 0, m, k, n, e))), []).append((m, n, k, e))
        out.setdefault((P.DW, 0, 0, *_key(P.plan(P.DW, 0, n, k, m, e))), []).append((m, n, k, e))
    return out
