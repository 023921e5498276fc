"""The rule that picks a product's kernel, tile and slices, on the host (no
kernel is launched; runs without a GPU)."""
from __future__ import annotations

import os

import pytest

from tests import linear_plan as P


@pytest.fixture(scope="module", autouse=True)
def built():
    from activation_sparse_gated_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")


@pytest.mark.parametrize("n,k,groups", [(8, 8, 1), (64, 4096, 1), (256, 256, 1), (64, 64, 2)])
def test_weight_gradient_over_2_30_rows_and_more(n, k, groups):
    # the rows of x are the contraction: more of them, up to the most there may be, change no tile
    want = P.plan(P.DW, 0, n, k, 2 ** 28, groups)
    for m in (2 ** 29, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 2 ** 20, 2 ** 31 - 2 ** 16):
        assert P.plan(P.DW, 0, n, k, m, groups) == want, m


def test_the_cases_take_every_instance():
    # what the GPU tests of the tiles run: every kernel that a product may take, with and without slices
    from tests import linear_cases as C
    got = C.instances()
    tiles = [(64, 128), (128, 128), (128, 256), (256, 256)]
    few = [("few", 1, 8, "whole"), ("few", 1, 16, "whole"), ("few", 1, 16, "sliced"), ("few", 2, 8, "whole"), ("few", 2, 8, "sliced")]
    for cut in ("whole", "sliced"):
        for t in tiles:
            for exact in (0, 1):
                if exact and t == (256, 256):
                    continue                             # exact sums end at 128 x 256
                for rows in (1, 128):
                    assert (P.FP8, exact, rows, *t, cut) in got
            assert (P.FWD, 0, 0, *t, cut) in got and (P.DX, 0, 0, *t, cut) in got
            assert cut == "sliced" or (P.DW, 0, 0, *t, cut) in got
    for f in few:
        assert all((P.FP8, exact, rows, *f) in got for exact in (0, 1) for rows in (1, 128)) and (P.FWD, 0, 0, *f) in got
    # and both with offsets and without
    for exact in (0, 1):
        for key in [(*t, c) for t in tiles for c in ("whole", "sliced") if not (exact and t == (256, 256))] + few:
            cases = got[(P.FP8, exact, 128, *key)]
            assert any(c[3] for c in cases) and any(not c[3] for c in cases), (exact, key, cases)
