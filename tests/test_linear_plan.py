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
