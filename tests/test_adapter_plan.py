"""The grid of the adapters' backward pass, on the host (no kernel is launched;
runs without a GPU): every workgroup has a piece of work of its own, or none."""
from __future__ import annotations

import ctypes
import os

import pytest

GRADIENTS, DX, NOTHING = range(3)


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("rt", "ks", "kd", "tiles", "few", "split", "slices")] + [("part", ctypes.c_size_t)]


class Grid(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("a", "b", "groups", "z", "x")] + [(n, ctypes.c_uint) for n in ("gx", "gy")] +
                [(n, ctypes.c_longlong) for n in ("dw", "all")])


@pytest.fixture(scope="module")
def lib():
    from activation_sparse_gated_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return _lib.load()


def grid(lib, m, n, k, r, groups, dx, da, db):
    """(plan, grid, part) of csrc/adapter.cuh: part(w) is what workgroup w of the grid has to do."""
    plan = lib._ZN3ffn12adapter_planEiiiiib
    plan.restype, plan.argtypes = Plan, [ctypes.c_int] * 5 + [ctypes.c_bool]
    p = plan(m, n, k, r, groups, True)
    make = lib._ZN3ffn17adapter_back_gridERKNS_11AdapterPlanEiiiibbb
    make.restype, make.argtypes = Grid, [ctypes.POINTER(Plan)] + [ctypes.c_int] * 4 + [ctypes.c_bool] * 3
    g = make(p, n, k, r, groups, dx, da, db)
    part = lib._ZN3ffn17adapter_back_partERKNS_8BackGridEx
    part.restype, part.argtypes = ctypes.c_int, [ctypes.POINTER(Grid), ctypes.c_longlong]
    return p, g, lambda w: part(g, w)


WIDE = 2 ** 22
SHAPES = [(5, 64, 64, 16, 2), (31, 4096, 4096, 64, 1), (4095, 8192, 2048, 16, 8), (8450, 264, 136, 128, 100), (2050, 72, 16392, 24, 64),
          # more than 2^23 workgroups of gradients, an odd number of them among others
          (64, 4600, WIDE, 8, 1023), (64, 4600, WIDE, 8, 1022), (64, WIDE, 4600, 8, 1023), (2 ** 20, 4600, WIDE - 8, 8, 1023),
          # and of dx
          (2 ** 22, 8, 65536, 8, 1024), (2 ** 26, 8, 4096, 256, 1024), (2 ** 26, 64, 2056, 16, 1)]


@pytest.mark.parametrize("need", [(1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1), (1, 1, 0)], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_workgroups_past_the_work_do_nothing(lib, shape, need):
    m, n, k, r, groups = shape
    dx, da, db = map(bool, need)
    p, g, part = grid(lib, m, n, k, r, groups, dx, da, db)
    there = g.gx * g.gy
    assert g.gx < 2 ** 24 and g.gy <= 65535              # 256 threads each: fewer than 2^32 a dimension
    assert (g.a > 0, g.b > 0, g.x > 0) == (da, db, dx)
    gradients, rows = (g.a + g.b) * groups * g.z, g.x * p.tiles
    assert g.dw == gradients and g.all == gradients + rows and g.all <= there < g.all + g.gy
    for at, many, what in ((0, gradients, GRADIENTS), (gradients, rows, DX), (gradients + rows, there - gradients - rows, NOTHING)):
        for w in {at, at + many // 2, at + many - 1} if many else ():
            assert part(w) == what, (w, g.all, there)
    if dx:                                               # the last one's tile is the last there is
        assert (g.all - 1 - g.dw) // g.x == p.tiles - 1


def test_a_surplus_workgroup_is_among_the_cases(lib):
    _, g, _ = grid(lib, 64, 4600, WIDE, 8, 1023, False, True, True)
    assert g.gy > 1 and g.gx * g.gy > g.all
