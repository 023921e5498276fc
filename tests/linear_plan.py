"""Which kernel, tile and slices a product takes: lin_plan of the built library
(a rule on sizes alone, csrc/linear.cuh), called on the host."""
from __future__ import annotations

import ctypes

FP8, FWD, DX, DW = range(4)


class _Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("skinny", "mb", "nw", "rt", "ct", "ks")]


def plan(kind, exact, rows, cols, k, groups):
    """("few", 16-row blocks, waves, slices) or (tile rows, tile columns, slices)."""
    from activation_sparse_gated_amd import _lib
    fn = getattr(_lib.load(), "_ZN3ffn8lin_planEiiiiii")
    fn.restype, fn.argtypes = _Plan, [ctypes.c_int] * 6
    p = fn(kind, int(exact), rows, cols, k, groups)
    return ("few", p.mb, p.nw, p.ks) if p.skinny else (p.rt, p.ct, p.ks)
