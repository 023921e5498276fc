"""Python binding of the low-rank adapters (include/ffn_adapter.h).

Argument checks and marshalling only, as in linear.py: tensors are contiguous
and on one GPU, outputs that are not passed in are allocated, `stream` is taken
by every function, and what does not fit raises ValueError before anything is
launched.

`offsets` and `rows` say which rows an adapter has: rows[offsets[g]] ..
rows[offsets[g + 1] - 1], or those rows themselves without `rows`. Both come from
group_rows(adapter of each row, n_adapters); they are the same for every layer of
a step.
"""
from __future__ import annotations

import functools

import torch

from . import _lib
from .linear import (_DTYPES, _accumulator, _again, _call, _check, _fail, _first, _nbytes, _no_size,
                     _product_out, _ptr, _workspace)


@functools.lru_cache(maxsize=256)
def _bytes(name, *shape):
    """A workspace's size, which the shape alone decides (the C call takes 0.6 us)."""
    return getattr(_lib.load(), name)(*shape)


def _shapes(x, a, b):
    """(device, m, k, adapters, r, n) of the rows and the adapters."""
    dev = _first("x", x, (torch.bfloat16,), (2,))
    for name, t in (("a", a), ("b", b)):
        if getattr(t, "ndim", 0) != 3:
            _fail(name, t, "bfloat16 tensor of 3 dimensions")
    m, k = x.shape
    groups, r, _ = a.shape
    n = b.shape[1]
    _check("a", a, torch.bfloat16, (groups, r, k), dev)
    _check("b", b, torch.bfloat16, (groups, n, r), dev)
    if (m | k | groups | r | n) >> 31:
        _no_size("x, a, b", m, k, groups, r, n)
    return dev, m, k, groups, r, n


def _order(offsets, rows, groups, m, dev):
    _check("offsets", offsets, torch.int32, (groups + 1,), dev)
    if rows is not None:
        _check("rows", rows, torch.int32, (m,), dev)


def adapter_forward(x, a, b, offsets, *, rows=None, scales=None, base=None, y=None, out_dtype=torch.bfloat16,
                    workspace=None, stream=None):
    """y[t] = base[t] + scales[g] B_g A_g x[t] for the rows t of each adapter g,
    base[t] for rows without one (ffn_adapter_forward).

    x [m, k] bf16; a [adapters, r, k], b [adapters, n, r] bf16; scales fp32
    [adapters] or None (ones); base [m, n], the shared projection's output, or
    None (zeros). y [m, n] of base's type (out_dtype without a base: bf16 or
    fp32); it may be base, which is then added to in place."""
    if stream is not None:
        return _again(adapter_forward, locals())
    dev, m, k, groups, r, n = _shapes(x, a, b)
    _order(offsets, rows, groups, m, dev)
    if scales is not None:
        _check("scales", scales, torch.float32, (groups,), dev)
    if base is not None:
        if getattr(base, "dtype", None) in _DTYPES:
            out_dtype = base.dtype
        _check("base", base, out_dtype, (m, n), dev)
        if y is None:
            y = torch.empty_like(base)
        elif y is not base:
            _check("y", y, out_dtype, (m, n), dev)
    else:
        y = _product_out(y, (m, n), out_dtype, dev)
    workspace = _workspace(workspace, _bytes("ffn_adapter_forward_workspace_bytes", m, n, k, r, groups), dev)
    _call(_lib.load().ffn_adapter_forward, dev, _ptr(x), _ptr(a), _ptr(b), _ptr(scales), _ptr(offsets), _ptr(rows), groups, m, n,
          k, r, _ptr(base), _ptr(y), _DTYPES[y.dtype], _ptr(workspace), _nbytes(workspace))
    return y


def adapter_backward(x, a, b, dy, offsets, *, rows=None, scales=None, base=None, need_dx=True, need_da=True, need_db=True,
                     dx=None, da=None, db=None, accumulate=False, workspace=None, stream=None):
    """Gradients of adapter_forward (ffn_adapter_backward): (dx, da, db); that of
    base is dy itself.

    dy [m, n] bf16. dx [m, k] bf16: base[t] (the shared projection's gradient of
    x, or None: zeros) + scales[g] A_g^T B_g^T dy[t]; it may be base. da
    [adapters, r, k] and db [adapters, n, r] fp32, written (zeros for an adapter
    without rows) or added to with accumulate. One that is not needed is not
    computed: None in its place."""
    if stream is not None:
        return _again(adapter_backward, locals())
    if not (need_dx or need_da or need_db):
        raise ValueError("need_dx, need_da, need_db: one of the gradients at least")
    for name, need, t in (("dx", need_dx, dx), ("base", need_dx, base), ("da", need_da, da), ("db", need_db, db)):
        if t is not None and not need:
            raise ValueError(f"{name}: given without need_{'dx' if name == 'base' else name}")
    if accumulate and not (need_da or need_db):
        raise ValueError("accumulate: given without need_da or need_db")
    dev, m, k, groups, r, n = _shapes(x, a, b)
    _check("dy", dy, torch.bfloat16, (m, n), dev)
    _order(offsets, rows, groups, m, dev)
    if scales is not None:
        _check("scales", scales, torch.float32, (groups,), dev)
    if base is not None:
        _check("base", base, torch.bfloat16, (m, k), dev)
    if need_dx:
        if dx is None:
            dx = torch.empty_like(x)
        else:
            _check("dx", dx, torch.bfloat16, (m, k), dev)
    if need_da:
        da = _accumulator("da", da, accumulate, (groups, r, k), dev)
    if need_db:
        db = _accumulator("db", db, accumulate, (groups, n, r), dev)
    workspace = _workspace(workspace, _bytes("ffn_adapter_backward_workspace_bytes", m, n, k, r, groups), dev)
    _call(_lib.load().ffn_adapter_backward, dev, _ptr(x), _ptr(a), _ptr(b), _ptr(scales), _ptr(dy), _ptr(offsets), _ptr(rows),
          groups, m, n, k, r, _ptr(base), _ptr(dx), _ptr(da), _ptr(db), int(bool(accumulate)), _ptr(workspace),
          _nbytes(workspace))
    return dx, da, db
