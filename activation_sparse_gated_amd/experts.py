"""Python binding of routing to experts (include/ffn_experts.h).

Argument checks and marshalling only, as in linear.py: tensors are contiguous
and on one GPU, outputs that are not passed in are allocated, `stream` is taken
by every function, and what does not fit raises ValueError before anything is
launched.

A layer of experts, forward (backward the same way back):

    weights, ids, _ = route_forward(logits, 2)
    offsets, rows, slots = group_rows(ids, n_experts)
    y = grouped_forward(gather_forward(x, slots), w, offsets)
    out = combine_forward(y, slots, weights)
"""
from __future__ import annotations

import torch

from . import _lib
from .linear import (_DTYPES, FP8, Fp8Tensor, _again, _blocks, _call, _check, _check_fp8, _fail, _first, _nbytes,
                     _no_size, _ptr, _workspace)

_TYPES = (torch.bfloat16, torch.float32)


def _score(score):
    if score not in _lib.SCORES:
        raise ValueError(f"score: {' or '.join(_lib.SCORES)}, got {score!r}")
    return _lib.SCORES[score]


def _out(name, t, dtype, shape, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _check(name, t, dtype, shape, dev)
    return t


def _out_like(name, t, ref, shape):
    """The same in ref's type, on its device."""
    if t is None:
        return ref.new_empty(shape)
    _check(name, t, ref.dtype, shape, ref.device)
    return t


def _pairs(name, t, m, dev):
    """The second dimension of an int32 tensor [m, .]; m None: any."""
    if getattr(t, "ndim", 0) != 2:
        _fail(name, t, "int32 tensor of 2 dimensions")
    _check(name, t, torch.int32, t.shape if m is None else (m, t.shape[1]), dev)
    top_k = t.shape[1]
    if top_k >> 31:
        _no_size(name, top_k)
    return top_k


# ---------------------------------------------------------------- router
def route_forward(logits, top_k, *, score="softmax", bias=None, groups=1, top_groups=None, group_best=1,
                  renormalize=True, scale=1.0, scores=False, weights=None, ids=None, stream=None):
    """The choice of top_k experts for each token and their weights
    (ffn_route_forward): (weights, ids, scores).

    logits [m, experts] bf16 or fp32; score "softmax" or "sigmoid"; bias fp32
    [experts] is added for the choice alone. With groups, experts come from the
    top_groups groups (all of them if None) with the largest sums of their
    group_best (1 or 2) best values. weights fp32 [m, top_k]: scale * the chosen
    scores, over their sum with renormalize. ids int32 [m, top_k], best first,
    ties to the lower index; -1 (and weight 0) where no expert with a logit above
    -inf is left. scores: fp32 [m, experts], or None unless asked for (True, or
    the tensor that they are written to)."""
    if stream is not None:
        return _again(route_forward, locals())
    dev = _first("logits", logits, _TYPES, (2,))
    m, experts = logits.shape
    if top_k < 1:
        raise ValueError(f"top_k: 1 at least, got {top_k}")
    if top_groups is None:
        top_groups = groups
    if (top_k | groups | top_groups | group_best) >> 31:
        _no_size("top_k, groups, top_groups, group_best", top_k, groups, top_groups, group_best)
    if bias is not None:
        _check("bias", bias, torch.float32, (experts,), dev)
    weights = _out("weights", weights, torch.float32, (m, top_k), dev)
    ids = _out("ids", ids, torch.int32, (m, top_k), dev)
    if scores is False or scores is None:
        scores = None
    else:
        scores = _out("scores", None if scores is True else scores, torch.float32, (m, experts), dev)
    _call(_lib.load().ffn_route_forward, dev, logits.data_ptr(), _DTYPES[logits.dtype], m, experts, top_k,
          _score(score), _ptr(bias), groups, top_groups, group_best,
          int(bool(renormalize)), float(scale), weights.data_ptr(), ids.data_ptr(), _ptr(scores))
    return weights, ids, scores


def route_backward(logits, ids, dweights, *, dscores=None, score="softmax", renormalize=True, scale=1.0, dlogits=None,
                   stream=None):
    """Gradient of route_forward (ffn_route_backward): dlogits [m, experts] of the
    logits' type, the choice held fixed.

    ids [m, top_k] as route_forward gave them; dweights fp32 [m, top_k]; dscores
    fp32 [m, experts] or None. score, renormalize and scale as there."""
    if stream is not None:
        return _again(route_backward, locals())
    dev = _first("logits", logits, _TYPES, (2,))
    m, experts = logits.shape
    top_k = _pairs("ids", ids, m, dev)
    _check("dweights", dweights, torch.float32, (m, top_k), dev)
    if dscores is not None:
        _check("dscores", dscores, torch.float32, (m, experts), dev)
    dlogits = _out_like("dlogits", dlogits, logits, (m, experts))
    _call(_lib.load().ffn_route_backward, dev, logits.data_ptr(), _DTYPES[logits.dtype], m, experts, top_k, _score(score),
          int(bool(renormalize)), float(scale), ids.data_ptr(), dweights.data_ptr(), _ptr(dscores), dlogits.data_ptr())
    return dlogits


# ---------------------------------------------------------------- rows to experts and back
def group_rows(ids, groups, *, offsets=None, rows=None, slots=None, workspace=None, stream=None):
    """The order of entries by group (ffn_group_rows): (offsets, rows, slots).

    ids int32, [m, top_k] experts of route_forward or [m] adapters; what lies
    outside 0 .. groups - 1 has no group and comes last. offsets int32
    [groups + 1], as the products take them; rows int32 [m * top_k], the flat
    index into ids at each place; slots of ids' shape, the place of each entry
    (-1 without a group)."""
    if stream is not None:
        return _again(group_rows, locals())
    dev = _first("ids", ids, (torch.int32,), (1, 2))
    n = ids.numel()
    if groups < 1:
        raise ValueError(f"groups: 1 at least, got {groups}")
    if (n | groups) >> 31:
        _no_size("ids, groups", n, groups)
    offsets = _out("offsets", offsets, torch.int32, (groups + 1,), dev)
    rows = _out_like("rows", rows, ids, (n,))
    slots = _out_like("slots", slots, ids, ids.shape)
    lib = _lib.load()
    workspace = _workspace(workspace, lib.ffn_group_rows_workspace_bytes(n, groups), dev)
    _call(lib.ffn_group_rows, dev, _ptr(ids), n, groups, _ptr(offsets), _ptr(rows), _ptr(slots), _ptr(workspace),
          _nbytes(workspace))
    return offsets, rows, slots


def gather_forward(x, slots, *, fp8=False, y=None, stream=None):
    """y[slots[t, s]] = x[t] (ffn_gather_forward): the tokens' rows in the order of
    group_rows.

    x [m, d] bf16 or fp32; slots int32 [m, top_k], different places (-1: none). y
    [m * top_k, d] of x's type, or with fp8 an Fp8Tensor of blocks of 1 x 128;
    rows that no slot names are left as they were."""
    if stream is not None:
        return _again(gather_forward, locals())
    dev = _first("x", x, _TYPES, (2,))
    m, d = x.shape
    top_k = _pairs("slots", slots, m, dev)
    n = m * top_k
    if fp8:
        if y is None:
            y = Fp8Tensor(torch.empty(n, d, dtype=FP8, device=dev),
                          torch.empty(_blocks(d), n, dtype=torch.float32, device=dev), 1)
        else:
            _check_fp8("y", y, (n, d), 1, dev)
        out, q, scale = None, y.q, y.scale
    else:
        y = _out_like("y", y, x, (n, d))
        out, q, scale = y, None, None
    _call(_lib.load().ffn_gather_forward, dev, _ptr(x), _DTYPES[x.dtype], m, d, _ptr(slots), top_k, _ptr(out), _ptr(q),
          _ptr(scale))
    return y


def gather_backward(dy, slots, *, dx=None, stream=None):
    """Gradient of gather_forward: dx[t] = the sum over s of dy[slots[t, s]]
    (ffn_combine_forward without weights), [m, d] of dy's type."""
    if stream is not None:
        return _again(gather_backward, locals())
    return _combine(dy, slots, None, None, dx, "dy", "dx")


def combine_forward(y, slots, weights=None, *, residual=None, out=None, stream=None):
    """out[t] = residual[t] + the sum over s of weights[t, s] y[slots[t, s]]
    (ffn_combine_forward).

    y [m * top_k, d] bf16 or fp32; slots int32 [m, top_k] of group_rows (-1: adds
    nothing); weights fp32 [m, top_k] or None (ones); residual [m, d] of y's type
    or None; out may be residual."""
    if stream is not None:
        return _again(combine_forward, locals())
    return _combine(y, slots, weights, residual, out, "y", "out")


def _combine(y, slots, weights, residual, out, y_name, out_name):
    dev = _first(y_name, y, _TYPES, (2,))
    top_k = _pairs("slots", slots, None, dev)
    m, (n, d) = slots.shape[0], y.shape
    if n != m * top_k:
        _fail(y_name, y, f"tensor of {m * top_k} rows")
    if weights is not None:
        _check("weights", weights, torch.float32, (m, top_k), dev)
    if residual is not None:
        _check("residual", residual, y.dtype, (m, d), dev)
    out = _out_like(out_name, out, y, (m, d))
    _call(_lib.load().ffn_combine_forward, dev, _ptr(y), _DTYPES[y.dtype], m, d, _ptr(slots), top_k, _ptr(weights),
          _ptr(residual), _ptr(out))
    return out


def combine_backward(y, slots, weights, dout, *, need_dy=True, need_dweights=True, dy=None, dweights=None, stream=None):
    """Gradients of combine_forward (ffn_combine_backward): (dy, dweights); that of
    the residual is dout itself.

    dout [m, d] of y's type. dy [m * top_k, d]: dy[slots[t, s]] = weights[t, s]
    dout[t], rows that no slot names left as they were; it may be y. dweights fp32
    [m, top_k], 0 for a slot without a row. One that is not needed is not
    computed: None in its place. Without dweights, y may be None."""
    if stream is not None:
        return _again(combine_backward, locals())
    if not (need_dy or need_dweights):
        raise ValueError("need_dy, need_dweights: one of the gradients at least")
    if (not need_dy and dy is not None) or (not need_dweights and dweights is not None):
        raise ValueError("dy, dweights: given without need_dy or need_dweights")
    dev = _first("dout", dout, _TYPES, (2,))
    m, d = dout.shape
    top_k = _pairs("slots", slots, m, dev)
    if need_dweights or y is not None:
        _check("y", y, dout.dtype, (m * top_k, d), dev)
    if weights is not None:
        _check("weights", weights, torch.float32, (m, top_k), dev)
    if need_dy:
        dy = _out_like("dy", dy, dout, (m * top_k, d))
    if need_dweights:
        dweights = _out("dweights", dweights, torch.float32, (m, top_k), dev)
    _call(_lib.load().ffn_combine_backward, dev, _ptr(y), _DTYPES[dout.dtype], m, d, _ptr(slots), top_k, _ptr(weights),
          _ptr(dout), _ptr(dy), _ptr(dweights))
    return dy, dweights
