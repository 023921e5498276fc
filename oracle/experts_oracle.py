"""Plain fp64 definitions of routing to experts, the rows' way to the experts and
back, and low-rank adapters (test infrastructure only). Shares no code with the
kernels.
"""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------- router
def scores(logits, sigmoid):
    l = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if sigmoid:
            return 1 / (1 + np.exp(-l))
        top = np.max(l, -1, keepdims=True)
        e = np.exp(l - np.where(np.isneginf(top), 0, top))
        s = e.sum(-1, keepdims=True)
        return np.where(s > 0, e / np.where(s > 0, s, 1), 0)


def route(logits, top_k, *, sigmoid=False, bias=None, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0):
    """(weights, ids, scores), token by token."""
    l = np.asarray(logits, np.float64)
    m, experts = l.shape
    p = scores(l, sigmoid)
    size = experts // groups
    ids, w = np.full((m, top_k), -1, np.int32), np.zeros((m, top_k))
    for t in range(m):
        v = p[t] + (0 if bias is None else np.asarray(bias, np.float64))
        # without a bias the scores are in the logits' order, which does not saturate
        order = v if bias is not None else l[t]
        of_group = v if bias is not None or group_best == 2 else l[t]
        alive = [e for e in range(experts) if not np.isneginf(l[t, e])]
        if top_groups < groups:
            of = {}
            for g in range(groups):
                best = sorted((of_group[e] for e in alive if e // size == g), reverse=True)[:group_best]
                if best:
                    of[g] = sum(best)
            kept = sorted(of, key=lambda g: (-of[g], g))[:top_groups]
            alive = [e for e in alive if e // size in kept]
        chosen = sorted(alive, key=lambda e: (-order[e], e))[:top_k]
        ids[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = weights(l[t, chosen], p[t, chosen], sigmoid, renormalize)
    return scale * w, ids, p


def weights(l, p, sigmoid, renormalize):
    """Of the chosen ones, from their logits and scores, without the scale."""
    if not renormalize or len(l) == 0:
        return p
    log = -np.logaddexp(0, -l) if sigmoid else l
    e = np.exp(log - log.max())
    return e / e.sum()


def route_backward(logits, ids, dweights, dscores, *, sigmoid=False, renormalize=True, scale=1.0):
    l, dw = np.asarray(logits, np.float64), np.asarray(dweights, np.float64)
    p = scores(l, sigmoid)
    out = np.zeros(l.shape)
    for t in range(len(l)):
        g = np.zeros(l.shape[1]) if dscores is None else np.array(dscores[t], np.float64)
        live = [s for s in range(ids.shape[1]) if 0 <= ids[t, s] < l.shape[1]]
        e = [ids[t, s] for s in live]
        if renormalize:
            # of the logits themselves: w = the softmax of the chosen log scores
            w = weights(l[t, e], p[t, e], sigmoid, True)
            d = scale * w * (dw[t, live] - np.sum(dw[t, live] * w))
            if sigmoid:
                d = d * (1 - p[t, e])
            np.add.at(out[t], e, d)
        else:
            np.add.at(g, e, scale * dw[t, live])
        out[t] += g * p[t] * (1 - p[t]) if sigmoid else p[t] * (g - np.sum(g * p[t]))
    return out


# ---------------------------------------------------------------- rows
def group(ids, groups):
    """(offsets, rows, slots)."""
    flat = [int(v) if 0 <= v < groups else groups for v in np.asarray(ids).reshape(-1)]
    rows = sorted(range(len(flat)), key=lambda i: flat[i])
    slots = np.full(len(flat), -1, np.int32)
    for place, i in enumerate(rows):
        if flat[i] < groups:
            slots[i] = place
    offsets = np.array([sum(v < g for v in flat) for g in range(groups + 1)], np.int32)
    return offsets, np.array(rows, np.int32), slots.reshape(np.shape(ids))


def gather(x, slots, y0):
    y = np.array(y0)
    for t, s in np.ndindex(*slots.shape):
        if 0 <= slots[t, s] < slots.size:
            y[slots[t, s]] = x[t]
    return y


def combine(y, slots, w, residual):
    y = np.asarray(y, np.float64)
    out = np.zeros((len(slots), y.shape[1])) if residual is None else np.array(residual, np.float64)
    for t, s in np.ndindex(*slots.shape):
        if 0 <= slots[t, s] < slots.size:
            out[t] += (1.0 if w is None else float(w[t, s])) * y[slots[t, s]]
    return out


def combine_backward(y, slots, w, dout, dy0):
    y, dout = np.asarray(y, np.float64), np.asarray(dout, np.float64)
    dy, dw = np.array(dy0, np.float64), np.zeros(slots.shape)
    for t, s in np.ndindex(*slots.shape):
        if 0 <= slots[t, s] < slots.size:
            dy[slots[t, s]] = (1.0 if w is None else float(w[t, s])) * dout[t]
            dw[t, s] = np.sum(dout[t] * y[slots[t, s]])
    return dy, dw


# ---------------------------------------------------------------- adapters
def adapter_rows(offsets, rows, m, groups):
    """The rows of each adapter, offsets and rows kept inside 0..m as the contract says."""
    at, out = [min(max(int(v), 0), m) for v in offsets], []
    for g in range(1, groups + 1):
        at[g] = max(at[g], at[g - 1])
    for g in range(groups):
        places = range(at[g], at[g + 1])
        out.append([r for r in (places if rows is None else (int(rows[p]) for p in places)) if 0 <= r < m])
    return out


def adapter(x, a, b, scales, offsets, rows, base):
    x, a, b = (np.asarray(v, np.float64) for v in (x, a, b))
    y = np.zeros((len(x), b.shape[1])) if base is None else np.array(base, np.float64)
    for g, of in enumerate(adapter_rows(offsets, rows, len(x), len(a))):
        s = 1.0 if scales is None else float(scales[g])
        y[of] += s * (x[of] @ a[g].T) @ b[g].T
    return y


def adapter_backward(x, a, b, scales, dy, offsets, rows, base):
    x, a, b, dy = (np.asarray(v, np.float64) for v in (x, a, b, dy))
    dx = np.zeros(x.shape) if base is None else np.array(base, np.float64)
    da, db = np.zeros(a.shape), np.zeros(b.shape)
    for g, of in enumerate(adapter_rows(offsets, rows, len(x), len(a))):
        s = 1.0 if scales is None else float(scales[g])
        dh = s * dy[of] @ b[g]
        dx[of] += dh @ a[g]
        da[g] = dh.T @ x[of]
        db[g] = s * dy[of].T @ (x[of] @ a[g].T)
    return dx, da, db
