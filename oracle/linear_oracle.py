"""Plain fp64 definitions of the operators around the FFN (test infrastructure
only): RMS norm and its gradients, 8-bit blocks, their product, products
grouped by expert. Shares no code with the kernels.

`blocks` is the one function that also evaluates the fp32 steps of its
definition (the scale, its reciprocal and the product with it are fp32 by
definition), so its codes can be compared bit for bit.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
FLOOR = np.float32(2.0 ** -100)


# ---------------------------------------------------------------- e4m3
def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes (OCP e4m3: no infinities, 0x7F is NaN)."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e.astype(np.float64) - 7))
    v[(c & 0x7F) == 0x7F] = np.nan
    return np.where(c >= 128, -v, v)


def e4m3_round(x) -> np.ndarray:
    """Codes of the nearest e4m3 values, ties to the even code; |x| < 464. NaN gives 0x7F."""
    table = e4m3_values()[:127]                  # the finite magnitudes, ascending
    a = np.abs(np.asarray(x, dtype=np.float64))
    up = np.clip(np.searchsorted(table, a), 1, 126)
    lo, hi = table[up - 1], table[up]
    code = np.where((a - lo < hi - a) | ((a - lo == hi - a) & ((up - 1) % 2 == 0)), up - 1, up)
    code = np.where(a == 0, 0, code)
    code = np.where(np.isnan(a), 0x7F, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


# ---------------------------------------------------------------- blocks
def blocks(x, rows):
    """(codes uint8 [m, k], scales fp32 [ceil(m / rows), ceil(k / 128)]) of x [m, k]."""
    x = np.asarray(x, dtype=np.float32)
    m, k = x.shape
    codes = np.zeros((m, k), np.uint8)
    scales = np.zeros((-(-m // rows), -(-k // BLOCK)), np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(scales.shape[0]):
            for j in range(scales.shape[1]):
                b = x[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK]
                s = np.max(np.abs(b)) * np.float32(1.0 / 448.0)
                s = FLOOR if s < FLOOR else np.float32(s)
                scales[i, j] = s
                codes[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK] = e4m3_round(b * (np.float32(1) / s))
    return codes, scales


def values(codes, scales, rows):
    """What blocks stand for, in fp64 (a block with a NaN or infinite scale: NaN)."""
    m, k = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), rows, 0)[:m], BLOCK, 1)[:, :k]
    s = np.where(np.isfinite(s), s, np.nan)
    return e4m3_values()[codes] * s


# ---------------------------------------------------------------- norm
def rmsnorm(r, w, eps):
    r, w = np.asarray(r, np.float64), np.asarray(w, np.float64)
    return r / np.sqrt(np.mean(r * r, -1, keepdims=True) + eps) * w


def rmsnorm_backward(r, w, dy, dr, eps):
    """(dx, dw) of <dy, y> + <dr, r>."""
    r, w, dy = (np.asarray(v, np.float64) for v in (r, w, dy))
    size = np.sqrt(np.mean(r * r, -1, keepdims=True) + eps)
    v = dy * w
    dx = v / size - r * np.mean(v * r, -1, keepdims=True) / size ** 3
    return dx + (0.0 if dr is None else np.asarray(dr, np.float64)), np.sum(dy * r / size, 0)


# ---------------------------------------------------------------- experts
def grouped(x, w, offsets, y0):
    """Rows of y0 that belong to an expert replaced by W_e x."""
    y = np.array(y0, np.float64)
    for e in range(len(w)):
        a, b = offsets[e], offsets[e + 1]
        y[a:b] = np.asarray(x[a:b], np.float64) @ np.asarray(w[e], np.float64).T
    return y


def grouped_backward(x, w, dy, offsets, dx0):
    x, w, dy = (np.asarray(v, np.float64) for v in (x, w, dy))
    dx, dw = np.array(dx0, np.float64), np.zeros(w.shape)
    for e in range(len(w)):
        a, b = offsets[e], offsets[e + 1]
        dx[a:b] = dy[a:b] @ w[e]
        dw[e] = dy[a:b].T @ x[a:b]
    return dx, dw
