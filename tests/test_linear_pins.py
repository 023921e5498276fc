"""Pins of the fp64 definitions of the operators around the FFN (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import linear_oracle as L


def test_e4m3_table():
    v = L.e4m3_values()
    assert v[0x7E] == 448.0 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0x38] == 1.0
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF]) and v[0xB8] == -1.0
    assert np.all(np.diff(v[:127]) > 0)


def test_e4m3_round_is_nearest_even():
    v = L.e4m3_values()[:127]
    assert np.array_equal(L.e4m3_round(v), np.arange(127))
    mid = (v[:-1] + v[1:]) / 2
    want = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127))
    assert np.array_equal(L.e4m3_round(mid), want)
    assert np.array_equal(L.e4m3_round(np.nextafter(mid, 0)), np.arange(126))
    assert np.array_equal(L.e4m3_round(np.nextafter(mid, 1e9)), np.arange(1, 127))
    assert np.array_equal(L.e4m3_round(-mid), want | 0x80)


def test_e4m3_matches_torch():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(0).normal(0, 60, 4000).astype(np.float32)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(L.e4m3_round(x), want)


@pytest.mark.parametrize("rows", [1, 128])
def test_blocks_stand_for_x(rows):
    x = np.random.default_rng(1).normal(0, 3, (130, 200)).astype(np.float32)
    x[5] = 0
    q, s = L.blocks(x, rows)
    assert s.shape == (-(-130 // rows), 2)
    back = L.values(q, s, rows)
    step = np.repeat(np.repeat(s, rows, 0)[:130], 128, 1)[:, :200]
    # half a step: 2^-4 relative, or half of the smallest step 2^-9 of the scale
    assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x) * (1 + 1e-6), 2.0 ** -10 * step))
    assert np.all(back[5] == 0)


def test_blocks_of_extremes():
    x = np.zeros((4, 128), np.float32)
    x[1, 3], x[2, 7], x[3, :] = np.inf, np.nan, 1e-42
    x[1, 4] = x[2, 4] = 1.0
    q, s = L.blocks(x, 1)
    v = L.values(q, s, 1)
    assert s[0, 0] == L.FLOOR and np.all(v[0] == 0) and np.all(np.isnan(v[1])) and np.all(np.isnan(v[2]))
    assert s[3, 0] == L.FLOOR and np.all(v[3] == 0)


def test_norm_gradients_against_differences():
    g = np.random.default_rng(2)
    r, w, dy, dr = g.normal(0, 2, (3, 24)), g.normal(1, .3, 24), g.normal(0, 1, (3, 24)), g.normal(0, 1, (3, 24))
    dx, dw = L.rmsnorm_backward(r, w, dy, dr, 1e-3)
    loss = lambda r, w: np.sum(dy * L.rmsnorm(r, w, 1e-3)) + np.sum(dr * r)  # noqa: E731
    h = 1e-5
    for _ in range(8):
        u, v = g.normal(0, 1, r.shape), g.normal(0, 1, w.shape)
        assert abs((loss(r + h * u, w) - loss(r - h * u, w)) / (2 * h) - np.sum(dx * u)) < 1e-7
        assert abs((loss(r, w + h * v) - loss(r, w - h * v)) / (2 * h) - np.sum(dw * v)) < 1e-7


def test_grouped_gradients_against_differences():
    g = np.random.default_rng(3)
    x, w, dy, off = g.normal(0, 1, (7, 5)), g.normal(0, 1, (3, 4, 5)), g.normal(0, 1, (7, 4)), [1, 3, 3, 6]
    dx, dw = L.grouped_backward(x, w, dy, off, np.zeros((7, 5)))
    loss = lambda x, w: np.sum(dy * L.grouped(x, w, off, np.zeros((7, 4))))  # noqa: E731
    for _ in range(6):
        u, v = g.normal(0, 1, x.shape), g.normal(0, 1, w.shape)
        # linear in each argument: the difference is exact but for rounding
        assert abs(loss(x + u, w) - loss(x, w) - np.sum(dx * u)) < 1e-10
        assert abs(loss(x, w + v) - loss(x, w) - np.sum(dw * v)) < 1e-10
    assert np.all(dx[[0, 6]] == 0) and np.all(dw[1] == 0)
