"""Pins of the fp64 definitions of routing to experts, rows and adapters (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import experts_oracle as E


def test_route_by_hand():
    l = np.log([[1.0, 2.0, 4.0, 1.0]])
    w, ids, p = E.route(l, 2)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[2 / 3, 1 / 3]]) and np.allclose(p, [[.125, .25, .5, .125]])
    w, ids, _ = E.route(l, 2, renormalize=False, scale=2.0)
    assert np.allclose(w, [[1.0, 0.5]])
    # a bias for the choice alone; ties to the lower index
    w, ids, _ = E.route(l, 2, bias=[0.375, 0.0, 0.0, 0.0], renormalize=False)
    assert ids.tolist() == [[0, 2]] and np.allclose(w, [[.125, .5]])
    # two groups: by the best one, and by the sum of the best two
    l = np.log([[8.0, 1.0, 6.0, 5.0]])
    assert E.route(l, 2, groups=2, top_groups=1)[1].tolist() == [[0, 1]]
    assert E.route(l, 2, groups=2, top_groups=1, group_best=2)[1].tolist() == [[2, 3]]


def test_route_without_experts():
    l = np.array([[-np.inf] * 4, [-np.inf, 0.0, -np.inf, 1.0]])
    w, ids, p = E.route(l, 3)
    assert ids.tolist() == [[-1] * 3, [3, 1, -1]] and np.all(w[0] == 0) and np.all(p[0] == 0) and w[1, 2] == 0
    assert np.isclose(w[1].sum(), 1)
    w, ids, p = E.route(l, 3, sigmoid=True, bias=np.ones(4), groups=2, top_groups=1, group_best=2)
    assert ids.tolist() == [[-1] * 3, [3, -1, -1]]


def test_small_sigmoids_keep_their_ratio():
    w, _, _ = E.route(np.array([[-1000.0, -1001.0]]), 2, sigmoid=True)
    assert np.allclose(w, [[1 / (1 + np.exp(-1.0)), 1 / (1 + np.exp(1.0))]])


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_against_differences(sigmoid, renormalize):
    g = np.random.default_rng(5)
    l, dw, ds = g.normal(0, 1, (3, 9)), g.normal(0, 1, (3, 4)), g.normal(0, 1, (3, 9))
    kw = dict(sigmoid=sigmoid, renormalize=renormalize, scale=1.7)
    ids = E.route(l, 4, **kw)[1]

    def loss(l):
        p = E.scores(l, sigmoid)
        w = np.stack([1.7 * E.weights(l[t, ids[t]], p[t, ids[t]], sigmoid, renormalize) for t in range(3)])
        return np.sum(dw * w) + np.sum(ds * p)
    got = E.route_backward(l, ids, dw, ds, **kw)
    for _ in range(8):
        u, h = g.normal(0, 1, l.shape), 1e-5
        assert abs((loss(l + h * u) - loss(l - h * u)) / (2 * h) - np.sum(got * u)) < 1e-8


def test_group_by_hand():
    off, rows, slots = E.group(np.array([[2, 0], [-1, 2], [0, 7]]), 3)
    assert off.tolist() == [0, 2, 2, 4] and rows.tolist() == [1, 4, 0, 3, 2, 5]
    assert slots.tolist() == [[2, 0], [-1, 3], [1, -1]]


def test_combine_gradients_against_differences():
    g = np.random.default_rng(6)
    slots = np.array([[3, 0], [-1, 5], [2, 4]])
    y, w, dout = g.normal(0, 1, (6, 8)), g.normal(0, 1, (3, 2)), g.normal(0, 1, (3, 8))
    dy, dw = E.combine_backward(y, slots, w, dout, np.zeros((6, 8)))
    u, v = g.normal(0, 1, y.shape), g.normal(0, 1, w.shape)
    f = lambda y, w: np.sum(dout * E.combine(y, slots, w, None))  # noqa: E731
    assert abs(f(y + u, w) - f(y, w) - np.sum(dy * u)) < 1e-12 and abs(f(y, w + v) - f(y, w) - np.sum(dw * v)) < 1e-12
    # the gather's gradient is the combination without weights
    x = g.normal(0, 1, (3, 8))
    assert abs(np.sum(y * E.gather(x, slots, np.zeros((6, 8)))) - np.sum(x * E.combine(y, slots, None, None))) < 1e-12


def test_adapter_gradients_against_differences():
    g = np.random.default_rng(7)
    x, a, b, dy = g.normal(0, 1, (7, 5)), g.normal(0, 1, (3, 2, 5)), g.normal(0, 1, (3, 4, 2)), g.normal(0, 1, (7, 4))
    s, off, rows = [0.5, 2.0, 1.5], [1, 3, 3, 6], [6, 2, 0, 1, 5, 4, 3]
    base = g.normal(0, 1, (7, 4))
    dx, da, db = E.adapter_backward(x, a, b, s, dy, off, rows, None)
    f = lambda x, a, b: np.sum(dy * E.adapter(x, a, b, s, off, rows, base))  # noqa: E731
    for _ in range(4):
        u, v, w = g.normal(0, 1, x.shape), g.normal(0, 1, a.shape), g.normal(0, 1, b.shape)
        # linear in each: the difference is exact but for rounding
        assert abs(f(x + u, a, b) - f(x, a, b) - np.sum(dx * u)) < 1e-10
        assert abs(f(x, a + v, b) - f(x, a, b) - np.sum(da * v)) < 1e-10
        assert abs(f(x, a, b + w) - f(x, a, b) - np.sum(db * w)) < 1e-10
    y = E.adapter(x, a, b, s, off, rows, base)
    assert np.array_equal(y[[6, 3]], base[[6, 3]]) and np.all(da[1] == 0) and np.all(dx[[6, 3]] == 0)


def test_offsets_out_of_range():
    assert E.adapter_rows([-3, 2, 1, 99], None, 4, 3) == [[0, 1], [], [2, 3]]
    assert E.adapter_rows([0, 3], [1, 9, -1, 0], 4, 1) == [[1]]
