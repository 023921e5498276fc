"""How the products of 8-bit blocks are summed (ffn_fp8_linear in
include/ffn_linear.h), on inputs whose exact sums fp32 holds.

Products are integers (times powers of two), and the magnitudes of all products
of an output add up to less than 2^24 of their unit: fp32 holds every partial
sum, in whatever order, so an fp32 output has to be equal, bit for bit. In every
eight (8 consecutive k) that has them, 2^16 and -2^16 cancel and leave the small
products beside them, which the e4m3 instructions cut 13 bits below 2^16, that
is below 2^3.
"""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def asg(lib):
    return lib


def blocks_of(asg, values, scale, rows):
    """Blocks of e4m3 values and given scales, on the GPU."""
    import torch
    v = torch.from_numpy(np.ascontiguousarray(values, dtype=np.float32)).cuda()
    q = v.to(torch.float8_e4m3fn)
    assert bool((q.float() == v).all())                  # e4m3 values already
    return asg.Fp8Tensor(q, torch.from_numpy(np.ascontiguousarray(scale, dtype=np.float32)).cuda(), rows)


# rows: the few-row kernel with 16 and 32, then every tile a small product takes
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("m", [1, 16, 24, 70, 300, 700])
def test_small_products_beside_cancelling_ones(asg, m, rows):
    import torch
    print("[case] cancelling", m, rows, flush=True)
    n, k = 136, 208
    g = np.random.default_rng([51, m, rows])
    x, w = np.zeros((m, k)), np.zeros((n, k))
    small = np.zeros((m, n))
    for e in range(k // 8):                              # in each eight: the pair at two places, one small product at a third
        a, b, c = 8 * e + g.permutation(8)[:3]
        sign = g.choice([-1, 1], m)
        x[:, a], x[:, b], w[:, a], w[:, b] = 256 * sign, 256 * sign, 256, -256
        x[:, c], w[:, c] = g.integers(-3, 4, m), g.integers(-2, 3, n)
        small += np.outer(np.abs(x[:, c]), np.abs(w[:, c]))
    kb = -(-k // 128)
    xs = 2.0 ** g.integers(0, 2, (kb, m))
    ws = 2.0 ** g.integers(0, 2, (kb, n) if rows == 1 else (-(-n // 128), kb))
    X = x * np.repeat(xs.T, 128, 1)[:, :k]
    W = w * (np.repeat(ws.T, 128, 1)[:, :k] if rows == 1 else np.repeat(np.repeat(ws, 128, 0)[:n], 128, 1)[:, :k])
    want = X @ W.T                                       # integers: exact in fp64
    assert np.max(np.abs(X) @ np.abs(W).T) < 2 ** 24 and np.any(want)
    xb, wb = blocks_of(asg, x, xs, 1), blocks_of(asg, w, ws, rows)
    got = asg.fp8_linear(xb, wb, out_dtype=torch.float32).cpu().numpy()
    assert np.array_equal(got, want)
    acc = torch.full((m, n), 3.0, device="cuda")
    assert np.array_equal(asg.fp8_linear(xb, wb, y=acc, accumulate=True).cpu().numpy(), want + 3)
    # bf16: the pair is exact, the one small product of each eight loses less than 2^-13 2^16 (scaled), and no more than
    # there is of it; then one rounding of half a bf16 step
    got = asg.fp8_linear(xb, wb).float().cpu().numpy()
    lost = np.zeros((m, n))
    for e in range(k // 8):
        ax, aw = X[:, 8 * e:8 * e + 8], W[:, 8 * e:8 * e + 8]
        p = ax[:, None, :] * aw[None]
        lost += np.sum(np.abs(np.where(np.abs(p) < 8 * np.max(np.abs(p), -1, keepdims=True) / 2 ** 16, p, 0)), -1)
    assert np.all(np.abs(got - want) <= lost + 2.0 ** -8 * (np.abs(want) + lost))


@pytest.mark.parametrize("m", [1, 24, 70, 300])
def test_bits_kept_below_the_largest_product(asg, m):
    # 2^16 - 2^16 + v in one eight, at every place: v = 2^3 is kept; in different eights any v is
    print("[case] bits kept", m, flush=True)
    n, k = 56, 144
    for v, apart, kept in ((8, False, True), (24, False, True), (1, True, True), (4, True, True), (2, False, False)):
        x, w = np.zeros((m, k)), np.zeros((n, k))
        places = [(a, b, c) for a in range(8) for b in range(8) for c in range(8) if len({a, b, c}) == 3]
        for i in range(n):
            a, b, c = places[i * 6 % len(places)]
            c = 16 + c if apart else c
            w[i, a], w[i, b], w[i, c] = 256, -256, v / 2
        x[:, :8], x[:, 16:24] = 256, 2
        if not apart:                                    # the small product's partner: 2 at its place, 256 at the pair's
            x[:, :8] = 256
            for i in range(n):
                a, b, c = places[i * 6 % len(places)]
                w[i, c] = v / 256                        # 256 * v / 256
        want = np.full((m, n), float(v))
        assert np.array_equal(x @ w.T, want)
        one = np.ones((2, m))
        xb, wb = blocks_of(asg, x, one, 1), blocks_of(asg, w, np.ones((1, 2)), 128)
        got = asg.fp8_linear(xb, wb).float().cpu().numpy()
        assert np.array_equal(got, want) if kept else np.all(np.abs(got - want) < 8), (v, apart)
        import torch
        assert np.array_equal(asg.fp8_linear(xb, wb, out_dtype=torch.float32).cpu().numpy(), want)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("m", [1, 24, 70, 300])
def test_scales_at_both_ends_of_their_range(asg, m, rows):
    """Products of two scales from 2^-126 to 2^127, and blocks of zeros whose scales' product is far below."""
    import torch
    print("[case] scales", m, rows, flush=True)
    n, k = 136, 272
    g = np.random.default_rng([53, m, rows])
    kb, nb = 3, 2
    x, w = np.zeros((m, k)), g.integers(-1, 2, (n, k)).astype(float)
    x[np.arange(m), g.integers(0, k, m)] = g.choice([-1, 1], m)      # one product an output: -1, 0 or 1
    for a, b in ((64, 63), (127, 0), (0, 127), (-63, -63), (-126, 0), (0, -126), (-100, 127), (127, -126)):
        xs, ws = np.full((kb, m), 2.0 ** a), np.full((kb, n) if rows == 1 else (nb, kb), 2.0 ** b)
        want = (x @ w.T) * 2.0 ** (a + b)
        xb, wb = blocks_of(asg, x, xs, 1), blocks_of(asg, w, ws, rows)
        for dtype in (torch.float32, torch.bfloat16):
            assert np.array_equal(asg.fp8_linear(xb, wb, out_dtype=dtype).double().cpu().numpy(), want), (a, b, dtype)
    # zeros from the quantiser have scales of 2^-100: nothing comes of them, whatever the other scale
    zero = asg.fp8_quantize(torch.zeros(m, k, dtype=torch.bfloat16, device="cuda"))
    for b in (-126, -100, 0, 127):
        wb = blocks_of(asg, w, np.full((kb, n) if rows == 1 else (nb, kb), 2.0 ** b), rows)
        for dtype in (torch.float32, torch.bfloat16):
            assert not bool(asg.fp8_linear(zero, wb, out_dtype=dtype).any())
