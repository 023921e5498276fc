"""GPU parity of the operators around the FFN (include/ffn_linear.h) against
their fp64 definitions (oracle/linear_oracle.py).

Bounds. u = 2^-24 is half an fp32 step, b = 2^-8 half a bf16 step (relative).
 * A sum of n fp32 terms, each through at most D additions, is within
   D * 2u * sum|terms| of the exact one, whole steps counted for every
   addition (matrix cores may truncate instead of rounding).
 * The norm: sum of squares D <= 8 * NC + 6 + 16 additions (NC <= 4 chunks a
   thread, the wave's butterfly, 16 waves), mean, eps, reciprocal root and two
   products: y is within (D + 16) * 2u relative of the exact one, then rounded
   once. D + 16 <= 70, so 140 u.
 * Its gradients: dx = rstd (v - h mean(v h)) + dr; each of its parts is within
   140 u of its own size, the mean within 140 u of mean|v h|, and
   dw sums m terms in at most m + 40 additions.
 * Products: K terms in at most K + 2 ceil(K / 128) + 8 additions.
 * A bf16 output of 8-bit blocks besides: the e4m3 matrix instruction aligns
   the products of 8 consecutive k to the largest of them and drops what lies
   13 bits below its leading bit, so each of the other seven loses less than
   2^-13 of it: 7 * 2^-13 * max|product| for every eight. (Shown with products
   that are powers of two: 2^16 + 2^3 comes out exact, 2^16 + 2^2 as 2^16,
   whichever of the eight places they stand in; 2^16 + 2^-7 in different
   eights is exact, as in any fp32 sum.) fp32 outputs are made on the bf16
   instructions and have no such term.
"""
from __future__ import annotations

import sys

import numpy as np
import pytest

from oracle import linear_oracle as L

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
EPS = 1e-6


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def asg(lib):
    return lib


def torch_():
    import torch
    return torch


def dev(a, dtype="bf16"):
    torch = torch_()
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def bits(t):
    torch = torch_()
    return t.view(torch.uint8).cpu().numpy()


def near(got, want, slack, what=""):
    """|got - want| <= slack elementwise; NaN where NaN is wanted."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    ok = ~np.isnan(want)
    over = (np.abs(got - want) - np.broadcast_to(slack, want.shape))[ok]
    assert over.size == 0 or over.max() <= 0, (what, float(over.max()))


def rng(*seed):
    return np.random.default_rng(np.random.SeedSequence([41, *seed]))


# ---------------------------------------------------------------- RMS norm
NORM_SHAPES = [(1, 8), (3, 64), (5, 520), (2, 1032), (7, 2048), (7, 2056), (4, 4096), (1, 4096), (2, 8200), (1, 16384),
               (3, 12296), (300, 256), (130, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,d", NORM_SHAPES)
def test_norm_forward(asg, m, d, dtype):
    say("norm forward", m, d, dtype)
    torch = torch_()
    g = rng(1, m, d)
    x, res = dev(g.normal(0, 3, (m, d)), dtype), dev(g.normal(0, 1, (m, d)), dtype)
    w = dev(g.normal(1, 0.3, d), dtype)
    x[0] = 0                                            # a row of zeros without a residual
    half = B if dtype == "bf16" else U
    y, r = asg.rmsnorm_forward(x, w, eps=EPS)
    assert r is x
    want = L.rmsnorm(f64(x), f64(w), EPS)
    near(f64(y), want, np.abs(want) * (half + 140 * U) + 1e-38, "y")
    y, r = asg.rmsnorm_forward(x, w, residual=res, eps=EPS)
    # the sum itself: one fp32 addition, rounded to the type
    assert np.array_equal(bits(r), bits((x.float() + res.float()).to(x.dtype)))
    want = L.rmsnorm(f64(r), f64(w), EPS)
    near(f64(y), want, np.abs(want) * (half + 140 * U) + 1e-38, "y of the sum")
    q, r2 = asg.rmsnorm_forward(x, w, residual=res, eps=EPS, fp8=True)
    assert np.array_equal(bits(r2), bits(r)) and q.q.dtype == torch.float8_e4m3fn
    check_blocks_near(q, want, np.abs(want) * 140 * U, 1)
    z, _ = asg.rmsnorm_forward(torch.zeros_like(x), w, eps=EPS, fp8=True)
    # zeros: 0 * w is -0 (code 0x80) where w is negative
    assert not (bits(z.q) & 0x7F).any() and bool((z.scale == 2.0 ** -100).all())


def check_blocks_near(t, want, off, rows):
    """Blocks of values within `off` of `want`: the scale within that, the values half a step more."""
    m, k = want.shape
    kb, mb = -(-k // 128), -(-m // rows)
    s = t.scale.cpu().numpy().astype(np.float64)
    s = s.T if rows == 1 else s
    assert s.shape == (mb, kb)
    for i in range(mb):
        for j in range(kb):
            wb = np.abs(want[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128])
            ob = off[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128]
            top = max(wb.max() / 448, 2.0 ** -100)
            assert abs(s[i, j] - top) <= ob.max() / 448 + 4 * U * top, (i, j)
    step = np.repeat(np.repeat(s, rows, 0)[:m], 128, 1)[:, :k]
    back = L.e4m3_values()[bits(t.q).reshape(m, k)] * step
    near(back, want, off + np.maximum(2.0 ** -4 * np.abs(want) * (1 + 1e-5) + 2.0 ** -4 * off, 2.0 ** -10 * step * (1 + 1e-5)), "blocks")


def test_norm_in_place_and_bad_numbers(asg):
    say("norm in place")
    torch = torch_()
    g = rng(2)
    x, res, w = dev(g.normal(0, 1, (6, 512))), dev(g.normal(0, 1, (6, 512))), dev(g.normal(1, .2, 512))
    x[1, 7], x[2, 300], x[3] = float("nan"), float("inf"), 1e30
    y0, r0 = asg.rmsnorm_forward(x, w, residual=res)
    q0, _ = asg.rmsnorm_forward(x, w, residual=res, fp8=True)
    for into in (0, 1):
        a, b = x.clone(), res.clone()
        y, r = asg.rmsnorm_forward(a, w, residual=b, r=(a, b)[into])
        assert r.data_ptr() == (a, b)[into].data_ptr()
        assert np.array_equal(bits(y), bits(y0)) and np.array_equal(bits(r), bits(r0))
    assert bool(y0[1].isnan().all()) and bool(r0[1, 7].isnan()) and bool(y0[2, 300].isnan())
    assert bool(torch.isfinite(y0[[0, 4, 5]]).all())
    v = q0.dequantize()
    assert bool(v[1].isnan().all()) and bool(torch.isfinite(v[[0, 4, 5]]).all())
    # 1e30 squared is past fp32: rstd is 0, as the fp32 definition gives
    assert not bool(y0[3].any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,d", NORM_SHAPES + [(2500, 64), (1030, 2056)])
def test_norm_backward(asg, m, d, dtype):
    say("norm backward", m, d, dtype)
    torch = torch_()
    g = rng(3, m, d)
    r, w = dev(g.normal(0, 2, (m, d)), dtype), dev(g.normal(1, 0.3, d), dtype)
    dy, dr = dev(g.normal(0, 1, (m, d)), dtype), dev(g.normal(0, 1, (m, d)), dtype)
    half = B if dtype == "bf16" else U
    R, W, DY = f64(r), f64(w), f64(dy)
    rstd = 1 / np.sqrt(np.mean(R * R, 1, keepdims=True) + EPS)
    for extra in (None, dr):
        dx, dw = asg.rmsnorm_backward(r, w, dy, dr=extra, eps=EPS)
        wdx, wdw = L.rmsnorm_backward(R, W, DY, None if extra is None else f64(dr), EPS)
        size = rstd * np.abs(DY * W) + np.abs(R) * rstd ** 2 * np.mean(np.abs(DY * W * R) * rstd, 1, keepdims=True)
        size = size + (0 if extra is None else np.abs(f64(dr)))
        near(f64(dx), wdx, 400 * U * size + half * np.abs(wdx), "dx")
        near(f64(dw), wdw, ((m + 40) * 2 + 140) * U * np.sum(np.abs(DY * R * rstd), 0), "dw")
    acc = torch.ones(d, dtype=torch.float32, device="cuda")
    into = dy.clone()
    dx2, dw2 = asg.rmsnorm_backward(r, w, into, dr=dr, eps=EPS, dx=into, dw=acc, accumulate=True)
    assert dx2.data_ptr() == into.data_ptr() and np.array_equal(bits(dx2), bits(dx))
    near(f64(dw2), wdw + 1, ((m + 41) * 2 + 140) * U * (1 + np.sum(np.abs(DY * R * rstd), 0)), "dw added to")
    again = asg.rmsnorm_backward(r, w, dy, dr=dr, eps=EPS)
    assert np.array_equal(bits(again[0]), bits(dx)) and np.array_equal(bits(again[1]), bits(dw))


# ---------------------------------------------------------------- 8-bit blocks
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("e,m,k", [(0, 1, 16), (0, 3, 128), (0, 16, 144), (0, 130, 272), (0, 129, 4096), (3, 200, 304),
                                   (2, 1, 2048), (0, 257, 128)])
def test_quantize(asg, e, m, k, rows, dtype):
    say("quantize", e, m, k, rows, dtype)
    g = rng(4, m, k, rows)
    x = g.normal(0, 1, (max(e, 1), m, k)) * np.exp(g.normal(0, 3, (max(e, 1), m, 1)))
    x[0, 0, :16] = 0
    if m > 2:
        x[-1, 2, 5], x[-1, 1, k - 1] = np.nan, -np.inf
        x[-1, 0] = 1e-42
    t = dev(x if e else x[0], dtype)
    one = asg.fp8_quantize(t, block_rows=rows)
    both = asg.fp8_quantize(t, block_rows=rows, transposed=True)
    assert np.array_equal(bits(one.q), bits(both[0].q)) and np.array_equal(bits(one.scale), bits(both[0].scale))
    mt = -(-m // 16) * 16
    X = t.float().cpu().numpy().reshape(max(e, 1), m, k)
    for i in range(max(e, 1)):
        pick = (lambda v: v[i]) if e else (lambda v: v)
        codes, scales = L.blocks(X[i], rows)
        # bit for bit: scale, reciprocal, product and rounding are all defined
        got = pick(one.scale).cpu().numpy()
        assert np.array_equal(got.T if rows == 1 else got, scales, equal_nan=True)
        same_codes(pick(one.q), codes)
        full = np.zeros((k, mt), np.float32)
        full[:, :m] = X[i].T
        codes, scales = L.blocks(full, rows)
        got = pick(both[1].scale).cpu().numpy()
        assert np.array_equal(got.T if rows == 1 else got, scales, equal_nan=True)
        same_codes(pick(both[1].q), codes)


def same_codes(q, want):
    got = bits(q).reshape(want.shape)
    nan = (want & 0x7F) == 0x7F                          # a NaN's sign says nothing
    assert np.array_equal(nan, (got & 0x7F) == 0x7F)
    assert np.array_equal(got[~nan], want[~nan])


# ---------------------------------------------------------------- product of 8-bit blocks
def fp8(asg, values, rows):
    """Blocks made by the oracle, on the GPU, and what they stand for."""
    torch = torch_()
    values = np.asarray(values, np.float32)
    lead = values.shape[:-2]
    parts = [L.blocks(v, rows) for v in values.reshape(-1, *values.shape[-2:])]
    q = np.stack([p[0] for p in parts]).reshape(values.shape)
    s = np.stack([p[1].T if rows == 1 else p[1] for p in parts])
    s = s.reshape(*lead, *s.shape[1:])
    t = asg.Fp8Tensor(torch.from_numpy(q).cuda().view(torch.float8_e4m3fn), torch.from_numpy(np.ascontiguousarray(s)).cuda(), rows)
    back = np.stack([L.values(*p, rows) for p in parts]).reshape(values.shape)
    return t, back


def eights(x, w):
    """The largest product of each 8 consecutive k, summed over them: [m, n]."""
    k = x.shape[1]
    pad = ((0, 0), (0, -k % 8))
    a, b = np.abs(np.pad(x, pad)).reshape(len(x), -1, 8), np.abs(np.pad(w, pad)).reshape(len(w), -1, 8)
    total = np.zeros((len(x), len(w)))
    for i in range(a.shape[1]):
        total += np.max(a[:, None, i] * b[None, :, i], -1)
    return total


def product_slack(x, w, out):
    """Bound of one product's error (module docstring); x, w as they are multiplied."""
    k = x.shape[-1]
    size = np.abs(x) @ np.abs(w).T
    d = k + 2 * -(-k // 128) + 8
    return 2 * U * d * size + (B if out == "bf16" else U) * np.abs(x @ w.T) * (1 + 2 * U * d) + 1e-38


FP8_SHAPES = [(1, 64, 128), (1, 1, 16), (1, 4096, 2048), (2, 77, 144), (5, 130, 1008), (16, 257, 512), (17, 256, 4096),
              (33, 64, 272), (64, 300, 1024), (65, 512, 640), (100, 128, 896), (128, 128, 128), (129, 129, 400),
              (250, 520, 768), (300, 1030, 384), (513, 264, 256), (700, 260, 2064),
              # the contraction in slices, with a ragged end, for every size of tile
              (3, 40, 8208), (24, 96, 8208), (40, 130, 8208), (200, 256, 8192), (300, 100, 6160)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("m,n,k", FP8_SHAPES)
def test_fp8_linear(asg, m, n, k, rows, out):
    say("fp8 linear", m, n, k, rows, out)
    torch = torch_()
    g = rng(5, m, n, k, rows)
    x, X = fp8(asg, g.normal(0, 1, (m, k)) * np.exp(g.normal(0, 1, (m, 1))), 1)
    w, W = fp8(asg, g.normal(0, k ** -0.5, (n, k)) * np.exp(g.normal(0, 1, (n, 1))), rows)
    y = asg.fp8_linear(x, w, out_dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    slack = product_slack(X, W, out) + (7 * 2.0 ** -13 * eights(X, W) if out == "bf16" else 0)
    near(f64(y), X @ W.T, slack, "y")
    if out == "f32":
        acc = torch.full((m, n), 2.0, device="cuda")
        y2 = asg.fp8_linear(x, w, y=acc, accumulate=True)
        assert y2.data_ptr() == acc.data_ptr()
        near(f64(y2), X @ W.T + 2, slack + 2 * U * (2 + np.abs(X @ W.T)), "added to")
    again = asg.fp8_linear(x, w, out_dtype=y.dtype)
    assert np.array_equal(bits(again), bits(y))


EXPERTS = [
    ([0, 3, 3, 10], 10, 96, 256), ([0, 0, 1], 1, 64, 144), ([2, 5, 9], 12, 77, 400), ([0, 40, 41, 41, 170], 170, 264, 512),
    ([0, 16, 48, 112, 120], 120, 128, 1024), ([5, 5, 5], 9, 64, 128), ([0, 300, 301, 700], 710, 300, 384),
    ([0, 1, 2, 3, 4, 5, 6, 7, 8], 8, 512, 2048), ([0, 129, 129, 130], 130, 520, 272), ([0, 30, 70], 80, 72, 8208),
    ([0, 200, 200, 500], 500, 136, 6160)]
WIDE = [sorted(int(v) for v in rng(6).integers(0, 512, 257)), 512, 48, 144]


@pytest.mark.parametrize("off,m,n,k", EXPERTS + [WIDE], ids=lambda v: f"e{len(v) - 1}" if isinstance(v, list) else str(v))
def test_fp8_linear_experts(asg, off, m, n, k):
    say("fp8 experts", len(off) - 1, m, n, k)
    torch = torch_()
    g = rng(7, m, n, k)
    x, X = fp8(asg, g.normal(0, 1, (m, k)), 1)
    w, W = fp8(asg, g.normal(0, k ** -0.5, (len(off) - 1, n, k)), 128)
    y0 = dev(g.normal(0, 1, (m, n)), "f32")
    y = asg.fp8_linear(x, w, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), y=y0.clone())
    want, slack = f64(y0), np.zeros((m, n))
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        want[a:b] = X[a:b] @ W[e].T
        slack[a:b] = product_slack(X[a:b], W[e], "f32")
    near(f64(y), want, slack, "experts")                 # rows of no expert: as they were


def test_fp8_linear_keeps_bad_blocks_apart(asg):
    say("fp8 bad blocks")
    g = rng(8)
    for m in (4, 40, 300):
        xv, wv = g.normal(0, 1, (m, 512)), g.normal(0, 1, (200, 512))
        xv[2, 300], xv[0, 17], wv[140, 3] = np.nan, np.inf, np.nan
        x, X = fp8(asg, xv, 1)
        for rows in (1, 128):
            w, W = fp8(asg, wv, rows)
            y = f64(asg.fp8_linear(x, w))
            bad = np.zeros((m, 200), bool)
            bad[[0, 2]] = True
            bad[:, 140 if rows == 1 else slice(128, 200)] = True
            assert np.array_equal(np.isnan(y), bad)


# ---------------------------------------------------------------- products by expert
GROUPED = [
    ([0, 3, 3, 10], 10, 96, 256), ([0, 0, 1], 1, 64, 136), ([2, 5, 9], 12, 72, 400), ([0, 40, 41, 41, 170], 170, 264, 512),
    ([0, 16, 48, 112, 120], 120, 128, 1024), ([5, 5, 5], 9, 64, 128), ([0, 300, 301, 700], 710, 304, 384), ([0, 1], 1, 8, 8),
    ([0, 1, 2, 3, 4, 5, 6, 7, 8], 8, 512, 2048), ([0, 129, 129, 130], 130, 520, 264), ([0, 260, 520], 520, 512, 512),
    ([0, 5, 20], 24, 72, 8200), ([0, 30, 70], 80, 72, 4104), ([0, 200, 200, 500], 500, 4104, 136), ([3, 4, 400], 401, 2056, 72),
    (WIDE[0], 512, 48, 144)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("off,m,n,k", GROUPED, ids=lambda v: f"e{len(v) - 1}" if isinstance(v, list) else str(v))
def test_grouped_forward(asg, off, m, n, k, out):
    say("grouped forward", len(off) - 1, m, n, k, out)
    torch = torch_()
    g = rng(9, m, n, k)
    x, w = dev(g.normal(0, 1, (m, k))), dev(g.normal(0, k ** -0.5, (len(off) - 1, n, k)))
    y0 = dev(g.normal(0, 1, (m, n)), out)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    y = asg.grouped_forward(x, w, o, y=y0.clone())
    want = L.grouped(f64(x), f64(w), off, f64(y0))
    slack = np.zeros((m, n))
    for e in range(len(off) - 1):
        slack[off[e]:off[e + 1]] = product_slack(f64(x)[off[e]:off[e + 1]], f64(w[e]), out)
    near(f64(y), want, slack, "y")
    assert np.array_equal(bits(asg.grouped_forward(x, w, o, y=y0.clone())), bits(y))


@pytest.mark.parametrize("off,m,n,k", GROUPED, ids=lambda v: f"e{len(v) - 1}" if isinstance(v, list) else str(v))
def test_grouped_backward(asg, off, m, n, k):
    say("grouped backward", len(off) - 1, m, n, k)
    torch = torch_()
    g = rng(10, m, n, k)
    e_n = len(off) - 1
    x, w = dev(g.normal(0, 1, (m, k))), dev(g.normal(0, k ** -0.5, (e_n, n, k)))
    dy, dx0 = dev(g.normal(0, 1, (m, n))), dev(g.normal(0, 1, (m, k)))
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    dx, dw = asg.grouped_backward(x, w, dy, o, dx=dx0.clone())
    wdx, wdw = L.grouped_backward(f64(x), f64(w), f64(dy), off, f64(dx0))
    sdx, sdw = np.zeros((m, k)), np.zeros((e_n, n, k))
    for e in range(e_n):
        a, b = off[e], off[e + 1]
        if b > a:
            sdx[a:b] = product_slack(f64(dy)[a:b], f64(w[e]).T, "bf16")
            sdw[e] = product_slack(f64(dy)[a:b].T, f64(x)[a:b].T, "f32")
    near(f64(dx), wdx, sdx, "dx")
    near(f64(dw), wdw, sdw, "dw")                        # an expert without rows: exact zeros
    acc = torch.full((e_n, n, k), 0.5, device="cuda")
    dx2, dw2 = asg.grouped_backward(x, w, dy, o, dx=dx0.clone(), dw=acc, accumulate=True)
    assert np.array_equal(bits(dx2), bits(dx))
    near(f64(dw2), wdw + 0.5, sdw + 2 * U * (0.5 + np.abs(wdw)), "dw added to")


def test_offsets_out_of_range_stay_inside(asg):
    say("offsets out of range")
    torch = torch_()
    g = rng(11)
    x, w = dev(g.normal(0, 1, (20, 128))), dev(g.normal(0, 1, (3, 64, 128)))
    y0, dy = dev(g.normal(0, 1, (20, 64))), dev(g.normal(0, 1, (20, 64)))
    for wild, same in (([-5, 7, 7, 99], [0, 7, 7, 20]), ([4, 2, 9, 9], [4, 4, 9, 9]), ([0, 12, 5, 20], [0, 12, 12, 20]), ([30, 40, 50, 60], [20] * 4),
                       ([-2 ** 31, 3, 2 ** 31 - 1, -1], [0, 3, 20, 20])):
        a, b = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (wild, same))
        assert np.array_equal(bits(asg.grouped_forward(x, w, a, y=y0.clone())), bits(asg.grouped_forward(x, w, b, y=y0.clone())))
        p = asg.grouped_backward(x, w, dy, a, dx=x.clone())
        q = asg.grouped_backward(x, w, dy, b, dx=x.clone())
        assert np.array_equal(bits(p[0]), bits(q[0])) and np.array_equal(bits(p[1]), bits(q[1]))


def test_wild_offsets_of_many_experts(asg):
    say("wild offsets, many experts")
    torch = torch_()
    g = rng(15)
    for m in (200, 3000):
        x, w = dev(g.normal(0, 1, (m, 64))), dev(g.normal(0, 1, (256, 16, 64)))
        wild = g.integers(-50, m + 400, 257)
        wild[::2], wild[100] = 0, 2 ** 31 - 1
        same = np.maximum.accumulate(np.clip(wild, 0, m))
        y0, dy = dev(g.normal(0, 1, (m, 16))), dev(g.normal(0, 1, (m, 16)))
        a, b = (torch.from_numpy(v.astype(np.int32)).cuda() for v in (wild, same))
        assert np.array_equal(bits(asg.grouped_forward(x, w, a, y=y0.clone())), bits(asg.grouped_forward(x, w, b, y=y0.clone())))
        p, q = (asg.grouped_backward(x, w, dy, o, dx=x.clone()) for o in (a, b))
        assert np.array_equal(bits(p[0]), bits(q[0])) and np.array_equal(bits(p[1]), bits(q[1]))
        want = L.grouped(f64(x), f64(w), same, f64(y0))
        got = f64(asg.grouped_forward(x, w, b, y=y0.clone()))
        near(got, want, 2 * U * 74 * 64 * 16 + B * np.abs(want) * (1 + 1e-4), "y")


def test_bad_numbers_stay_in_their_rows(asg):
    say("grouped bad numbers")
    torch = torch_()
    g = rng(12)
    for m in (24, 300):
        off = [0, m // 2, m]
        x, w = g.normal(0, 1, (m, 200)), g.normal(0, 1, (2, 72, 200))
        x[3, 50], x[m - 1, 199], w[1, 70, 0] = np.nan, np.inf, np.nan
        xt, wt, o = dev(x), dev(w), torch.tensor(off, dtype=torch.int32, device="cuda")
        y = f64(asg.grouped_forward(xt, wt, o))
        bad = np.zeros((m, 72), bool)
        bad[3], bad[m - 1], bad[m // 2:, 70] = True, True, True
        assert np.array_equal(~np.isfinite(y), bad)
        dx, dw = asg.grouped_backward(xt, wt, torch.ones(m, 72, dtype=torch.bfloat16, device="cuda"), o)
        assert np.array_equal(~np.isfinite(f64(dx)), np.isin(np.arange(m)[:, None], np.arange(m // 2, m)) & (np.arange(200) == 0))
        bad = np.zeros((2, 72, 200), bool)
        bad[0, :, 50], bad[1, :, 199] = True, True
        assert np.array_equal(~np.isfinite(f64(dw)), bad)


def test_calls_without_rows(asg):
    say("no rows")
    torch = torch_()
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    y, r = asg.rmsnorm_forward(e(0, 64), e(64), fp8=True)
    assert y.q.shape == (0, 64) and y.scale.shape == (1, 0)
    dx, dw = asg.rmsnorm_backward(e(0, 64), e(64), e(0, 64), dw=torch.ones(64, device="cuda"))
    assert dx.shape == (0, 64) and not bool(dw.any())
    q, qt = asg.fp8_quantize(e(0, 64), transposed=True)
    assert q.q.shape == (0, 64) and qt.q.shape == (64, 0)
    w = asg.fp8_quantize(torch.ones(48, 64, dtype=torch.bfloat16, device="cuda"), block_rows=128)
    assert asg.fp8_linear(q, w).shape == (0, 48)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert asg.grouped_forward(e(0, 64), e(2, 48, 64), off).shape == (0, 48)
    dx, dw = asg.grouped_backward(e(0, 64), e(2, 48, 64), e(0, 48), off, dw=torch.ones(2, 48, 64, device="cuda"))
    assert dx.shape == (0, 64) and not bool(dw.any())


def test_binding_refuses(asg):
    say("refusals")
    torch = torch_()
    x = torch.zeros(8, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(x=x.half()), dict(x=x[:, ::2]), dict(w=w.float()), dict(w=w[:64]), dict(residual=x[:4]),
                dict(residual=x.cpu()), dict(y=x.float()), dict(r=x[:2])):
        with pytest.raises(ValueError):
            kw = dict(dict(x=x, w=w), **bad)
            asg.rmsnorm_forward(kw.pop("x"), kw.pop("w"), **kw)
    q, q128 = asg.fp8_quantize(x), asg.fp8_quantize(x, block_rows=128)
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    for a, b, kw in ((x, q, {}), (q128, q, {}), (q, asg.Fp8Tensor(q.q, q128.scale, 1), {}), (q, q, dict(offsets=off)),
                     (q, q128, dict(offsets=off)), (q, q, dict(accumulate=True)), (q, q, dict(out_dtype=torch.float16)),
                     (q, q, dict(y=torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda"), accumulate=True)),
                     (q, asg.Fp8Tensor(q.q, q.scale, 3), {})):
        with pytest.raises(ValueError):
            asg.fp8_linear(a, b, **kw)
    with pytest.raises(ValueError):
        asg.fp8_quantize(x, block_rows=64)
    with pytest.raises(asg.FFNError):
        asg.fp8_quantize(torch.zeros(4, 24, dtype=torch.bfloat16, device="cuda"))
    we = torch.zeros(2, 64, 128, dtype=torch.bfloat16, device="cuda")
    o3 = torch.zeros(3, dtype=torch.int32, device="cuda")
    for a, b, o in ((x, we, off), (x, we, o3.long()), (x, we[:, :, :64], o3), (x.float(), we, o3)):
        with pytest.raises(ValueError):
            asg.grouped_forward(a, b, o)
    # unaligned: a row view of an odd width starts between 16-byte boundaries
    odd = torch.zeros(129 * 8, dtype=torch.bfloat16, device="cuda")[1:1 + 8 * 128].view(8, 128)
    with pytest.raises(asg.FFNError):
        asg.rmsnorm_forward(odd, w)


def test_workspaces_given_by_hand(asg):
    say("workspaces")
    torch = torch_()
    from activation_sparse_gated_amd import _lib
    lib, g = _lib.load(), rng(16)
    byte = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    m, n, k = 48, 128, 8192
    x, w = dev(g.normal(0, 1, (m, k))), dev(g.normal(0, k ** -0.5, (2, n, k)))
    off = torch.tensor([0, 17, m], dtype=torch.int32, device="cuda")
    need = lib.ffn_grouped_forward_workspace_bytes(m, n, k, 2)
    assert need > 0                                      # a shape that is cut along k
    want = L.grouped(f64(x), f64(w), [0, 17, m], np.zeros((m, n)))
    slack = np.concatenate([product_slack(f64(x)[a:b], f64(w[e]), "bf16") for e, (a, b) in enumerate(((0, 17), (17, m)))])
    own = asg.grouped_forward(x, w, off)
    full = asg.grouped_forward(x, w, off, workspace=byte(need))
    assert np.array_equal(bits(full), bits(own))
    for small in (byte(16), byte(need - 16)):            # too small: not used, not written
        small.fill_(0x5A)
        near(f64(asg.grouped_forward(x, w, off, workspace=small)), want, slack, "whole sums")
        assert bool((small == 0x5A).all())
    near(f64(own), want, slack, "slices")
    with pytest.raises(asg.FFNError):
        asg.grouped_forward(x, w, off, workspace=byte(need + 64)[8:])
    with pytest.raises(ValueError):
        asg.grouped_forward(x, w, off, workspace=torch.empty(4, device="cuda"))
    with pytest.raises(asg.FFNError):
        asg.rmsnorm_backward(x, dev(g.normal(1, .1, k)), x, workspace=byte(64))
    # one workspace, one call after the other on the same stream
    both = byte(max(need, lib.ffn_rmsnorm_backward_workspace_bytes(m, k)))
    a = asg.grouped_forward(x, w, off, workspace=both)
    asg.rmsnorm_backward(x, dev(g.normal(1, .1, k)), x, workspace=both)
    b = asg.grouped_forward(x, w, off, workspace=both)
    assert np.array_equal(bits(a), bits(own)) and np.array_equal(bits(b), bits(own))


# ---------------------------------------------------------------- together
def block_step(asg, s):
    """One training step of an 8-bit gated block's products with a residual
    stream, and an expert layer behind it: every operator, as used together."""
    a, r = asg.rmsnorm_forward(s["x"], s["w"], residual=s["res"], fp8=True)
    wq, wt = asg.fp8_quantize(s["up"], block_rows=128, transposed=True)
    u = asg.fp8_linear(a, wq)
    y = asg.grouped_forward(u, s["experts"], s["off"])
    # backward of <g, y>
    du, dexp = asg.grouped_backward(u, s["experts"], s["g"], s["off"])
    dq, dqt = asg.fp8_quantize(du, transposed=True)
    da = asg.fp8_linear(dq, wt)
    n, _ = asg.rmsnorm_forward(r, s["w"])
    _, at = asg.fp8_quantize(n, transposed=True)
    dup = asg.fp8_linear(dqt, at, out_dtype=s["f32"])
    dx, dw = asg.rmsnorm_backward(r, s["w"], da, dr=s["dr"])
    return y, dexp, dup, dx, dw


def block_state(m, seed):
    torch = torch_()
    g = rng(13, m, seed)
    d, f, o = 256, 384, 128
    # the experts' rows cover the batch: the first expert has none
    off = [0, 0, m // 3, m]
    return dict(x=dev(g.normal(0, 1, (m, d))), res=dev(g.normal(0, 1, (m, d))), w=dev(g.normal(1, .2, d)),
                up=dev(g.normal(0, d ** -0.5, (f, d))), experts=dev(g.normal(0, f ** -0.5, (3, o, f))),
                off=torch.tensor(off, dtype=torch.int32, device="cuda"), offs=off, g=dev(g.normal(0, 1, (m, o))),
                dr=dev(g.normal(0, 1, (m, d))), f32=torch.float32)


def block_exact(s):
    x = f64(s["x"]) + f64(s["res"])
    r = f64(dev(x))
    w, up, ex, gr, off = f64(s["w"]), f64(s["up"]), f64(s["experts"]), f64(s["g"]), s["offs"]
    a = L.rmsnorm(r, w, EPS)
    u = a @ up.T
    y = L.grouped(u, ex, off, np.zeros((len(x), ex.shape[1])))
    du, dexp = L.grouped_backward(u, ex, gr, off, np.zeros_like(u))
    dx, dw = L.rmsnorm_backward(r, w, du @ up, f64(s["dr"]), EPS)
    return y, dexp, du.T @ a, dx, dw


@pytest.mark.parametrize("m", [1, 6, 100, 600])
def test_block_step(asg, m):
    say("block step", m)
    s = block_state(m, 0)
    # 8-bit values: half a step of 2^-4 relative on both sides of a product is
    # at most 2^-3, in quadrature over hundreds of terms far less; two or three
    # of them in a row stay under 0.1 in the 2-norm
    for got, want, name in zip(block_step(asg, s), block_exact(s), ("y", "dexperts", "dup", "dx", "dw")):
        got = f64(got)
        off = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert got.shape == want.shape and off < 0.1, (name, off)


def test_block_step_captured(asg):
    say("captured")
    torch = torch_()
    s, other = block_state(70, 0), block_state(70, 1)
    want = [[t.clone() for t in block_step(asg, v)] for v in (s, other)]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(stream):
        block_step(asg, s)
    torch.cuda.synchronize()
    for _ in range(2):                                   # two graphs of the same step
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = block_step(asg, s)
        graphs.append((graph, out))
    first = {k: v.clone() for k, v in s.items() if hasattr(v, "clone")}
    for n in range(4):
        for k in first:
            s[k].copy_((first, other)[n % 2][k])
        for graph, out in graphs:
            for t in out:
                t.fill_(float("nan"))
        for graph, _ in graphs:
            graph.replay()
        eager = block_step(asg, s)
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, b, c in zip(out, want[n % 2], eager):
                assert np.array_equal(bits(a), bits(b)) and np.array_equal(bits(c), bits(b))


def test_two_streams_at_once(asg):
    say("two streams")
    torch = torch_()
    states = [block_state(300, 2), block_state(90, 3)]
    want = [[t.clone() for t in block_step(asg, s)] for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(block_step(asg, states[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for out in got[i]:
            for a, b in zip(out, want[i]):
                assert np.array_equal(bits(a), bits(b))
    # a stream passed by hand
    y = asg.fp8_linear(*(asg.fp8_quantize(states[0][k], stream=streams[0]) for k in ("x", "res")), stream=streams[0])
    streams[0].synchronize()
    ref = asg.fp8_linear(asg.fp8_quantize(states[0]["x"]), asg.fp8_quantize(states[0]["res"]))
    assert np.array_equal(bits(y), bits(ref))


def test_outputs_stay_in_their_buffers(asg):
    say("guards")
    torch = torch_()

    def guarded(n, dtype):
        t = torch.full((n * dtype.itemsize + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        return t, t[256:256 + n * dtype.itemsize].view(dtype)

    g = rng(14)
    bufs = []

    def out(*shape, dtype=torch.bfloat16):
        n = int(np.prod(shape))
        whole, t = guarded(n, dtype)
        bufs.append(whole)
        return t.view(*shape)

    for m, d in ((3, 264), (130, 136)):
        x, w, dy = dev(g.normal(0, 1, (m, d))), dev(g.normal(0, 1, d)), dev(g.normal(0, 1, (m, d)))
        asg.rmsnorm_forward(x, w, residual=dy, r=out(m, d), y=out(m, d))
        f8 = torch.float8_e4m3fn
        kb, mb, mt = -(-d // 128), -(-m // 128), -(-m // 16) * 16
        asg.rmsnorm_forward(x, w, fp8=True, y=asg.Fp8Tensor(out(m, d, dtype=f8), out(kb, m, dtype=torch.float32), 1))
        asg.rmsnorm_backward(x, w, dy, dx=out(m, d), dw=out(d, dtype=torch.float32))
        k = d // 16 * 16
        xk = x[:, :k].contiguous()
        kb = -(-k // 128)
        for rows in (1, 128):
            a = asg.Fp8Tensor(out(m, k, dtype=f8), out(*((kb, m) if rows == 1 else (mb, kb)), dtype=torch.float32), rows)
            b = asg.Fp8Tensor(out(k, mt, dtype=f8), out(*((mb, k) if rows == 1 else (kb, mb)), dtype=torch.float32), rows)
            asg.fp8_quantize(xk, block_rows=rows, transposed=True, out=a, out_t=b)
        a = asg.fp8_quantize(xk)
        for n in (1, 77, 264):
            wq = asg.fp8_quantize(dev(g.normal(0, 1, (n, k))))
            asg.fp8_linear(a, wq, y=out(m, n))
            asg.fp8_linear(a, wq, y=out(m, n, dtype=torch.float32))
        we, off = dev(g.normal(0, 1, (2, 72, d))), torch.tensor([0, 2, m], dtype=torch.int32, device="cuda")
        asg.grouped_forward(x, we, off, y=out(m, 72))
        asg.grouped_backward(x, we, dev(g.normal(0, 1, (m, 72))), off, dx=out(m, d), dw=out(2, 72, d, dtype=torch.float32))
    torch.cuda.synchronize()
    for t in bufs:
        assert bool((t[:256] == 0xA5).all()) and bool((t[-256:] == 0xA5).all())


# ---------------------------------------------------------------- past 2^31 elements
def test_norm_and_blocks_past_32_bits(asg):
    say("large norm")
    torch = torch_()
    m, d = 135_000, 16384                                # 2.2e9 elements
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(m, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w = torch.empty(d, dtype=torch.bfloat16, device="cuda").normal_(1, 0.2, generator=gen)
    rows = [0, 1, 131_072, m - 2, m - 1]
    y, r = asg.rmsnorm_forward(x, w, residual=x)
    q, _ = asg.rmsnorm_forward(x, w, residual=x, fp8=True)
    want = L.rmsnorm(f64(r[rows]), f64(w), EPS)
    near(f64(y[rows]), want, np.abs(want) * (B + 140 * U), "y")
    part = asg.Fp8Tensor(q.q[rows].contiguous(), q.scale[:, rows].contiguous(), 1)
    check_blocks_near(part, want, np.abs(want) * 140 * U, 1)
    del y, r, q
    dx, dw = asg.rmsnorm_backward(x, w, x, dr=x)
    wdx, _ = L.rmsnorm_backward(f64(x[rows]), f64(w), f64(x[rows]), f64(x[rows]), EPS)
    near(f64(dx[rows]), wdx, 400 * U * 3 * (1 + np.abs(f64(x[rows])) * 4) + B * np.abs(wdx), "dx")
    del dx
    a, b = asg.fp8_quantize(x, transposed=True)
    codes, scales = L.blocks(x[rows].float().cpu().numpy(), 1)
    same_codes(a.q[rows].contiguous(), codes)
    assert np.array_equal(a.scale[:, rows].cpu().numpy().T, scales)
    cols = [0, 8191, d - 1]
    tail = m // 128 * 128                                # the last, partial block of the transposed rows
    codes, scales = L.blocks(x[tail:][:, cols].float().cpu().numpy().T.copy(), 1)
    same_codes(b.q[cols][:, tail:m].contiguous(), codes)
    assert np.array_equal(b.scale[-1, cols].cpu().numpy(), scales[:, 0])


def test_products_past_32_bits(asg):
    say("large products")
    torch = torch_()
    gen = torch.Generator(device="cuda").manual_seed(4)
    normal = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)  # noqa: E731
    m, k, n = 532_000, 4096, 64                          # x: 2.2e9 elements
    x, w = normal(m, k), normal(2, n, k)
    off = torch.tensor([0, 7, m], dtype=torch.int32, device="cuda")
    y = asg.grouped_forward(x, w, off)
    rows = [0, 7, 524_287, 524_288, m - 1]
    X, W = f64(x[rows]), f64(w)
    for i, t in enumerate(rows):
        e = int(t >= 7)
        near(f64(y[t]), X[i] @ W[e].T, product_slack(X[i:i + 1], W[e], "bf16")[0], t)
    q, wq = asg.fp8_quantize(x), asg.fp8_quantize(w[0].contiguous(), block_rows=128)
    v = asg.Fp8Tensor(q.q[rows].contiguous(), q.scale[:, rows].contiguous(), 1).dequantize().double().cpu().numpy()
    wv = wq.dequantize().double().cpu().numpy()
    y = asg.fp8_linear(q, wq)
    near(f64(y[rows]), v @ wv.T, product_slack(v, wv, "bf16") + 7 * 2.0 ** -13 * eights(v, wv), "8-bit")
    del x, y, q
    # 9 x 16384 x 16384 gradients: 2.4e9 elements, and as many weights
    g, n, k, m = 9, 16384, 16384, 40
    w, x, dy = normal(g, n, k), normal(m, k), normal(m, n)
    off = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, 8, m], dtype=torch.int32, device="cuda")
    dx, dw = asg.grouped_backward(x, w, dy, off)
    X, D = f64(x), f64(dy)
    near(f64(dw[8, -3:]), D[8:, -3:].T @ X[8:], product_slack(D[8:, -3:].T, X[8:].T, "f32"), "dw")
    near(f64(dw[7, :2]), np.outer(D[7, :2], X[7]), 4 * U * np.abs(np.outer(D[7, :2], X[7])), "dw of one row")
    near(f64(dx[8:, -5:]), D[8:] @ f64(w[8, :, -5:]), product_slack(D[8:], f64(w[8, :, -5:]).T, "bf16"), "dx")
    y = asg.grouped_forward(x, w, off)
    near(f64(y[8:, -5:]), X[8:] @ f64(w[8, -5:]).T, product_slack(X[8:], f64(w[8, -5:]), "bf16"), "y")


def test_products_of_operands_of_4_gib(asg):
    # the bytes from the first tile's first row to the operand's last one are 2^32 and seven rows
    say("operands of 4 GiB")
    torch = torch_()
    gen = torch.Generator(device="cuda").manual_seed(5)
    normal = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)  # noqa: E731
    big, few, k = 2 ** 18 + 8, 64, 8192
    a, b = normal(big, k), normal(few, k)
    A, Bv = f64(a[:256]), f64(b)
    want, slack = A @ Bv.T, product_slack(A, Bv, "bf16")
    off = lambda m: torch.tensor([0, m], dtype=torch.int32, device="cuda")  # noqa: E731
    y = asg.grouped_forward(a, b[None], off(big))
    near(f64(y[:256]), want, slack, "rows")
    y = asg.grouped_forward(b, a[None], off(few))
    near(f64(y[:, :256]), want.T, slack.T, "columns")
    dx, _ = asg.grouped_backward(normal(big, few), b.t().contiguous()[None], a, off(big))
    near(f64(dx[:256]), want, slack, "dx")
    del a, y, dx
    k *= 2
    a, b = asg.fp8_quantize(normal(big, k)), asg.fp8_quantize(normal(few, k), block_rows=128)
    A, Bv = (t.double().cpu().numpy() for t in (asg.Fp8Tensor(a.q[:256], a.scale[:, :256], 1).dequantize(), b.dequantize()))
    y = asg.fp8_linear(a, b)
    near(f64(y[:256]), A @ Bv.T, product_slack(A, Bv, "bf16") + 7 * 2.0 ** -13 * eights(A, Bv), "8-bit rows")


def test_many_rows(asg):
    # more rows than a grid of one dimension holds, more workgroups than one of few-row products may have
    say("many rows")
    torch = torch_()
    gen = torch.Generator(device="cuda").manual_seed(6)
    normal = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)  # noqa: E731
    m, d = 2 ** 26 + 5, 8
    x, w = normal(m, d), normal(d)
    y, _ = asg.rmsnorm_forward(x, w)
    rows = [0, 3, 2 ** 25 - 1, 2 ** 25, 2 ** 26 - 1, 2 ** 26, m - 1]
    want = L.rmsnorm(f64(x[rows]), f64(w), EPS)
    near(f64(y[rows]), want, np.abs(want) * (B + 140 * U), "norm")
    del x, y
    g, n, k = 256, 2 ** 19, 16
    m = 2 * g
    x, w = normal(m, k), normal(g, n, k)
    y = asg.grouped_forward(x, w, torch.arange(0, m + 1, 2, dtype=torch.int32, device="cuda"))
    for e in (0, 1, 100, 255):
        X, W = f64(x[2 * e:2 * e + 2]), f64(w[e, -300:])
        near(f64(y[2 * e:2 * e + 2, -300:]), X @ W.T, product_slack(X, W, "bf16"), e)


def test_stream_with_keywords_in_any_order(asg):
    say("stream")
    torch = torch_()
    stream = torch.cuda.Stream()
    x, w = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    stream.wait_stream(torch.cuda.current_stream())
    y, _ = asg.rmsnorm_forward(eps=1e-6, fp8=False, residual=None, w=w, x=x, stream=stream)
    q = asg.fp8_quantize(block_rows=128, x=x, stream=stream)
    with pytest.raises(TypeError):
        asg.fp8_quantize(block_rows=128, stream=stream)
    stream.synchronize()
    assert bool((y == 1).all()) and bool((q.dequantize() == 1).all())
