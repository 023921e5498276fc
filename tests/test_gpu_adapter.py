"""GPU parity of the low-rank adapters (include/ffn_adapter.h) against their fp64
definitions (oracle/experts_oracle.py).

Bounds. u = 2^-24 is half an fp32 step (relative), b = 2^-8 half a bf16 step;
whole steps 2u are counted for every addition (matrix cores may truncate).
 * h = x A^T over k: a matrix instruction adds 32 products at a time, waves and
   slices share the k / 32 of them, so a term goes through at most k / 8 + 80
   additions: e(k) = (k / 8 + 80) 2u of the sum of the terms' sizes.
 * h enters the second product as two bf16 numbers, which lose b^2 = 2^-16 of it
   (three, b^3 = 2^-24, for fp32 outputs); that product has at most r / 16 + 3
   instructions of 32 products and three parts: (3 r + 100) 2u, the scale's
   multiplication among them.
 * The adapters' gradients sum their rows: at most m / 8 + 80 additions, times
   three parts, with h or dh as above in three parts.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import experts_oracle as E
from tests.test_gpu_experts import B, TINY, U, dev, f64, near, rng, say, torch_

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def asg(lib):
    return lib


def order(g, m, groups, kind):
    """(offsets, rows): adapters in any order with rows of none between, or row after row; one adapter without rows."""
    if kind == "rows":
        ids = g.integers(-1, groups, m)
        if groups > 2:
            ids[ids == 1] = 0
        off, rows, _ = E.group(ids, groups)
        return off, rows
    lo, hi = (min(2, m), max(0, m - 3)) if m > 20 else (0, m)
    cuts = np.sort(g.integers(lo, hi + 1, groups - 1))
    off = np.concatenate([[lo], cuts, [hi]]).astype(np.int32)
    if groups > 2:
        off[2] = off[1]
    return off, None


def make(m, n, k, r, groups, kind, *seed):
    g = rng(*seed, m, n, k, r, groups)
    s = dict(x=dev(g.normal(0, 1, (m, k)), "bf16"), a=dev(g.normal(0, k ** -0.5, (groups, r, k)), "bf16"),
             b=dev(g.normal(0, r ** -0.5, (groups, n, r)), "bf16"), dy=dev(g.normal(0, 1, (m, n)), "bf16"))
    s["scales"] = g.uniform(0.5, 2, groups).astype(np.float32)
    s["offsets"], s["rows"] = order(g, m, groups, kind)
    return s, g


def call(s):
    return dict(rows=None if s["rows"] is None else dev(s["rows"]), scales=None if s["scales"] is None else dev(s["scales"]))


def check_forward(asg, s, base, out):
    torch = torch_()
    x, a, b = (f64(s[v]) for v in ("x", "a", "b"))
    m, k, r = len(x), x.shape[1], a.shape[1]
    t = torch.bfloat16 if out == "bf16" else torch.float32
    y = asg.adapter_forward(s["x"], s["a"], s["b"], dev(s["offsets"]), base=base, out_dtype=t, **call(s))
    assert y.dtype == t
    b64 = None if base is None else f64(base)
    want = E.adapter(x, a, b, s["scales"], s["offsets"], s["rows"], b64)
    none = None if base is None else np.abs(b64)
    size = E.adapter(np.abs(x), np.abs(a), np.abs(b), s["scales"], s["offsets"], s["rows"], None)
    lost = B ** (2 if out == "bf16" else 3)
    slack = ((k / 8 + 80) * 2 * U + lost + (3 * r + 100) * 2 * U) * size + 2 * U * (size + (0 if none is None else none))
    near(f64(y), want, slack + (B if out == "bf16" else U) * np.abs(want) * (1 + 1e-3) + TINY, "y")
    return y


# rows, n, k, rank, adapters
SHAPES = [(1, 72, 136, 8, 1), (1, 520, 264, 16, 5), (3, 136, 72, 24, 2), (17, 264, 520, 16, 3), (48, 1032, 2056, 16, 33),
          (16, 8, 8, 8, 2), (130, 136, 264, 40, 7), (33, 2056, 1032, 64, 70), (257, 520, 136, 72, 4), (70, 264, 328, 136, 3),
          (40, 136, 264, 256, 2), (1024, 264, 200, 32, 5), (1030, 392, 264, 16, 9), (2100, 200, 136, 64, 300), (1500, 136, 72, 8, 1024),
          (1111, 72, 136, 128, 3), (1033, 136, 200, 200, 6), (5, 200, 4104, 16, 4),
          # contractions in slices, rows in slices, both
          (700, 264, 2056, 16, 3), (1030, 1048, 1032, 64, 4), (600, 136, 4104, 128, 2), (520, 2056, 264, 200, 3), (4200, 264, 136, 16, 1),
          (2600, 136, 72, 64, 1), (3000, 72, 72, 136, 1), (8500, 72, 136, 24, 5), (2056, 1160, 1096, 32, 1), (90, 1032, 1544, 72, 3),
          (17, 4104, 136, 128, 2)]


@pytest.mark.parametrize("kind", ["rows", "ordered"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(asg, shape, kind):
    say("adapter forward", shape, kind)
    m, n, k, r, groups = shape
    s, g = make(m, n, k, r, groups, kind, 1)
    for out in ("bf16", "f32"):
        base = dev(g.normal(0, 1, (m, n)), out)
        y = check_forward(asg, s, base, out)
        check_forward(asg, s, None, out)
        again = base.clone()                            # in place
        z = asg.adapter_forward(s["x"], s["a"], s["b"], dev(s["offsets"]), base=again, y=again, **call(s))
        assert z is again and torch_().equal(z, y)
    check_forward(asg, dict(s, scales=None), None, "bf16")


def check_backward(asg, s, base, accumulate=False):
    torch = torch_()
    x, a, b, dy = (f64(s[v]) for v in ("x", "a", "b", "dy"))
    (m, k), n, r = x.shape, dy.shape[1], a.shape[1]
    kw = call(s)
    if accumulate:
        g = rng(9, m, n)
        da0, db0 = g.normal(0, 1, a.shape).astype(np.float32), g.normal(0, 1, b.shape).astype(np.float32)
        kw.update(da=dev(da0), db=dev(db0), accumulate=True)
    dx, da, db = asg.adapter_backward(s["x"], s["a"], s["b"], s["dy"], dev(s["offsets"]), base=base, **kw)
    assert dx.dtype == torch.bfloat16 and da.dtype == db.dtype == torch.float32
    b64 = None if base is None else f64(base)
    want = list(E.adapter_backward(x, a, b, s["scales"], dy, s["offsets"], s["rows"], b64))
    size = E.adapter_backward(*(np.abs(v) for v in (x, a, b)), s["scales"], np.abs(dy), s["offsets"], s["rows"], None)
    e = lambda c: (c / 8 + 80) * 2 * U  # noqa: E731
    slack = (e(n) + B ** 2 + (3 * r + 100) * 2 * U) * size[0] + 2 * U * (size[0] + (0 if base is None else np.abs(b64)))
    near(f64(dx), want[0], slack + B * np.abs(want[0]) * (1 + 1e-3) + TINY, "dx")
    rows = 3 * e(m) + B ** 3 + 8 * U
    for i, (got, c) in enumerate(((da, n), (db, k)), 1):
        old = 0 if not accumulate else (da0, db0)[i - 1].astype(np.float64)
        near(f64(got), want[i] + old, (e(c) + rows) * size[i] + 2 * U * (np.abs(old) + size[i]) + TINY, ("dx", "da", "db")[i])
    return dx, da, db


# few rows with long contractions, which take two launches, and many tiles of few rows in one
FEW = [(1, 136, 16392, 16, 1), (48, 264, 5128, 24, 33), (130, 136, 8200, 8, 7), (33, 520, 4104, 64, 70), (1300, 72, 2056, 40, 200),
       (90, 1032, 4104, 32, 3), (5000, 264, 136, 16, 1000), (16, 10248, 136, 8, 1), (300, 2056, 328, 32, 40)]
# many rows of few adapters (tiles of 64), every number of ranks, whole and in slices
MANY = [(8200, 136, 264, 16, 9), (8300, 200, 136, 64, 250), (8192, 200, 200, 200, 6), (2100, 264, 8200, 64, 3),
        (2056, 136, 4104, 128, 20), (9000, 200, 136, 40, 1), (8400, 520, 1032, 8, 200), (8201, 264, 392, 256, 2),
        (8333, 136, 328, 72, 3), (16500, 72, 136, 32, 4), (8450, 264, 136, 128, 100), (4100, 136, 8200, 16, 7),
        (2050, 72, 16392, 24, 64)]


@pytest.mark.parametrize("kind", ["rows", "ordered"])
@pytest.mark.parametrize("shape", FEW + MANY, ids=lambda s: "x".join(map(str, s)))
def test_forward_of_few_and_many_rows(asg, shape, kind):
    say("adapter forward, few and many rows", shape, kind)
    m, n, k, r, groups = shape
    s, g = make(m, n, k, r, groups, kind, 7)
    for out in ("bf16", "f32"):
        base = dev(g.normal(0, 1, (m, n)), out)
        y = check_forward(asg, s, base, out)
        check_forward(asg, dict(s, scales=None), None, out)
        again = base.clone()
        z = asg.adapter_forward(s["x"], s["a"], s["b"], dev(s["offsets"]), base=again, y=again, **call(s))
        assert z is again and torch_().equal(z, y)


@pytest.mark.parametrize("kind", ["rows", "ordered"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(asg, shape, kind):
    say("adapter backward", shape, kind)
    torch = torch_()
    m, n, k, r, groups = shape
    s, g = make(m, n, k, r, groups, kind, 2)
    base = dev(g.normal(0, 1, (m, k)), "bf16")
    dx, da, db = check_backward(asg, s, base)
    check_backward(asg, dict(s, scales=None), None, accumulate=True)
    inputs, off, kw = (s["x"], s["a"], s["b"], s["dy"]), dev(s["offsets"]), call(s)
    for need in ("dx", "da", "db"):                     # one alone is the same
        got = asg.adapter_backward(*inputs, off, base=base if need == "dx" else None,
                                   **{f"need_{v}": v == need for v in ("dx", "da", "db")}, **kw)
        for v, one, all_ in zip(("dx", "da", "db"), got, (dx, da, db)):
            assert one is None if v != need else torch.equal(one, all_)
    again = base.clone()
    assert torch.equal(asg.adapter_backward(*inputs, off, base=again, dx=again, need_da=False, need_db=False, **kw)[0], dx)


@pytest.mark.parametrize("kind", ["rows", "ordered"])
@pytest.mark.parametrize("shape", MANY, ids=lambda s: "x".join(map(str, s)))
def test_backward_of_many_rows(asg, shape, kind):
    say("adapter backward, many rows", shape, kind)
    m, n, k, r, groups = shape
    s, g = make(m, n, k, r, groups, kind, 8)
    check_backward(asg, s, dev(g.normal(0, 1, (m, k)), "bf16"))
    check_backward(asg, dict(s, scales=None), None, accumulate=True)


def test_offsets_and_rows_out_of_range(asg):
    say("adapter offsets")
    torch = torch_()
    for off, rows in (([-5, 4, 2, 99], None), ([3, 3, 3, 3], None), ([0, 9, 30, 2 ** 31 - 1], None), ([7, 1, 1, 12], None),
                      ([0, 5, 9, 16], [3, 1, 99, 2, -4, 15, 0, 2 ** 31 - 1, 4, 5, 6, 7, 8, 9, 10, 11])):
        s, g = make(16, 72, 136, 16, 3, "ordered", 3)
        s["offsets"], s["rows"] = np.array(off, np.int32), None if rows is None else np.array(rows, np.int32)
        base = dev(g.normal(0, 1, (16, 72)), "bf16")
        if rows is None:
            check_forward(asg, s, base, "bf16")
            check_backward(asg, s, None)
        else:                                           # rows that are not named are left as they were
            left = sorted(set(range(16)) - set(rows))
            y = torch.full((16, 72), 9.0, dtype=torch.bfloat16, device="cuda")
            asg.adapter_forward(s["x"], s["a"], s["b"], dev(s["offsets"]), base=base, y=y, **call(s))
            want = E.adapter(f64(s["x"]), f64(s["a"]), f64(s["b"]), s["scales"], off, rows, f64(base))
            want[left] = 9.0
            near(f64(y), want, 2 * B * np.abs(want) + 1e-2, "y")


def test_bad_numbers_stay_in_their_rows(asg):
    # a row of NaN, an infinity, and an adapter of NaN that no row has
    say("adapter bad numbers")
    torch = torch_()
    s, g = make(40, 136, 264, 24, 4, "ordered", 4)
    s["offsets"] = np.array([3, 15, 15, 30, 36], np.int32)
    good = asg.adapter_forward(s["x"], s["a"], s["b"], dev(s["offsets"]), **call(s))
    x, a, b = s["x"].clone(), s["a"].clone(), s["b"].clone()
    x[0], x[5], x[20, 7], x[39] = float("nan"), float("nan"), float("inf"), float("nan")
    a[1], b[1] = float("nan"), float("nan")
    y = asg.adapter_forward(x, a, b, dev(s["offsets"]), **call(s))
    keep = [i for i in range(40) if i not in (5, 20)]
    assert torch.equal(y[keep], good[keep]) and bool(torch.isnan(y[5]).all()) and not bool(torch.isfinite(y[20]).any())
    assert not y[0].any() and not y[39].any()
    dx, da, db = asg.adapter_backward(x, a, b, s["dy"], dev(s["offsets"]), **call(s))
    dx0, da0, db0 = asg.adapter_backward(s["x"], s["a"], s["b"], s["dy"], dev(s["offsets"]), **call(s))
    assert torch.equal(dx, dx0) and torch.equal(da[3], da0[3]) and torch.equal(db[3], db0[3])
    assert not da[1].any() and not db[1].any() and bool(torch.isnan(da[0]).all())


def test_rows_past_2_to_the_31_elements(asg):
    say("adapter large")
    torch = torch_()
    m, n, k, r = 140_000, 16384, 16448, 8               # 2.3e9 elements of x, y and dy
    x = torch.randn(m, k, device="cuda", dtype=torch.bfloat16)
    a, b = (torch.randn(1, *shape, device="cuda", dtype=torch.bfloat16) / 16 for shape in ((r, k), (n, r)))
    off = torch.tensor([3, m - 5], dtype=torch.int32, device="cuda")
    y = asg.adapter_forward(x, a, b, off)
    at = [0, 2, 3, 70_001, m - 70, m - 6, m - 5, m - 1]
    want = E.adapter(f64(x[at]), f64(a), f64(b), None, [2, 6], None, None)
    size = E.adapter(np.abs(f64(x[at])), np.abs(f64(a)), np.abs(f64(b)), None, [2, 6], None, None)
    near(f64(y[at]), want, ((k / 8 + 80 + 3 * r + 101) * 2 * U + B ** 2) * size + B * np.abs(want) * (1 + 1e-3), "y")
    dx, da, _ = asg.adapter_backward(x, a, b, y, off, need_db=False)
    y[3:m - 5] = 0                                      # one row of gradient alone: its outer product
    y[m - 70] = 1.0
    _, da, _ = asg.adapter_backward(x, a, b, y, off, need_dx=False, need_db=False)
    want = E.adapter_backward(f64(x[m - 70:m - 69]), f64(a), f64(b), None, f64(y[m - 70:m - 69]), [0, 1], None, None)[1]
    size = np.abs(f64(b)).sum(1)[:, :, None] * np.abs(f64(x[m - 70]))
    near(f64(da), want, (n / 8 + m / 8 + 200) * 2 * U * size + 1e-30, "da")


def test_same_from_run_to_run(asg):
    say("adapter again")
    torch = torch_()
    s, g = make(1100, 520, 1032, 32, 6, "rows", 5)
    off, kw = dev(s["offsets"]), call(s)
    y = asg.adapter_forward(s["x"], s["a"], s["b"], off, **kw)
    grads = asg.adapter_backward(s["x"], s["a"], s["b"], s["dy"], off, **kw)
    for _ in range(3):
        assert torch.equal(asg.adapter_forward(s["x"], s["a"], s["b"], off, **kw), y)
        assert all(torch.equal(p, q) for p, q in zip(asg.adapter_backward(s["x"], s["a"], s["b"], s["dy"], off, **kw), grads))


def test_without_rows(asg):
    say("adapter no rows")
    torch = torch_()
    x, dy = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 72, dtype=torch.bfloat16, device="cuda")
    a, b = torch.ones(2, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(2, 72, 8, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert asg.adapter_forward(x, a, b, off).shape == (0, 72)
    dx, da, db = asg.adapter_backward(x, a, b, dy, off)
    assert dx.shape == (0, 64) and not da.any() and not db.any()
    da.fill_(2.0)
    db.fill_(3.0)
    asg.adapter_backward(x, a, b, dy, off, da=da, db=db, accumulate=True)
    assert bool((da == 2).all()) and bool((db == 3).all())
    # rows, none of which has an adapter
    x = torch.ones(20, 64, dtype=torch.bfloat16, device="cuda")
    assert not asg.adapter_forward(x, a, b, off).any()


def test_refusals(asg):
    say("adapter refusals")
    torch = torch_()
    s, _ = make(4, 72, 64, 8, 2, "ordered", 6)
    off = dev(s["offsets"])
    x, a, b, dy = s["x"], s["a"], s["b"], s["dy"]
    bf = dict(dtype=torch.bfloat16, device="cuda")
    for f in (lambda: asg.adapter_forward(x, a, b[:1], off), lambda: asg.adapter_forward(x.float(), a, b, off),
              lambda: asg.adapter_forward(x, a, b, off[:2]), lambda: asg.adapter_forward(x, a, b, off.long()),
              lambda: asg.adapter_forward(x, a, b, off, rows=off), lambda: asg.adapter_forward(x, a, b, off, base=dy[:3]),
              lambda: asg.adapter_forward(x, a, b, off, base=dy, y=torch.empty(4, 72, device="cuda")),
              lambda: asg.adapter_forward(x, a, b, off, out_dtype=torch.float16),
              lambda: asg.adapter_forward(x, a.transpose(1, 2), b, off), lambda: asg.adapter_forward(x, a, b, off, scales=off),
              lambda: asg.adapter_backward(x, a, b, x, off), lambda: asg.adapter_backward(x, a, b, dy, off, accumulate=True),
              lambda: asg.adapter_backward(x, a, b, dy, off, need_dx=False, base=x)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(asg.FFNError):
        asg.adapter_forward(x, torch.zeros(2, 12, 64, **bf), torch.zeros(2, 72, 12, **bf), off)
    with pytest.raises(asg.FFNError):
        asg.adapter_forward(x, torch.zeros(2, 40, 64, **bf), torch.zeros(2, 72, 40, **bf), off, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(asg.FFNError):
        asg.adapter_backward(x, a, b, dy, off, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
