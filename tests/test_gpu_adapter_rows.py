"""The adapters' rows and offsets out of range, NaN and infinities, in every form
of the kernels: one launch, two launches, tiles of 16 and of 64 rows, whole and in
slices, ranks over 64. Against the fp64 definitions (oracle/experts_oracle.py),
within the bounds of test_gpu_adapter.py; what bad numbers do not enter is equal
bit for bit to what it is without them.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import experts_oracle as E
from tests.test_gpu_adapter import call, make
from tests.test_gpu_experts import B, TINY, U, dev, f64, near, say, torch_

pytestmark = pytest.mark.gpu

# rows, n, k, rank, adapters
SHAPES = [(40, 136, 264, 24, 4), (90, 1032, 4104, 72, 3), (130, 136, 264, 40, 7), (300, 2056, 328, 32, 40), (70, 264, 328, 136, 3),
          (1500, 136, 72, 8, 33), (4200, 264, 136, 16, 3), (8200, 136, 264, 16, 9), (8450, 264, 136, 128, 100), (2100, 264, 8200, 64, 3),
          (4100, 136, 8200, 16, 7), (2056, 1160, 1096, 32, 3), (8192, 200, 200, 200, 6), (2050, 72, 16392, 24, 64)]
shapes = pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def asg(lib):
    return lib


def e(c):
    return (c / 8 + 80) * 2 * U


@shapes
@pytest.mark.parametrize("kind", ["rows", "ordered"])
def test_offsets_and_rows_out_of_range(asg, shape, kind):
    say("adapter rows out of range", shape, kind)
    torch = torch_()
    m, n, k, r, groups = shape
    s, g = make(m, n, k, r, groups, kind, 21)
    off = s["offsets"].astype(np.int64)
    off[0], off[-1] = (-3, 2 ** 31 - 1) if kind == "ordered" else (off[0], m + 77)
    off[groups // 2] -= 5 if kind == "rows" else 9 * m  # below the ones before it
    s["offsets"] = off.astype(np.int32)
    left = []
    if kind == "rows":                                  # places without a row: the rows that stood there are not named
        at = np.concatenate([np.flatnonzero(s["rows"] == 0), g.choice(m, max(4, m // 9), replace=False)])
        left = sorted(set(s["rows"][at].tolist()))
        s["rows"] = s["rows"].copy()
        s["rows"][at] = g.choice([-1, -4, m, m + 1, -2 ** 31, 2 ** 31 - 1], len(at))
    base_y, base_x = dev(g.normal(0, 1, (m, n)), "bf16"), dev(g.normal(0, 1, (m, k)), "bf16")
    for t in (s["x"], s["dy"], base_y, base_x):         # and are not read
        t[left] = NAN
    of, args = dev(s["offsets"]), (f64(s["x"]), f64(s["a"]), f64(s["b"]), s["scales"])
    where = (s["offsets"], s["rows"])
    sizes = [np.abs(v) for v in args[:3]] + [s["scales"]]

    y = torch.full((m, n), 9.0, dtype=torch.bfloat16, device="cuda")
    asg.adapter_forward(s["x"], s["a"], s["b"], of, base=base_y, y=y, **call(s))
    want, size = E.adapter(*args, *where, f64(base_y)), E.adapter(*sizes, *where, None)
    want[left] = 9.0
    slack = (e(k) + B ** 2 + (3 * r + 100) * 2 * U) * size + 2 * U * (size + np.nan_to_num(np.abs(f64(base_y))))
    near(f64(y), want, slack + B * np.abs(want) * (1 + 1e-3) + TINY, "y")
    again = base_y.clone()                              # in place
    asg.adapter_forward(s["x"], s["a"], s["b"], of, base=again, y=again, **call(s))
    named = sorted(set(range(m)) - set(left))
    assert torch.equal(again[named], y[named]) and bool(torch.isnan(again[left]).all())

    dx = torch.full((m, k), 7.0, dtype=torch.bfloat16, device="cuda")
    dx, da, db = asg.adapter_backward(s["x"], s["a"], s["b"], s["dy"], of, base=base_x, dx=dx, **call(s))
    dy = f64(s["dy"])
    want = list(E.adapter_backward(*args, dy, *where, f64(base_x)))
    size = E.adapter_backward(*sizes, np.abs(dy), *where, None)
    want[0][left] = 7.0
    slack = (e(n) + B ** 2 + (3 * r + 100) * 2 * U) * size[0] + 2 * U * (size[0] + np.nan_to_num(np.abs(f64(base_x))))
    near(f64(dx), want[0], slack + B * np.abs(want[0]) * (1 + 1e-3) + TINY, "dx")
    rows = 3 * e(m) + B ** 3 + 8 * U
    for got, i, c in ((da, 1, n), (db, 2, k)):
        near(f64(got), want[i], (e(c) + rows) * size[i] + 2 * U * size[i] + TINY, ("dx", "da", "db")[i])


def run(asg, s, x, a, b, dy):
    of, kw = dev(s["offsets"]), call(s)
    return (asg.adapter_forward(x, a, b, of, **kw), *asg.adapter_backward(x, a, b, dy, of, **kw))


def same_but(got, good, bad):
    """Not finite where `bad` says, and equal everywhere else."""
    torch = torch_()
    assert bool((torch.isfinite(got) != bad).all()) and torch.equal(torch.where(bad, 0, got), torch.where(bad, 0, good))


@shapes
@pytest.mark.parametrize("kind", ["rows", "ordered"])
def test_bad_numbers_stay_where_they_enter(asg, shape, kind):
    say("adapter bad numbers", shape, kind)
    torch = torch_()
    m, n, k, r, groups = shape
    s, g = make(m, n, k, r, groups, kind, 22)
    of = E.adapter_rows(s["offsets"], s["rows"], m, groups)
    live = [e for e in range(groups) if of[e]]
    none = sorted(set(range(m)) - {t for rows in of for t in rows})
    good = run(asg, s, s["x"], s["a"], s["b"], s["dy"])
    zero = [torch.zeros(v.shape, dtype=torch.bool, device="cuda") for v in good]

    # rows without an adapter, and adapters without rows
    x, a, b, dy = (s[v].clone() for v in ("x", "a", "b", "dy"))
    x[none], dy[none] = NAN, INF
    idle = [e for e in range(groups) if not of[e]]
    a[idle], b[idle] = NAN, INF
    for got, want in zip(run(asg, s, x, a, b, dy), good):
        assert torch.equal(got, want)

    # one number of a row of an adapter, or of an adapter's weights
    one = live[int(g.integers(len(live)))]
    t, i, c, j = of[one][int(g.integers(len(of[one])))], *(int(g.integers(v)) for v in (k, n, r))
    for value in (INF, -INF, NAN):
        x, bad = s["x"].clone(), [v.clone() for v in zero]
        x[t, i] = value
        bad[0][t], bad[2][one, :, i], bad[3][one] = True, True, True
        for got, want, v in zip(run(asg, s, x, s["a"], s["b"], s["dy"]), good, bad):
            same_but(got, want, v)
        dy, bad = s["dy"].clone(), [v.clone() for v in zero]
        dy[t, c] = value
        bad[1][t], bad[2][one], bad[3][one, c] = True, True, True
        for got, want, v in zip(run(asg, s, s["x"], s["a"], s["b"], dy), good, bad):
            same_but(got, want, v)
        a, bad = s["a"].clone(), [v.clone() for v in zero]
        a[one, j, i] = value
        bad[0][of[one]], bad[3][one, :, j] = True, True
        bad[1][of[one], i] = True
        for got, want, v in zip(run(asg, s, s["x"], a, s["b"], s["dy"]), good, bad):
            same_but(got, want, v)
        b, bad = s["b"].clone(), [v.clone() for v in zero]
        b[one, c, j] = value
        bad[0][of[one], c] = True
        bad[1][of[one]], bad[2][one, j] = True, True
        for got, want, v in zip(run(asg, s, s["x"], s["a"], b, s["dy"]), good, bad):
            same_but(got, want, v)
