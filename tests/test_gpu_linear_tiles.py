"""Every instance of the product kernels, element by element, on integers.

Inputs are integers (8-bit blocks: times scales of 1 and 2) whose products'
magnitudes add up to less than 2^24 in every output: fp32 holds every partial
sum in whatever order, so fp32 outputs are equal to the exact ones and bf16
outputs are those rounded once, and no tolerance is needed. The sizes
(tests/linear_cases.py) take every tile, way of summing and slicing; a test on
the host checks that they do.

8-bit products with a bf16 output: the largest product of an eight is below 2^8
and the least 1, so nothing lies 13 bits below it. With an fp32 output the
inputs have eights with 2^16 and -2^16 besides, beside which the e4m3
instructions would lose the small ones (test_gpu_linear_sums.py).
"""
from __future__ import annotations

import pytest

from tests import linear_cases as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def asg(lib):
    return lib


@pytest.fixture
def rnd():
    import torch
    gen = torch.Generator(device="cuda").manual_seed(71)

    def ints(top, *shape):
        return torch.randint(-top, top + 1, shape, generator=gen, device="cuda", dtype=torch.float32)
    return ints


def same(got, want, what):
    """got is the exact result `want` (fp64) in its type; the first difference is named."""
    import torch
    want = want.float().to(got.dtype)
    if torch.equal(got, want):
        return
    at = (got != want).nonzero()
    i = tuple(at[0].tolist())
    raise AssertionError(f"{what}: {len(at)} of {got.numel()} differ, first at {i}: {got[i].item()}, not {want[i].item()}; "
                         f"last at {tuple(at[-1].tolist())}")


def repeat(scale, rows, m, k):
    """The scale of every value: blocks of rows x 128."""
    s = scale.transpose(-1, -2) if rows == 1 else scale.repeat_interleave(128, -2)[..., :m, :]
    return s.repeat_interleave(128, -1)[..., :k]


def product_inputs(asg, rnd, m, n, k, experts, rows, wide):
    """Blocks of x and w and the values they stand for, in fp64."""
    import torch
    top = 3 if wide else 15                              # 36 k or 900 k of 2^24
    lead = (experts,) if experts else ()
    x, w = rnd(top, m, k), rnd(top, *lead, n, k)
    if wide:                                             # 20 eights: 20 * 2 * 2^16 * 4 of 2^24
        step = max(1, k // 8 // 20)
        for i in range(20):
            e = 8 * (i * step % (k // 8))
            a, b = e + i % 8, e + (i * 3 + 1 + i % 8) % 8
            if a == b:
                b = e + (a - e + 1) % 8
            sign = torch.where(rnd(1, m) < 0, -256.0, 256.0)
            x[:, a], x[:, b] = sign, sign
            w[..., a], w[..., b] = 256, -256
    kb, nb = -(-k // 128), -(-n // 128)
    xs = torch.where(rnd(1, kb, m) > 0, 2.0, 1.0)
    ws = torch.where(rnd(1, *lead, *((kb, n) if rows == 1 else (nb, kb))) > 0, 2.0, 1.0)
    fp8 = torch.float8_e4m3fn
    xb, wb = asg.Fp8Tensor(x.to(fp8), xs, 1), asg.Fp8Tensor(w.to(fp8), ws, rows)
    assert bool((xb.q.float() == x).all()) and bool((wb.q.float() == w).all())
    return xb, wb, x.double() * repeat(xs, 1, m, k), w.double() * repeat(ws, rows, n, k)


def by_expert(x, w, off, y):
    """y with the rows of each expert replaced by x w_e^T."""
    y = y.clone()
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        if b > a:
            y[a:b] = x[a:b] @ w[e].T.contiguous()
    return y


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k,e", C.FP8)
def test_products_of_blocks(asg, rnd, m, n, k, e, out):
    import torch
    print("[case] 8-bit", m, n, k, e, out, flush=True)
    dtype = torch.bfloat16 if out == "bf16" else torch.float32
    for rows in (1, 128) if not e else (128,):
        x, w, X, W = product_inputs(asg, rnd, m, n, k, e, rows, out == "f32")
        off = C.offsets(m, e) if e else [0, m]
        kw = dict(offsets=torch.tensor(off, dtype=torch.int32, device="cuda")) if e else {}
        y0 = rnd(100, m, n).to(dtype)
        want = by_expert(X, W if e else W[None], off, y0.double())
        same(asg.fp8_linear(x, w, y=y0.clone(), **kw), want, f"rows {rows}")   # rows of no expert: as they were
        if out == "f32":
            got = asg.fp8_linear(x, w, y=y0.clone(), accumulate=True, **kw)
            want[off[0]:off[-1]] += y0[off[0]:off[-1]].double()
            same(got, want, f"rows {rows}, added to")
        del x, w, X, W, want


@pytest.mark.parametrize("m,n,k,e", C.FWD)
def test_products_by_expert(asg, rnd, m, n, k, e):
    import torch
    print("[case] forward", m, n, k, e, flush=True)
    x, w = rnd(15, m, k).bfloat16(), rnd(15, e, n, k).bfloat16()
    off = C.offsets(m, e)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        y0 = rnd(100, m, n).to(dtype)
        want = by_expert(x.double(), w.double(), off, y0.double())
        same(asg.grouped_forward(x, w, o, y=y0.clone()), want, dtype)


@pytest.mark.parametrize("m,n,k,e", C.BWD)
def test_gradients_by_expert(asg, rnd, m, n, k, e):
    import torch
    print("[case] backward", m, n, k, e, flush=True)
    x, w, dy = rnd(15, m, k).bfloat16(), rnd(15, e, n, k).bfloat16(), rnd(15, m, n).bfloat16()
    off = C.offsets(m, e)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    dx0, dw0 = rnd(100, m, k).bfloat16(), rnd(100, e, n, k)
    dx, dw = asg.grouped_backward(x, w, dy, o, dx=dx0.clone())
    wdx, wdw = dx0.double(), torch.zeros(e, n, k, dtype=torch.float64, device="cuda")
    for i in range(e):
        a, b = off[i], off[i + 1]
        if b > a:
            wdx[a:b] = dy[a:b].double() @ w[i].double()
            wdw[i] = dy[a:b].double().T.contiguous() @ x[a:b].double()
    same(dx, wdx, "dx")
    same(dw, wdw, "dw")                                  # an expert without rows: zeros
    dx, dw = asg.grouped_backward(x, w, dy, o, dx=dx0.clone(), dw=dw0.clone(), accumulate=True)
    same(dx, wdx, "dx again")
    same(dw, wdw + dw0.double(), "dw added to")
