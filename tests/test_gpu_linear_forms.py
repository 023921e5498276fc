"""Forms of the calls in include/ffn_linear.h that leave an output out or ask
for one more: one gradient alone, the norm's plain and 8-bit output at once.
Each has to equal, bit for bit, what the whole call gives, which
test_gpu_linear.py and test_gpu_linear_tiles.py hold to the formulas."""
from __future__ import annotations

import pytest

from tests import linear_cases as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def asg(lib):
    return lib


def normal(seed, *shape, dtype=None):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype or torch.bfloat16)


def equal(a, b):
    import torch
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,d", [(0, 64), (1, 8), (7, 520), (300, 2048), (9, 8200), (2500, 264)])
def test_norm_one_gradient(asg, m, d, dtype):
    import torch
    print("[case] norm gradients", m, d, dtype, flush=True)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    r, w, dy, dr = normal(1, m, d, dtype=t), normal(2, d, dtype=t), normal(3, m, d, dtype=t), normal(4, m, d, dtype=t)
    for extra in (None, dr):
        dx, dw = asg.rmsnorm_backward(r, w, dy, dr=extra)
        a, none = asg.rmsnorm_backward(r, w, dy, dr=extra, need_dw=False)
        assert none is None and equal(a, dx)
        none, b = asg.rmsnorm_backward(r, w, dy, dr=extra, need_dx=False)
        assert none is None and equal(b, dw)
    one = torch.ones(d, device="cuda")
    both = asg.rmsnorm_backward(r, w, dy, dw=one.clone(), accumulate=True)[1]
    _, b = asg.rmsnorm_backward(r, w, dy, need_dx=False, dw=one.clone(), accumulate=True)
    assert equal(b, both)


@pytest.mark.parametrize("m,n,k,e", [(0, 64, 72, 2), (1, 8, 8, 1), (79, 872, 136, 3), (300, 264, 520, 5), (1294, 1888, 136, 3)])
def test_one_gradient_by_expert(asg, m, n, k, e):
    import torch
    print("[case] gradients by expert", m, n, k, e, flush=True)
    x, w, dy = normal(1, m, k), normal(2, e, n, k), normal(3, m, n)
    o = torch.tensor(C.offsets(m, e) if m else [0] * (e + 1), dtype=torch.int32, device="cuda")
    dx0, dw0 = normal(4, m, k), normal(5, e, n, k, dtype=torch.float32)
    dx, dw = asg.grouped_backward(x, w, dy, o, dx=dx0.clone())
    _, added = asg.grouped_backward(x, w, dy, o, dw=dw0.clone(), accumulate=True)
    for xs in (x, None):
        a, none = asg.grouped_backward(xs, w, dy, o, need_dw=False, dx=dx0.clone())
        assert none is None and equal(a, dx)
    for ws in (w, None):
        none, b = asg.grouped_backward(x, ws, dy, o, need_dx=False)
        assert none is None and equal(b, dw)
        _, b = asg.grouped_backward(x, ws, dy, o, need_dx=False, dw=dw0.clone(), accumulate=True)
        assert equal(b, added)


def test_refusals_of_one_gradient(asg):
    import torch
    print("[case] refusals", flush=True)
    r, w, dy = normal(1, 4, 64), normal(2, 64), normal(3, 4, 64)
    x, we, g = normal(1, 8, 64), normal(2, 2, 48, 64), normal(3, 8, 48)
    o = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    dw, dwe = torch.zeros(64, device="cuda"), torch.zeros(2, 48, 64, device="cuda")
    for kw in (dict(need_dx=False, need_dw=False), dict(need_dx=False, dx=r.clone()), dict(need_dw=False, dw=dw),
               dict(need_dw=False, accumulate=True), dict(need_dx=False, accumulate=True)):
        with pytest.raises(ValueError):
            asg.rmsnorm_backward(r, w, dy, **kw)
    for a, b, kw in ((x, we, dict(need_dx=False, need_dw=False)), (x, we, dict(need_dx=False, dx=x.clone())),
                     (x, we, dict(need_dw=False, dw=dwe)), (x, we, dict(need_dw=False, accumulate=True)),
                     (None, we, {}), (x, None, {}), (None, we, dict(need_dx=False)), (x, None, dict(need_dw=False)),
                     (x[:4], we, dict(need_dw=False)), (x, we[:, :, :32].contiguous(), dict(need_dx=False)), (None, None, dict(need_dw=False))):
        with pytest.raises(ValueError):
            asg.grouped_backward(a, b, g, o, **kw)
    with pytest.raises(ValueError):
        asg.grouped_backward(x, None, g, o.long(), need_dx=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,d", [(1, 8), (5, 520), (33, 2048), (3, 16384)])
def test_norm_plain_and_8_bit_at_once(asg, m, d, dtype):
    # the C entry writes both in one pass; the binding asks for one of them
    import torch
    from activation_sparse_gated_amd import _lib
    print("[case] norm, both outputs", m, d, dtype, flush=True)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, res, w = normal(1, m, d, dtype=t), normal(2, m, d, dtype=t), normal(3, d, dtype=t)
    want, r = asg.rmsnorm_forward(x, w, residual=res)
    q, _ = asg.rmsnorm_forward(x, w, residual=res, fp8=True)
    y, r2 = torch.empty_like(x), torch.empty_like(x)
    q2, s2 = torch.empty_like(q.q), torch.empty_like(q.scale)
    stream = torch.cuda.current_stream().cuda_stream
    code = _lib.load().ffn_rmsnorm_forward(x.data_ptr(), res.data_ptr(), w.data_ptr(), _lib.DTYPES[dtype], m, d, 1e-6, r2.data_ptr(),
                                           y.data_ptr(), q2.data_ptr(), s2.data_ptr(), stream)
    assert code == _lib.FFN_OK
    assert equal(y, want) and equal(r2, r) and equal(q2, q.q) and equal(s2, q.scale)


def test_stream_handle_is_the_current_stream(asg, monkeypatch):
    import torch
    from activation_sparse_gated_amd import linear
    print("[case] stream handle", flush=True)
    streams = [torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        with torch.cuda.stream(s):
            fast = linear._stream_handle(torch.cuda.current_device())
            with monkeypatch.context() as m:
                m.setattr(linear, "_raw_stream", None)
                assert fast == linear._stream_handle(torch.cuda.current_device()) == s.cuda_stream


@pytest.mark.parametrize("m,n,k", [(24, 72, 328), (40, 136, 4104), (300, 264, 520), (1294, 1888, 136), (6100, 408, 2360)])
def test_rows_and_weights_that_nobody_uses_are_not_read(asg, m, n, k):
    # NaN in the rows of no expert, and in the weights of experts without rows, reaches nothing
    import torch
    print("[case] unread", m, n, k, flush=True)
    x, w, dy = normal(1, m, k), normal(2, 4, n, k), normal(3, m, n)
    off = [5, 5, m // 2, m // 2, m - 7]
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    y0, dx0 = normal(4, m, n), normal(5, m, k)
    want = asg.grouped_forward(x, w, o, y=y0.clone()), *asg.grouped_backward(x, w, dy, o, dx=dx0.clone())
    q, wq = asg.fp8_quantize(x[:, :k // 16 * 16].contiguous()), asg.fp8_quantize(w[..., :k // 16 * 16].contiguous(), block_rows=128)
    want8 = [asg.fp8_linear(q, wq, offsets=o, y=y0.to(t, copy=True)) for t in (torch.bfloat16, torch.float32)]
    for t in (x, dy, q.q.view(torch.uint8)):
        t[:5], t[m - 7:] = (float("nan"), float("nan")) if t.is_floating_point() else (0x7F, 0x7F)
    q.scale[:, :5], q.scale[:, m - 7:] = float("nan"), float("nan")
    for e in (0, 2):
        w[e], wq.q.view(torch.uint8)[e], wq.scale[e] = float("nan"), 0x7F, float("nan")
    got = asg.grouped_forward(x, w, o, y=y0.clone()), *asg.grouped_backward(x, w, dy, o, dx=dx0.clone())
    got8 = [asg.fp8_linear(q, wq, offsets=o, y=y0.to(t, copy=True)) for t in (torch.bfloat16, torch.float32)]
    for a, b in zip((*got, *got8), (*want, *want8)):
        assert equal(a, b) and bool(torch.isfinite(a).all())
