"""Host-side checks of include/ffn_linear.h and its binding (no kernel is
launched; runs without a GPU): exports, refusals before anything is launched,
calls without rows."""
from __future__ import annotations

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
P = 4096           # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    from activation_sparse_gated_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return _lib.load()


def test_exports(lib):
    from activation_sparse_gated_amd import _lib
    text = open(os.path.join(ROOT, "include", "ffn_linear.h")).read()
    names = set(re.findall(r"\b(ffn_(?:linear|rmsnorm|fp8|grouped)_[a-z_]+)\s*\(", text)) | {"ffn_fp8_linear"}
    assert names == set(_lib.LINEAR_EXPORTS)
    assert all(hasattr(lib, n) for n in names) and lib.ffn_linear_abi_version() == 1


def norm(lib, x=P, res=None, w=P, dtype=1, m=4, d=64, eps=1e-6, r=None, y=P, q=None, s=None):
    return lib.ffn_rmsnorm_forward(x, res, w, dtype, m, d, eps, r, y, q, s, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(x=P + 8), dict(y=P + 2), dict(dtype=2), dict(m=-1), dict(d=0), dict(d=12),
    dict(d=16392), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(y=None), dict(q=P),
    dict(y=None, s=P), dict(res=P), dict(res=P + 4, r=P)])
def test_norm_refusals(lib, kw):
    assert norm(lib, **kw) == INVALID


def norm_b(lib, r=P, w=P, dy=P, dr=None, dtype=1, m=4, d=64, eps=1e-6, dx=P, dw=P, acc=0, ws=P, nb=1 << 20):
    return lib.ffn_rmsnorm_backward(r, w, dy, dr, dtype, m, d, eps, dx, dw, acc, ws, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(r=None), INVALID), (dict(dy=None), INVALID), (dict(dx=None, dw=None), INVALID), (dict(acc=2), INVALID),
    (dict(dr=P + 1), INVALID), (dict(ws=None), INVALID), (dict(nb=16), WORKSPACE), (dict(d=20), INVALID),
    (dict(m=-3), INVALID), (dict(dw=P + 4), INVALID)])
def test_norm_backward_refusals(lib, kw, want):
    assert norm_b(lib, **kw) == want
    assert lib.ffn_rmsnorm_backward_workspace_bytes(4, 64) > 0
    assert lib.ffn_rmsnorm_backward_workspace_bytes(-1, 64) == 0 == lib.ffn_rmsnorm_backward_workspace_bytes(4, 12)


def test_row_limits(lib):
    top = 2 ** 31 - 2 ** 16
    assert lib.ffn_rmsnorm_backward_workspace_bytes(top, 64) > 0 == lib.ffn_rmsnorm_backward_workspace_bytes(top + 1, 64)
    assert norm(lib, m=top + 1) == INVALID == norm_b(lib, m=2 ** 31 - 1)
    assert linear(lib, m=2 ** 31 - 1, n=16, k=16) == INVALID == fwd(lib, m=2 ** 31 - 1, n=16, k=16)
    assert bwd(lib, m=top + 1, n=16, k=16) == INVALID
    for kw in (dict(m=top + 1, k=16), dict(g=2 ** 24, m=1, k=16), dict(g=2 ** 31 - 1, m=2 ** 30, k=2 ** 30), dict(k=2 ** 31 - 16)):
        assert quant(lib, **kw) == UNSUPPORTED


def quant(lib, x=P, dtype=1, g=1, m=4, k=64, rows=1, q=P, s=P, qt=None, st=None):
    return lib.ffn_fp8_quantize(x, dtype, g, m, k, rows, q, s, qt, st, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(k=24), INVALID), (dict(k=0), INVALID),
    (dict(rows=2), INVALID), (dict(rows=0), INVALID), (dict(g=0), INVALID), (dict(m=-1), INVALID), (dict(dtype=-1), INVALID),
    (dict(qt=P), INVALID), (dict(st=P), INVALID), (dict(q=P + 8), INVALID),
    (dict(m=0x7FFFFF01), UNSUPPORTED), (dict(m=1 << 30, k=1 << 20), UNSUPPORTED)])
def test_quantize_refusals(lib, kw, want):
    assert quant(lib, **kw) == want


def linear(lib, x=P, xs=P, w=P, ws=P, rows=128, m=4, n=64, k=64, off=None, g=1, y=P, yt=1, acc=0, wk=None, nb=0):
    return lib.ffn_fp8_linear(x, xs, w, ws, rows, m, n, k, off, g, y, yt, acc, wk, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(xs=None), INVALID), (dict(w=None), INVALID), (dict(ws=None), INVALID), (dict(y=None), INVALID),
    (dict(k=24), INVALID), (dict(n=0), INVALID), (dict(m=-1), INVALID), (dict(rows=64), INVALID), (dict(yt=5), INVALID),
    (dict(acc=3, yt=0), INVALID), (dict(acc=1), UNSUPPORTED), (dict(g=2), INVALID), (dict(off=P, g=0), INVALID),
    (dict(off=P, g=257), INVALID), (dict(off=P, g=2, rows=1), UNSUPPORTED), (dict(w=P + 8), INVALID),
    (dict(m=1 << 30, n=1 << 30), INVALID)])
def test_fp8_linear_refusals(lib, kw, want):
    assert linear(lib, **kw) == want


def fwd(lib, x=P, w=P, off=P, g=2, m=4, n=64, k=64, y=P, yt=1, wk=None, nb=0):
    return lib.ffn_grouped_forward(x, w, off, g, m, n, k, y, yt, wk, nb, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(off=None), dict(y=None), dict(g=0), dict(g=257), dict(n=12), dict(k=4), dict(m=-1),
    dict(yt=2), dict(off=P + 4), dict(y=P + 8)])
def test_grouped_forward_refusals(lib, kw):
    assert fwd(lib, **kw) == INVALID


def bwd(lib, x=P, w=P, dy=P, off=P, g=2, m=4, n=64, k=64, dx=P, dw=P, acc=0, wk=None, nb=0):
    return lib.ffn_grouped_backward(x, w, dy, off, g, m, n, k, dx, dw, acc, wk, nb, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(dy=None), dict(off=None), dict(dx=None, dw=None), dict(acc=2), dict(n=4), dict(k=20),
    dict(g=300), dict(m=-1), dict(dx=P + 4), dict(dw=P + 4)])
def test_grouped_backward_refusals(lib, kw):
    assert bwd(lib, **kw) == INVALID


def test_calls_without_rows(lib):
    # nothing to do: null pointers are taken
    assert norm(lib, x=None, w=None, y=None, m=0) == OK
    assert norm_b(lib, r=None, w=None, dy=None, dx=None, dw=None, ws=None, nb=0, m=0) == OK
    assert quant(lib, x=None, q=None, s=None, m=0) == OK
    assert linear(lib, x=None, xs=None, w=None, ws=None, y=None, m=0) == OK
    assert fwd(lib, x=None, w=None, off=None, y=None, m=0) == OK
    assert bwd(lib, x=None, w=None, dy=None, off=None, dx=None, dw=None, m=0) == OK
    assert bwd(lib, x=None, w=None, dy=None, off=None, dx=None, acc=1, m=0) == OK


def test_binding_refuses_host_tensors_and_wrong_shapes():
    torch = pytest.importorskip("torch")
    import activation_sparse_gated_amd as asg
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        asg.rmsnorm_forward(x, w)                       # host memory
    with pytest.raises(ValueError):
        asg.rmsnorm_backward(x, w, x)
    with pytest.raises(ValueError):
        asg.fp8_quantize(x)
    with pytest.raises(ValueError):
        asg.grouped_forward(x, torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        asg.fp8_linear(x, x)


def test_contract_says_how_8_bit_sums_are_made():
    # a bf16 output is summed to fewer bits than an fp32 one: the header and the binding say so, and by how much
    import activation_sparse_gated_amd as asg
    text = open(os.path.join(ROOT, "include", "ffn_linear.h")).read()
    about = re.sub(r"\s*\n \* ?", " ", text[text.index("/* y = x w^T of 8-bit blocks"):text.index("ffn_status ffn_fp8_linear")])
    for words in (about, re.sub(r"\s+", " ", asg.fp8_linear.__doc__)):
        assert "7 * 2^-13 of the largest product of each eight" in words and "13 bits below" in words
        assert "take FFN_F32" in words or "take fp32" in words


def test_contract_gives_the_range_of_scales():
    text = open(os.path.join(ROOT, "include", "ffn_linear.h")).read()
    about = re.sub(r"\s*\n \* ?", " ", text[text.index("/* y = x w^T of 8-bit blocks"):text.index("ffn_status ffn_fp8_linear")])
    assert "product of its two scales" in about and "has to lie in 2^-126 .. 2^128" in about


def test_stream_handle_without_the_private_entry(monkeypatch):
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace

    from activation_sparse_gated_amd import linear
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: SimpleNamespace(cuda_stream=1000 + index))
    monkeypatch.setattr(linear, "_raw_stream", None)
    assert linear._stream_handle(3) == 1003
