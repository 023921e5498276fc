"""Host-side checks of include/ffn_experts.h, include/ffn_adapter.h and their
binding (no kernel is launched; runs without a GPU): exports, refusals before
anything is launched, calls without rows."""
from __future__ import annotations

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
P = 4096           # an aligned address that no refused call touches
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from activation_sparse_gated_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return _lib.load()


@pytest.mark.parametrize("header,prefix", [("ffn_experts.h", "EXPERTS"), ("ffn_adapter.h", "ADAPTER")])
def test_exports(lib, header, prefix):
    from activation_sparse_gated_amd import _lib
    text = open(os.path.join(ROOT, "include", header)).read()
    names = set(re.findall(r"^(?:ffn_status|size_t|int32_t) (ffn_\w+)\(", text, re.M))
    assert names == set(getattr(_lib, prefix + "_EXPORTS")) and all(hasattr(lib, n) for n in names)
    assert getattr(lib, f"ffn_{prefix.lower()}_abi_version")() == 1


def route(lib, l=P, dtype=0, m=4, e=16, k=2, score=0, bias=None, g=1, tg=1, best=1, renorm=1, scale=1.0, w=P, ids=P, s=None):
    return lib.ffn_route_forward(l, dtype, m, e, k, score, bias, g, tg, best, renorm, scale, w, ids, s, None)


@pytest.mark.parametrize("kw", [
    dict(l=None), dict(w=None), dict(ids=None), dict(l=P + 8), dict(w=P + 4), dict(ids=P + 2), dict(s=P + 8), dict(bias=P + 4),
    dict(dtype=2), dict(m=-1), dict(e=0), dict(e=257), dict(k=0), dict(k=17), dict(e=4, k=5), dict(score=2), dict(score=-1),
    dict(g=0), dict(g=3), dict(g=33, e=33), dict(tg=0), dict(g=4, tg=5), dict(best=0), dict(best=3), dict(renorm=2),
    dict(scale=NAN), dict(scale=INF), dict(m=2 ** 31 - 1), dict(m=2 ** 30, k=2)])
def test_route_refusals(lib, kw):
    assert route(lib, **kw) == INVALID


def route_b(lib, l=P, dtype=0, m=4, e=16, k=2, score=0, renorm=1, scale=1.0, ids=P, dw=P, ds=None, dl=P):
    return lib.ffn_route_backward(l, dtype, m, e, k, score, renorm, scale, ids, dw, ds, dl, None)


@pytest.mark.parametrize("kw", [
    dict(l=None), dict(ids=None), dict(dw=None), dict(dl=None), dict(ds=P + 4), dict(dl=P + 8), dict(dtype=-1), dict(m=-1),
    dict(e=300), dict(k=17, e=64), dict(score=3), dict(renorm=-1), dict(scale=-INF)])
def test_route_backward_refusals(lib, kw):
    assert route_b(lib, **kw) == INVALID


def group(lib, ids=P, n=100, g=8, off=P, rows=P, slots=P, ws=None, nb=0):
    return lib.ffn_group_rows(ids, n, g, off, rows, slots, ws, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ids=None), INVALID), (dict(off=None), INVALID), (dict(off=None, n=0), INVALID), (dict(rows=P + 4), INVALID),
    (dict(slots=P + 8), INVALID), (dict(n=-1), INVALID), (dict(g=0), INVALID), (dict(g=1025), INVALID),
    (dict(n=2 ** 24 + 1), UNSUPPORTED), (dict(n=20000), INVALID), (dict(n=20000, ws=P, nb=16), WORKSPACE),
    (dict(n=20000, ws=P + 4, nb=1 << 20), INVALID)])
def test_group_refusals(lib, kw, want):
    assert group(lib, **kw) == want


def test_group_workspace(lib):
    f = lib.ffn_group_rows_workspace_bytes
    assert f(8192, 8) == 0 < f(8193, 8) <= f(2 ** 24, 1024) and f(2 ** 24 + 1, 8) == 0 == f(20000, 1025) == f(-1, 8)


def gather(lib, x=P, dtype=1, m=4, d=64, slots=P, k=2, y=P, q=None, s=None):
    return lib.ffn_gather_forward(x, dtype, m, d, slots, k, y, q, s, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(slots=None), dict(y=None), dict(q=P), dict(s=P), dict(y=P + 8), dict(q=P + 4, s=P), dict(d=12), dict(d=0),
    dict(d=2 ** 22 + 8), dict(k=0), dict(k=17), dict(m=-1), dict(dtype=3), dict(m=2 ** 30), dict(slots=P + 4)])
def test_gather_refusals(lib, kw):
    assert gather(lib, **kw) == INVALID


def combine(lib, y=P, dtype=1, m=4, d=64, slots=P, k=2, w=None, res=None, out=P):
    return lib.ffn_combine_forward(y, dtype, m, d, slots, k, w, res, out, None)


@pytest.mark.parametrize("kw", [
    dict(y=None), dict(slots=None), dict(out=None), dict(w=P + 4), dict(res=P + 8), dict(d=20), dict(k=0), dict(k=17), dict(m=-2),
    dict(dtype=2), dict(m=2 ** 29, k=4)])
def test_combine_refusals(lib, kw):
    assert combine(lib, **kw) == INVALID


def combine_b(lib, y=P, dtype=1, m=4, d=64, slots=P, k=2, w=P, dout=P, dy=P, dw=P):
    return lib.ffn_combine_backward(y, dtype, m, d, slots, k, w, dout, dy, dw, None)


@pytest.mark.parametrize("kw", [
    dict(y=None), dict(slots=None), dict(dout=None), dict(dy=None, dw=None), dict(dy=P + 8), dict(dw=P + 4), dict(w=P + 1),
    dict(d=4), dict(k=0), dict(m=-1)])
def test_combine_backward_refusals(lib, kw):
    assert combine_b(lib, **kw) == INVALID


BIG = 1 << 40


def adapter(lib, x=P, a=P, b=P, s=None, off=P, rows=None, g=2, m=4, n=64, k=64, r=16, base=None, y=P, yt=1, ws=P, nb=BIG):
    return lib.ffn_adapter_forward(x, a, b, s, off, rows, g, m, n, k, r, base, y, yt, ws, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(off=None), INVALID), (dict(y=None), INVALID),
    (dict(ws=None, r=40), INVALID), (dict(ws=P + 8), INVALID), (dict(nb=16, r=40), WORKSPACE), (dict(s=P + 4), INVALID),
    (dict(rows=P + 8), INVALID), (dict(base=P + 2), INVALID), (dict(g=0), INVALID), (dict(g=1025), INVALID), (dict(m=-1), INVALID),
    (dict(m=2 ** 26 + 1), INVALID), (dict(n=12), INVALID), (dict(k=4), INVALID), (dict(r=12), INVALID), (dict(r=0), INVALID),
    (dict(r=264), INVALID), (dict(n=2 ** 22 + 8), INVALID), (dict(yt=2), INVALID)])
def test_adapter_refusals(lib, kw, want):
    assert adapter(lib, **kw) == want


def adapter_b(lib, x=P, a=P, b=P, s=None, dy=P, off=P, rows=None, g=2, m=4, n=64, k=64, r=16, base=None, dx=P, da=P, db=P, acc=0,
              ws=P, nb=BIG):
    return lib.ffn_adapter_backward(x, a, b, s, dy, off, rows, g, m, n, k, r, base, dx, da, db, acc, ws, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(off=None), INVALID),
    (dict(dx=None, da=None, db=None), INVALID), (dict(dx=None, base=P), INVALID), (dict(acc=2), INVALID), (dict(ws=None), INVALID),
    (dict(nb=16), WORKSPACE), (dict(da=P + 4), INVALID), (dict(db=P + 8), INVALID), (dict(dx=P + 2), INVALID),
    (dict(x=None, dx=None, da=None), INVALID), (dict(a=None, dx=None, da=None), INVALID), (dict(b=None, dx=None, db=None), INVALID),
    (dict(r=20), INVALID), (dict(g=2000), INVALID)])
def test_adapter_backward_refusals(lib, kw, want):
    assert adapter_b(lib, **kw) == want


def test_adapter_workspace(lib):
    for f in (lib.ffn_adapter_forward_workspace_bytes, lib.ffn_adapter_backward_workspace_bytes):
        assert f(5, 64, 64, 40, 2) > 0 and f(0, 64, 64, 40, 2) == 0 == f(5, 60, 64, 40, 2) == f(5, 64, 64, 40, 1025)
    assert lib.ffn_adapter_forward_workspace_bytes(5, 64, 64, 16, 2) == 0 < lib.ffn_adapter_backward_workspace_bytes(5, 64, 64, 16, 2)


def test_calls_without_rows(lib):
    # nothing to do: null pointers are taken
    assert route(lib, l=None, w=None, ids=None, m=0) == OK
    assert route_b(lib, l=None, ids=None, dw=None, dl=None, m=0) == OK
    assert gather(lib, x=None, slots=None, y=None, m=0) == OK
    assert combine(lib, y=None, slots=None, out=None, m=0) == OK
    assert combine_b(lib, y=None, slots=None, dout=None, dy=None, dw=None, m=0) == OK
    assert adapter(lib, x=None, a=None, b=None, off=None, y=None, ws=None, nb=0, m=0) == OK
    assert adapter_b(lib, x=None, a=None, b=None, dy=None, off=None, dx=None, da=None, db=None, ws=None, nb=0, m=0) == OK
    assert adapter_b(lib, acc=1, m=0) == OK


def test_binding_refuses_host_tensors_and_bad_arguments():
    torch = pytest.importorskip("torch")
    import activation_sparse_gated_amd as asg
    x, ids = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    w = torch.zeros(4, 2)
    calls = [
        lambda: asg.route_forward(x, 2), lambda: asg.route_backward(x, ids, w), lambda: asg.group_rows(ids, 4),
        lambda: asg.gather_forward(x, ids), lambda: asg.gather_backward(x, ids), lambda: asg.combine_forward(x, ids, w),
        lambda: asg.combine_backward(x, ids, w, x), lambda: asg.combine_backward(x, ids, w, x, need_dy=False, need_dweights=False),
        lambda: asg.combine_backward(x, ids, w, x, need_dy=False, dy=x),
        lambda: asg.adapter_forward(x, x[None], x[None], ids[0]), lambda: asg.adapter_backward(x, x[None], x[None], x, ids[0]),
        lambda: asg.adapter_backward(x, x[None], x[None], x, ids[0], need_dx=False, need_da=False, need_db=False),
        lambda: asg.adapter_backward(x, x[None], x[None], x, ids[0], need_dx=False, base=x)]
    for call in calls:
        with pytest.raises(ValueError):
            call()
