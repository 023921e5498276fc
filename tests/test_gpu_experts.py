"""GPU parity of routing to experts and the rows' way there and back
(include/ffn_experts.h) against their fp64 definitions (oracle/experts_oracle.py).

Bounds. u = 2^-24 is half an fp32 step (relative), b = 2^-8 half a bf16 step.
 * Scores: the argument l - max is rounded once (u |l - max| in the exponential's
   result), exp and log1p are within 2u of theirs, a sum over a token has at most
   16 + 6 additions: (2 |l|max + 40) 2u relative, with |l|max over the token. The
   log of a sigmoid is off by u of itself, which is at most |l| + 1.
 * Their gradients: each of the products p G, p sum(G p), w g, w sum(g w) within
   that of its own size, with 12 more roundings.
 * A combination of K rows: K + 2 fused additions; the gradient of a weight: d
   terms, at most d / 256 + 18 of them one after the other.
 * A choice is compared as whole numbers: it is made in fp64, where random values
   do not come near enough to each other to be confused.
"""
from __future__ import annotations

import sys

import numpy as np
import pytest

from oracle import experts_oracle as E
from oracle import linear_oracle as L

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -120                    # below the smallest normal fp32 values' products


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def asg(lib):
    return lib


def torch_():
    import torch
    return torch


def dev(a, dtype="f32"):
    torch = torch_()
    a = np.ascontiguousarray(a)
    if a.dtype.kind == "i":
        return torch.from_numpy(a.astype(np.int32)).cuda()
    t = torch.from_numpy(a.astype(np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def half(dtype):
    return B if dtype == "bf16" else U


def near(got, want, slack, what=""):
    """|got - want| <= slack elementwise; NaN where NaN is wanted, infinities alike."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    ok = np.isfinite(want)
    assert np.array_equal(got[~ok & ~np.isnan(want)], want[~ok & ~np.isnan(want)]), what
    over = (np.abs(got - want) - np.broadcast_to(slack, want.shape))[ok]
    assert over.size == 0 or over.max() <= 0, (what, float(over.max()))


def rng(*seed):
    return np.random.default_rng(np.random.SeedSequence([43, *seed]))


# ---------------------------------------------------------------- router
FORMS = [dict(), dict(renormalize=False), dict(sigmoid=True), dict(sigmoid=True, renormalize=False, scale=2.5),
         dict(bias=True), dict(sigmoid=True, bias=True), dict(groups=True), dict(groups=True, group_best=2),
         dict(groups=True, sigmoid=True, bias=True, group_best=2, scale=2.5), dict(groups=True, bias=True, renormalize=False)]
# tokens, experts, top_k, groups, groups that stay
ROUTES = [(1, 256, 8, 8, 4), (37, 256, 8, 8, 3), (5, 8, 2, 4, 2), (3, 1, 1, 1, 1), (70, 16, 16, 2, 1), (33, 12, 5, 3, 2),
          (18, 60, 6, 5, 2), (129, 64, 6, 8, 8), (9, 128, 8, 32, 20), (21, 250, 16, 10, 3), (65, 33, 4, 11, 5), (300, 7, 7, 7, 7),
          (17, 96, 3, 2, 1)]


def settings(form, m, experts, top_k, groups, top_groups, g):
    kw = dict(form)
    bias = (0.2 * g.normal(0, 1, experts)).astype(np.float32) if kw.pop("bias", False) else None
    if kw.pop("groups", False):
        kw.update(groups=groups, top_groups=top_groups)
    return kw, bias


def args(kw):
    out = {k: v for k, v in kw.items() if k != "sigmoid"}
    return dict(out, score="sigmoid" if kw.get("sigmoid") else "softmax")


def check_route(asg, l, dtype, top_k, kw, bias):
    torch = torch_()
    t = dev(l, dtype)
    w, ids, s = asg.route_forward(t, top_k, bias=None if bias is None else dev(bias), scores=True, **args(kw))
    assert w.dtype == s.dtype == torch.float32 and ids.dtype == torch.int32
    want = E.route(f64(t), top_k, bias=bias, **kw)
    assert np.array_equal(ids.cpu().numpy(), want[1])
    big = np.abs(np.where(np.isfinite(f64(t)), f64(t), 0)).max(1, keepdims=True)
    rel = (2 * big + 40) * 2 * U
    near(f64(w), want[0], rel * np.abs(want[0]) + TINY, "weights")
    near(f64(s), want[2], rel * np.abs(want[2]) + TINY, "scores")
    # the same without the scores
    w2, ids2, none = asg.route_forward(t, top_k, bias=None if bias is None else dev(bias), **args(kw))
    assert none is None and torch.equal(w, w2) and torch.equal(ids, ids2)
    return t, w, ids, want


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_route(asg, form, dtype):
    for i, (m, experts, top_k, groups, top_groups) in enumerate(ROUTES):
        say("route", FORMS[form], dtype, m, experts, top_k)
        g = rng(1, form, i)
        kw, bias = settings(FORMS[form], m, experts, top_k, groups, top_groups, g)
        check_route(asg, g.normal(0, 2, (m, experts)), dtype, top_k, kw, bias)


# more tokens than a wave each would take: 16 lanes a token
MANY = [(1100, 256, 8, 8, 4), (1030, 128, 6, 16, 5), (1060, 100, 4, 10, 3), (1027, 250, 16, 2, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_route_many_tokens(asg, form, dtype):
    for i, (m, experts, top_k, groups, top_groups) in enumerate(MANY):
        say("route many", FORMS[form], dtype, m, experts, top_k)
        g = rng(9, form, i)
        kw, bias = settings(FORMS[form], m, experts, top_k, groups, top_groups, g)
        l = g.normal(0, 2, (m, experts))
        l[g.random((m, experts)) < 0.1] = -np.inf
        l[5] = 1.0                                      # equal values: the lowest indices
        l[6] = -np.inf
        l[7] = np.round(l[7])
        check_route(asg, l, dtype, top_k, kw, bias)


@pytest.mark.parametrize("form", range(len(FORMS)))
def test_route_masked_logits(asg, form):
    # experts that may not be chosen, tokens with fewer of them than slots, one without any
    for i, (m, experts, top_k, groups, top_groups) in enumerate([(40, 64, 6, 8, 3), (21, 256, 8, 8, 4), (12, 8, 2, 4, 2)]):
        say("route masked", FORMS[form], m, experts)
        g = rng(2, form, i)
        kw, bias = settings(FORMS[form], m, experts, top_k, groups, top_groups, g)
        l = g.normal(0, 2, (m, experts))
        l[g.random((m, experts)) < 0.6] = -np.inf
        l[3] = -np.inf
        l[4, 1:] = -np.inf
        l[5, : experts // 2] = -np.inf
        check_route(asg, l, "f32", top_k, kw, bias)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_route_ties_go_to_the_lower_index(asg, sigmoid, biased):
    say("route ties", sigmoid, biased)
    g = rng(3)
    for experts, top_k, groups, top_groups in ((256, 8, 8, 4), (40, 5, 4, 2), (8, 3, 2, 1)):
        l = g.integers(-2, 3, (50, experts)).astype(np.float64)
        l[7] = 0.0
        bias = np.full(experts, 0.25, np.float32) if biased else None
        for best in (1, 2):
            check_route(asg, l, "f32", top_k, dict(sigmoid=sigmoid, groups=groups, top_groups=top_groups, group_best=best), bias)
            check_route(asg, l, "f32", top_k, dict(sigmoid=sigmoid), bias)


@pytest.mark.parametrize("m", [33, 1040])
@pytest.mark.parametrize("experts", [64, 256])
def test_route_close_values_are_told_apart(asg, m, experts):
    # scores that are equal in fp32 and not in fp64: logits one fp32 step apart at 9 differ by 1e-10 in their sigmoids
    say("route close", m, experts)
    l = np.float32(9.0) + np.arange(experts, dtype=np.float32) * np.float32(2.0 ** -20)
    g = rng(4, m, experts)
    l = np.stack([g.permutation(l) for _ in range(m)])
    # and a few such among ordinary ones
    l[1::2] = np.where(g.random(l[1::2].shape) < 0.05, l[1::2], g.normal(0, 2, l[1::2].shape))
    zero = np.zeros(experts, np.float32)
    for kw in (dict(sigmoid=True), dict()):
        check_route(asg, l, "f32", 8, kw, zero)
        check_route(asg, l, "f32", 16, kw, None)
        for best in (1, 2):
            check_route(asg, l, "f32", 8, dict(kw, groups=8, top_groups=2, group_best=best), None)
            check_route(asg, l, "f32", 8, dict(kw, groups=8, top_groups=2, group_best=best), zero)


@pytest.mark.parametrize("m", [1, 1000, 1040])
@pytest.mark.parametrize("experts", [64, 256])
def test_route_groups_by_the_second_of_two_close_values(asg, m, experts):
    # two experts next to each other, equal in fp32, the second one larger in fp64: the best of their group, ahead of a value
    # between the two in another group
    say("route groups close", m, experts)
    g = rng(14, m, experts)
    step, size = 2.0 ** -20, experts // 8
    l = np.clip(g.normal(-2, 1, (m, experts)), None, 4).astype(np.float32)
    for t in range(m):
        one, two = g.permutation(8)[:2] * size + 2 * g.integers(0, size // 2, 2)
        l[t, one], l[t, one + 1], l[t, two] = 9, 9 + 2 * step, 9 + step
        if t % 2:
            l[t, two + 1] = 9 + step / 2 if t % 4 == 1 else 9 - 4 * step
    zero = np.zeros(experts, np.float32)
    for kw in (dict(sigmoid=True), dict()):
        for top_groups in (1, 2):
            check_route(asg, l, "f32", 4, dict(kw, groups=8, top_groups=top_groups, group_best=1), zero)
        check_route(asg, l, "f32", 4, dict(kw, groups=8, top_groups=1, group_best=1), None)


def test_route_far_logits(asg):
    # saturated and vanishing scores: the choice is the logits', the renormalised weights keep their ratio
    say("route far")
    g = rng(5)
    l = g.normal(0, 1, (20, 32)) + g.choice([-3e4, -200.0, -80.0, 80.0, 3e4], (20, 1))
    for kw in (dict(sigmoid=True), dict(), dict(sigmoid=True, renormalize=False), dict(renormalize=False)):
        check_route(asg, l, "f32", 4, kw, None)


def test_route_bad_numbers(asg):
    say("route bad numbers")
    torch = torch_()
    g = rng(6)
    l = g.normal(0, 1, (6, 24)).astype(np.float32)
    l[1, 5], l[2, 7], l[3, 2], l[3, 9] = np.nan, np.inf, np.nan, -np.inf
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(24, device="cuda")):
            w, ids, s = asg.route_forward(dev(l), 4, score=score, bias=bias, scores=True)
            w, ids, s = f64(w), ids.cpu().numpy(), f64(s)
            good = [0, 4, 5]
            want = E.route(l[good], 4, sigmoid=score == "sigmoid")
            assert np.array_equal(ids[good], want[1]) and np.isfinite(w[good]).all()
            assert ((ids >= 0) & (ids < 24)).all()
            if score == "softmax":
                assert np.isnan(w[[1, 2, 3]]).all() and np.isnan(s[1]).all()
            else:
                assert ids[1, 0] == 5 and ids[3, 0] == 2 and ids[2, 0] == 7 and np.isnan(w[[1, 3]]).all() and np.isfinite(w[2]).all()


def route_backward_slack(l, ids, dw, ds, *, sigmoid=False, renormalize=True, scale=1.0):
    """What the module's bounds allow: of the sizes of all products that make up a logit's gradient."""
    p = E.scores(l, sigmoid)
    G = np.abs(np.zeros(l.shape) if ds is None else ds).astype(np.float64)
    part = np.zeros(l.shape)
    for r in range(len(l)):
        live = ids[r] >= 0
        e, d = ids[r][live], np.abs(dw[r][live]).astype(np.float64)
        if renormalize:
            w = E.weights(l[r, e], p[r, e], sigmoid, True)
            np.add.at(part[r], e, scale * w * (d + np.sum(d * w)))
        else:
            np.add.at(G[r], e, scale * d)
    size = part + p * G + (0 if sigmoid else p * np.sum(p * G, 1, keepdims=True))
    big = np.abs(np.where(np.isfinite(l), l, 0)).max(1, keepdims=True)
    return (4 * big + 104) * 2 * U * size


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_backward(asg, dtype, sigmoid, renormalize):
    for i, (m, experts, top_k, _, _) in enumerate(ROUTES):
        say("route backward", dtype, sigmoid, renormalize, m, experts)
        g = rng(7, i)
        l = g.normal(0, 2, (m, experts))
        l[0, : experts // 3] = -np.inf
        t = dev(l, dtype)
        kw = dict(sigmoid=sigmoid, renormalize=renormalize, scale=2.5)
        ids = E.route(f64(t), top_k, **kw)[1]
        dw = g.normal(0, 1, (m, top_k)).astype(np.float32)
        for ds in (None, g.normal(0, 0.3, (m, experts)).astype(np.float32)):
            got = asg.route_backward(t, dev(ids), dev(dw), dscores=None if ds is None else dev(ds), **args(kw))
            assert got.dtype == t.dtype
            want = E.route_backward(f64(t), ids, dw, ds, **kw)
            slack = route_backward_slack(f64(t), ids, dw, ds, **kw)
            near(f64(got), want, slack + half(dtype) * np.abs(want) * (1 + 1e-4) + TINY, "dlogits")


def test_route_backward_slots_without_experts_and_in_place(asg):
    say("route backward slots")
    torch = torch_()
    g = rng(8)
    l, dw = g.normal(0, 1, (9, 20)), g.normal(0, 1, (9, 4)).astype(np.float32)
    ids = E.route(l.astype(np.float32), 4)[1]
    ids[2, 2:], ids[3], ids[4, 0], ids[5, 1] = -1, -1, 20, -77
    for kw in (dict(renormalize=False), dict(renormalize=True), dict(sigmoid=True, renormalize=True)):
        t = dev(l)
        want = E.route_backward(f64(t), ids, dw, None, **kw)
        got = asg.route_backward(t, dev(ids), dev(dw), **args(kw))
        near(f64(got), want, 1e-5)
        again = asg.route_backward(t, dev(ids), dev(dw), dlogits=t, **args(kw))
        assert again is t and torch.equal(again, got)
    # a token without any expert has no gradient
    t = torch.full((3, 12), -float("inf"), device="cuda")
    none = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    for score in ("softmax", "sigmoid"):
        for r in (False, True):
            z = asg.route_backward(t, none, torch.ones(3, 2, device="cuda"), dscores=torch.ones(3, 12, device="cuda"),
                                   score=score, renormalize=r)
            assert not z.any()


# ---------------------------------------------------------------- order by group
@pytest.mark.parametrize("groups", [1, 2, 7, 8, 63, 64, 255, 256, 1000, 1024])
@pytest.mark.parametrize("n", [1, 5, 64, 200, 256, 257, 1000, 4096, 4097, 8192, 8193, 9999, 16384, 16385, 40000, 70001])
def test_group_rows(asg, n, groups):
    say("group", n, groups)
    g = rng(10, n, groups)
    ids = g.integers(0, groups, n)
    if n > 4:
        ids[g.random(n) < 0.1] = -1
        ids[g.integers(0, n)], ids[g.integers(0, n)] = groups, 2 ** 31 - 1
    if n % 2:
        ids[ids == 0] = groups - 1                      # a group without entries
    off, rows, slots = asg.group_rows(dev(ids), groups)
    flat = np.where((ids < 0) | (ids >= groups), groups, ids)
    want = np.argsort(flat, kind="stable")
    assert np.array_equal(rows.cpu().numpy(), want)
    assert np.array_equal(off.cpu().numpy(), np.searchsorted(flat[want], np.arange(groups + 1)))
    place = np.empty(n, np.int64)
    place[want] = np.arange(n)
    assert np.array_equal(slots.cpu().numpy(), np.where(flat == groups, -1, place))


def test_group_rows_as_the_definition_says(asg):
    say("group small")
    g = rng(11)
    ids = g.integers(-1, 6, (37, 3))
    off, rows, slots = asg.group_rows(dev(ids), 5)
    want = E.group(ids, 5)
    for a, b in zip((off, rows, slots), want):
        assert a.cpu().numpy().shape == b.shape and np.array_equal(a.cpu().numpy(), b)
    torch = torch_()
    same = torch.full((4100,), 3, dtype=torch.int32, device="cuda")
    off, rows, slots = asg.group_rows(same, 8)
    assert off.tolist() == [0, 0, 0, 0, 4100, 4100, 4100, 4100, 4100] and torch.equal(rows, slots)
    off, rows, slots = asg.group_rows(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 3)
    assert off.tolist() == [0, 0, 0, 0] and rows.numel() == 0 == slots.numel()


def test_group_rows_workspace_and_many(asg):
    say("group many")
    torch = torch_()
    n, groups = 3_000_001, 33
    ids = torch.randint(-1, groups, (n,), dtype=torch.int32, device="cuda")
    from activation_sparse_gated_amd import _lib
    need = _lib.load().ffn_group_rows_workspace_bytes(n, groups)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    off, rows, slots = asg.group_rows(ids, groups, workspace=ws)
    key = torch.where(ids < 0, groups, ids)
    want = torch.sort(key, stable=True).indices
    assert torch.equal(rows.long(), want)
    assert torch.equal(off[1:].long(), torch.bincount(key, minlength=groups + 1)[:groups].cumsum(0))
    with pytest.raises(asg.FFNError):
        asg.group_rows(ids, groups, workspace=ws[: need // 512 * 256])


# ---------------------------------------------------------------- gather, combine
WIDTHS = [8, 64, 120, 128, 136, 504, 512, 520, 2048, 2056, 4104]


def places(g, m, top_k, drop=0.2):
    """Different places for the slots of m tokens, some without one."""
    s = g.permutation(m * top_k).reshape(m, top_k)
    s[g.random((m, top_k)) < drop] = -1
    if m > 2:
        s[1] = -1
        s[2, 0] = m * top_k + 5                         # no place either
    return s


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_gather(asg, d, dtype):
    torch = torch_()
    for m, top_k in ((1, 1), (3, 2), (17, 8), (70, 16), (33, 3)):
        say("gather", m, top_k, d, dtype)
        g = rng(20, m, top_k, d)
        x, slots = dev(g.normal(0, 2, (m, d)), dtype), places(g, m, top_k)
        y0 = torch.full((m * top_k, d), 7.5, dtype=x.dtype, device="cuda")
        want = E.gather(f64(x), slots, f64(y0))
        y = asg.gather_forward(x, dev(slots), y=y0)
        assert y is y0 and np.array_equal(f64(y), want)
        # 8-bit blocks: those of the rows themselves, others left
        out = asg.Fp8Tensor(torch.zeros(m * top_k, d, dtype=torch.float8_e4m3fn, device="cuda"),
                            torch.full((-(-d // 128), m * top_k), -1.0, device="cuda"), 1)
        q = asg.gather_forward(x, dev(slots), fp8=True, y=out)
        codes, scale = L.blocks(f64(x).astype(np.float32), 1)
        used = {int(slots[t, s]): t for t, s in np.ndindex(*slots.shape) if 0 <= slots[t, s] < m * top_k}
        got_q, got_s = q.q.view(torch.uint8).cpu().numpy(), q.scale.cpu().numpy()
        for p in range(m * top_k):
            if p in used:
                assert np.array_equal(got_q[p], codes[used[p]]) and np.array_equal(got_s[:, p], scale[used[p]])
            else:
                assert not got_q[p].any() and (got_s[:, p] == -1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_combine(asg, d, dtype):
    torch = torch_()
    for m, top_k in ((1, 1), (3, 2), (17, 8), (40, 16), (33, 3), (50, 5)):
        say("combine", m, top_k, d, dtype)
        g = rng(21, m, top_k, d)
        slots = places(g, m, top_k)
        y, res = dev(g.normal(0, 2, (m * top_k, d)), dtype), dev(g.normal(0, 2, (m, d)), dtype)
        named = np.zeros(m * top_k, bool)
        named[slots[(slots >= 0) & (slots < m * top_k)]] = True
        y[torch.from_numpy(~named).cuda()] = float("nan")       # rows that no slot names are not read
        w = g.normal(0, 1, (m, top_k)).astype(np.float32)
        for weights, residual in ((w, None), (w, res), (None, None), (None, res)):
            got = asg.combine_forward(y, dev(slots), None if weights is None else dev(weights), residual=residual)
            want = E.combine(f64(y), slots, weights, None if residual is None else f64(residual))
            size = E.combine(np.abs(f64(y)), slots, None if weights is None else np.abs(weights),
                             None if residual is None else np.abs(f64(residual)))
            near(f64(got), want, (top_k + 2) * 2 * U * size + half(dtype) * np.abs(want) * (1 + 1e-4) + TINY, "out")
        # without weights: the gather's gradient; in place of the residual
        assert torch.equal(asg.gather_backward(y, dev(slots)), asg.combine_forward(y, dev(slots)))
        out = asg.combine_forward(y, dev(slots), dev(w), residual=res)
        assert torch.equal(asg.combine_forward(y, dev(slots), dev(w), residual=res, out=res), out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_combine_backward(asg, d, dtype):
    torch = torch_()
    for m, top_k in ((1, 1), (3, 2), (17, 8), (40, 16), (33, 3), (50, 5)):
        say("combine backward", m, top_k, d, dtype)
        g = rng(22, m, top_k, d)
        slots = places(g, m, top_k)
        y, dout = dev(g.normal(0, 2, (m * top_k, d)), dtype), dev(g.normal(0, 1, (m, d)), dtype)
        w = g.normal(0, 1, (m, top_k)).astype(np.float32)
        for weights in (w, None):
            t = None if weights is None else dev(weights)
            dy0 = torch.full_like(y, 3.25)
            dy, dw = asg.combine_backward(y, dev(slots), t, dout, dy=dy0)
            want, wdw = E.combine_backward(f64(y), slots, weights, f64(dout), np.full(y.shape, 3.25))
            near(f64(dy), want, (U + half(dtype) * (1 + 1e-4)) * np.abs(want) + TINY, "dy")
            size = E.combine_backward(np.abs(f64(y)), slots, weights, np.abs(f64(dout)), np.zeros(y.shape))[1]
            near(f64(dw), wdw, (d / 256 + 18) * 2 * U * size, "dweights")
            one, none = asg.combine_backward(None, dev(slots), t, dout, need_dweights=False, dy=torch.full_like(y, 3.25))
            assert none is None and torch.equal(one, dy)
            none, one = asg.combine_backward(y, dev(slots), t, dout, need_dy=False)
            assert none is None and torch.equal(one, dw)
        z = y.clone()
        dy, dw2 = asg.combine_backward(z, dev(slots), t, dout, dy=z)        # in place of the rows
        assert torch.equal(dw, dw2)
        named = torch.from_numpy(np.isin(np.arange(m * top_k), slots)).cuda()
        assert torch.equal(dy[named], asg.combine_backward(y, dev(slots), t, dout)[0][named])


def test_rows_past_2_to_the_31_elements(asg):
    say("rows large")
    torch = torch_()
    m, top_k, d = 150_000, 2, 8192                      # 2.4e9 elements of y
    x = torch.randn(m, d, device="cuda", dtype=torch.bfloat16)
    slots = torch.randperm(m * top_k, device="cuda").to(torch.int32).view(m, top_k)
    y = asg.gather_forward(x, slots)
    for t in (0, 1, m // 2, m - 1):
        assert all(torch.equal(y[int(s)], x[t]) for s in slots[t])
    at = int(slots.flatten().argmax())
    assert torch.equal(y[m * top_k - 1], x[at // top_k])
    out = asg.combine_forward(y, slots, torch.full((m, top_k), 0.5, device="cuda"))
    assert torch.equal(out, x)
    dy, dw = asg.combine_backward(y, slots, torch.full((m, top_k), 2.0, device="cuda"), x, dy=y)
    assert torch.equal(dy[m * top_k - 1], 2 * x[at // top_k])


def test_without_rows(asg):
    say("no tokens")
    torch = torch_()
    x, s = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    w = torch.empty(0, 2, device="cuda")
    assert asg.route_forward(x, 2)[0].shape == (0, 2) and asg.route_backward(x, s, w).shape == (0, 64)
    assert asg.gather_forward(x, s).shape == (0, 64) and asg.gather_forward(x, s, fp8=True).q.shape == (0, 64)
    assert asg.combine_forward(x, s, w).shape == (0, 64)
    dy, dw = asg.combine_backward(x, s, w, x)
    assert dy.shape == (0, 64) and dw.shape == (0, 2)


def test_refusals(asg):
    say("refusals")
    torch = torch_()
    x, s = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    for call in (lambda: asg.route_forward(x, 0), lambda: asg.route_forward(x, 2, score="relu"),
                 lambda: asg.route_forward(x.half(), 2), lambda: asg.route_forward(x.t(), 2),
                 lambda: asg.route_forward(x, 2, bias=torch.zeros(63, device="cuda")),
                 lambda: asg.route_backward(x, s, w[:, :1]), lambda: asg.route_backward(x, s.long(), w),
                 lambda: asg.group_rows(s, 0), lambda: asg.group_rows(s.float(), 4), lambda: asg.gather_forward(x, s[:3]),
                 lambda: asg.gather_forward(x[:, ::2], s), lambda: asg.combine_forward(x, s, w),
                 lambda: asg.combine_backward(x, s, w, x), lambda: asg.combine_forward(torch.cat([x, x]), s, w.double())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: asg.route_forward(x, 65), lambda: asg.route_forward(x, 2, groups=5),
                 lambda: asg.route_forward(x, 2, groups=4, top_groups=5), lambda: asg.route_forward(x, 2, group_best=3),
                 lambda: asg.route_forward(x, 2, scale=float("nan")), lambda: asg.group_rows(s, 1025),
                 lambda: asg.gather_forward(torch.zeros(4, 12, dtype=torch.bfloat16, device="cuda"), s)):
        with pytest.raises(asg.FFNError):
            call()
