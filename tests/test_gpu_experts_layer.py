"""Routing, rows and adapters as they are used together: a layer of experts
forward and backward, its 8-bit form, the sparse experts' layer behind the router,
adapters beside a shared projection for several layers of one order; captured in
graphs, on streams of their own, two at once.

Each stage is compared with its fp64 definition on what the stage before it gave
(bounds as in test_gpu_experts.py, test_gpu_adapter.py and test_gpu_linear.py).
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import experts_oracle as E
from oracle import linear_oracle as L
from tests.test_gpu_experts import B, TINY, U, dev, f64, near, rng, route_backward_slack, say, torch_

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def asg(lib):
    return lib


def layer_state(m, d, f, experts, seed):
    g = rng(seed, m, d, f)
    return dict(x=dev(g.normal(0, 1, (m, d)), "bf16"), res=dev(g.normal(0, 1, (m, d)), "bf16"),
                wr=dev(g.normal(0, d ** -0.5, (experts, d)), "bf16"), bias=dev(0.05 * g.normal(0, 1, experts)),
                w1=dev(g.normal(0, d ** -0.5, (experts, f, d)), "bf16"), w2=dev(g.normal(0, f ** -0.5, (experts, d, f)), "bf16"),
                dout=dev(g.normal(0, 1, (m, d)), "bf16"))


ROUTE = dict(score="sigmoid", groups=4, top_groups=2, group_best=2, scale=1.5)


def layer_step(asg, s, top_k=3):
    """Forward and backward of out = residual + sum of w_e W2_e relu(W1_e x): every tensor on the way."""
    experts = s["w1"].shape[0]
    logits = s["x"] @ s["wr"].T
    w, ids, _ = asg.route_forward(logits, top_k, bias=s["bias"], **ROUTE)
    off, rows, slots = asg.group_rows(ids, experts)
    xg = asg.gather_forward(s["x"], slots)
    u = asg.grouped_forward(xg, s["w1"], off)
    h = u.relu()
    y = asg.grouped_forward(h, s["w2"], off)
    out = asg.combine_forward(y, slots, w, residual=s["res"])
    dy, dw = asg.combine_backward(y, slots, w, s["dout"])
    dh, dw2 = asg.grouped_backward(h, s["w2"], dy, off)
    du = dh * (u > 0)
    dxg, dw1 = asg.grouped_backward(xg, s["w1"], du, off)
    dx = asg.gather_backward(dxg, slots)
    dl = asg.route_backward(logits, ids, dw, score=ROUTE["score"], scale=ROUTE["scale"])
    return dict(logits=logits, w=w, ids=ids, off=off, rows=rows, slots=slots, xg=xg, u=u, h=h, y=y, out=out, dy=dy, dw=dw, dh=dh,
                dw2=dw2, du=du, dxg=dxg, dw1=dw1, dx=dx, dl=dl)


@pytest.mark.parametrize("m,d,f,experts", [(1, 64, 72, 8), (7, 136, 64, 12), (300, 256, 264, 16), (1100, 128, 136, 64)])
def test_layer(asg, m, d, f, experts):
    say("expert layer", m, d, f, experts)
    s = layer_state(m, d, f, experts, 1)
    t = layer_step(asg, s)
    bias = s["bias"].cpu().numpy()
    want = E.route(f64(t["logits"]), 3, sigmoid=True, bias=bias, groups=4, top_groups=2, group_best=2, scale=1.5)
    assert np.array_equal(t["ids"].cpu().numpy(), want[1])
    big = np.abs(f64(t["logits"])).max(1, keepdims=True)
    near(f64(t["w"]), want[0], (2 * big + 40) * 2 * U * np.abs(want[0]), "weights")
    off, rows, slots = E.group(want[1], experts)
    for name, v in (("off", off), ("rows", rows), ("slots", slots)):
        assert np.array_equal(t[name].cpu().numpy(), v)
    assert np.array_equal(f64(t["xg"]), E.gather(f64(s["x"]), slots, np.zeros((m * 3, d))))
    gemm = lambda got, x, w, dim: near(f64(got), L.grouped(x, w, off, np.zeros((m * 3, dim))),  # noqa: E731
                                       (x.shape[1] + 8) * 2 * U * L.grouped(np.abs(x), np.abs(w), off, np.zeros((m * 3, dim)))
                                       + B * np.abs(L.grouped(x, w, off, np.zeros((m * 3, dim)))) * (1 + 1e-3) + TINY, "product")
    w1, w2 = f64(s["w1"]), f64(s["w2"])
    gemm(t["u"], f64(t["xg"]), w1, f)
    gemm(t["y"], f64(t["h"]), w2, d)
    y, w = f64(t["y"]), f64(t["w"])
    out, size = E.combine(y, slots, w, f64(s["res"])), E.combine(np.abs(y), slots, np.abs(w), np.abs(f64(s["res"])))
    near(f64(t["out"]), out, 5 * 2 * U * size + B * np.abs(out) * (1 + 1e-4) + TINY, "out")
    dy, dw = E.combine_backward(y, slots, w, f64(s["dout"]), np.zeros(y.shape))
    near(f64(t["dy"]), dy, (U + B * (1 + 1e-4)) * np.abs(dy) + TINY, "dy")
    near(f64(t["dw"]), dw, (d / 256 + 18) * 2 * U * E.combine_backward(np.abs(y), slots, w, np.abs(f64(s["dout"])), y)[1], "dw")
    gemm(t["dh"], f64(t["dy"]), w2.transpose(0, 2, 1), f)
    gemm(t["dxg"], f64(t["du"]), w1.transpose(0, 2, 1), d)
    for got, a, b in ((t["dw2"], t["dy"], t["h"]), (t["dw1"], t["du"], t["xg"])):
        w64 = np.zeros(tuple(got.shape))
        wd = L.grouped_backward(f64(b), w64, f64(a), off, np.zeros((m * 3, got.shape[2])))[1]
        near(f64(got), wd, (m * 3 + 8) * 2 * U * L.grouped_backward(np.abs(f64(b)), w64, np.abs(f64(a)), off, np.zeros((m * 3, got.shape[2])))[1] + TINY, "dW")
    dx = E.combine(f64(t["dxg"]), slots, None, None)
    near(f64(t["dx"]), dx, 5 * 2 * U * E.combine(np.abs(f64(t["dxg"])), slots, None, None) + B * np.abs(dx) * (1 + 1e-4) + TINY, "dx")
    dl = E.route_backward(f64(t["logits"]), want[1], f64(t["dw"]), None, sigmoid=True, scale=1.5)
    slack = route_backward_slack(f64(t["logits"]), want[1], f64(t["dw"]), None, sigmoid=True, scale=1.5)
    near(f64(t["dl"]), dl, slack + B * np.abs(dl) * (1 + 1e-4) + TINY, "dlogits")


def test_layer_of_8_bit_rows(asg):
    # 8-bit rows to the experts: gathered blocks are the blocks of the gathered rows, and the products take them
    say("expert layer 8 bits")
    torch = torch_()
    s = layer_state(200, 256, 384, 8, 2)
    t = layer_step(asg, s)
    wq = asg.fp8_quantize(s["w1"], block_rows=128)
    xq = asg.gather_forward(s["x"], t["slots"], fp8=True)
    want = asg.fp8_quantize(t["xg"])
    assert torch.equal(xq.q.view(torch.uint8), want.q.view(torch.uint8)) and torch.equal(xq.scale, want.scale)
    assert torch.equal(asg.fp8_linear(xq, wq, offsets=t["off"]), asg.fp8_linear(want, wq, offsets=t["off"]))


def test_tokens_without_experts(asg):
    # padding: tokens whose logits are all -inf have no rows, and their output is the residual
    say("padded tokens")
    torch = torch_()
    s = layer_state(20, 64, 72, 8, 3)
    logits = s["x"] @ s["wr"].T
    logits[13:] = float("-inf")
    w, ids, _ = asg.route_forward(logits, 2)
    off, rows, slots = asg.group_rows(ids, 8)
    assert int(off[-1]) == 26 and bool((ids[13:] == -1).all()) and bool((slots[13:] == -1).all()) and not w[13:].any()
    x = s["x"].clone()
    x[13:] = float("nan")                               # what padding holds does not matter
    xg = torch.full((40, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    y = torch.full((40, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    asg.gather_forward(x, slots, y=xg)
    u = asg.grouped_forward(xg, s["w1"], off)
    asg.grouped_forward(u, s["w2"], off, y=y)
    assert bool(torch.isnan(y[26:]).all())              # rows of no expert are left
    out = asg.combine_forward(y, slots, w, residual=s["res"])
    assert torch.equal(out[13:], s["res"][13:]) and bool(torch.isfinite(out).all())
    dy, dw = asg.combine_backward(y, slots, w, s["dout"], dy=torch.full_like(y, 7.0))
    assert bool((dy[26:] == 7).all()) and not dw[13:].any() and bool(torch.isfinite(dw).all())


def test_router_before_the_sparse_experts(asg):
    # the layer of sparse FFN experts takes its routing from the host: that of the router here
    say("router and sparse experts")
    from oracle import ffn_oracle as O
    from synth.moe import make_moe
    from tests.gpu_util import check_y, f32_dev, make_ffn, to_dev
    mw = make_moe(6, n_experts=4, topk=2, seed=0, d=256, f=1024, rank=32, T=64, E=64)
    experts = [make_ffn(wl, max_m=6) for wl in mw.experts]
    logits = np.full((6, 4), -9.0)
    np.put_along_axis(logits, np.asarray(mw.expert_ids), np.log(np.asarray(mw.weights, np.float64)), 1)
    w, ids, _ = asg.route_forward(dev(logits), 2)
    # the workload's own experts, in the order of its weights
    order = np.argsort(-np.asarray(mw.weights), axis=1, kind="stable")
    assert np.array_equal(np.sort(ids.cpu().numpy(), 1), np.sort(mw.expert_ids, 1))
    back = np.argsort(order, axis=1)
    w = np.take_along_axis(w.cpu().numpy(), back, 1) * np.asarray(mw.weights).sum(1, keepdims=True)
    near(w, np.asarray(mw.weights, np.float64), 1e-5)
    y = asg.moe_forward(experts, to_dev(mw.experts[0], mw.x), np.take_along_axis(ids.cpu().numpy(), back, 1), w.astype(np.float32),
                        tau=f32_dev(mw.tau))
    torch_().cuda.synchronize()
    check_y(y[:6].float().cpu().numpy().astype(np.float64), O.moe_forward(mw)["y"])


# ---------------------------------------------------------------- adapters beside projections
def adapter_state(m, d, f, r, groups, seed):
    g = rng(seed, m, d, f, r)
    bf = lambda *shape, s=1.0: dev(g.normal(0, s, shape), "bf16")  # noqa: E731
    return dict(x=bf(m, d), w_up=bf(f, d, s=d ** -0.5), w_down=bf(d, f, s=f ** -0.5), a1=bf(groups, r, d, s=d ** -0.5),
                b1=bf(groups, f, r, s=r ** -0.5), a2=bf(groups, r, f, s=f ** -0.5), b2=bf(groups, d, r, s=r ** -0.5),
                scales=dev(g.uniform(0.5, 2, groups)), ids=dev(g.integers(-1, groups, m)), dout=bf(m, d))


def adapter_step(asg, s):
    """Two projections, each with its adapters, one order for both; forward and backward."""
    groups = s["a1"].shape[0]
    off, rows, _ = asg.group_rows(s["ids"], groups)
    one = s["one"]                                      # all rows are the shared projection's
    kw = dict(rows=rows, scales=s["scales"])
    u = asg.grouped_forward(s["x"], s["w_up"][None], one)
    u = asg.adapter_forward(s["x"], s["a1"], s["b1"], off, base=u, y=u, **kw)
    h = u.relu()
    y = asg.grouped_forward(h, s["w_down"][None], one)
    y = asg.adapter_forward(h, s["a2"], s["b2"], off, base=y, y=y, **kw)
    dh, _ = asg.grouped_backward(h, s["w_down"][None], s["dout"], one, need_dw=False)
    dh, da2, db2 = asg.adapter_backward(h, s["a2"], s["b2"], s["dout"], off, base=dh, dx=dh, **kw)
    du = dh * (u > 0)
    dx, _ = asg.grouped_backward(s["x"], s["w_up"][None], du, one, need_dw=False)
    dx, da1, db1 = asg.adapter_backward(s["x"], s["a1"], s["b1"], du, off, base=dx, dx=dx, **kw)
    return u, y, dh, da2, db2, dx, da1, db1


@pytest.mark.parametrize("m,r,groups", [(5, 16, 3), (40, 8, 33), (600, 24, 4)])
def test_adapters_beside_projections(asg, m, r, groups):
    say("adapters beside projections", m, r, groups)
    torch = torch_()
    s = adapter_state(m, 136, 264, r, groups, 4)
    s["one"] = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    u, y, dh, da2, db2, dx, da1, db1 = adapter_step(asg, s)
    n = {k: f64(v) for k, v in s.items() if k != "one"}
    off, rows, _ = E.group(s["ids"].cpu().numpy(), groups)
    sc = n["scales"]

    def close(got, want, size, K):
        # the base is rounded to bf16 before the adapter's part is added, and the sum again
        near(f64(got), want, 2.1 * B * size + (K + 3 * r + 200) * 2 * U * size + TINY)
    for got, x, w, a, b, K in ((u, n["x"], n["w_up"], n["a1"], n["b1"], 136), (y, f64(u.relu()), n["w_down"], n["a2"], n["b2"], 264)):
        close(got, E.adapter(x, a, b, sc, off, rows, x @ w.T),
              E.adapter(np.abs(x), np.abs(a), np.abs(b), sc, off, rows, np.abs(x) @ np.abs(w).T), K)
    du = f64(dh * (u > 0))
    for got, da, db, x, w, a, b, g in ((dh, da2, db2, f64(u.relu()), n["w_down"], n["a2"], n["b2"], n["dout"]),
                                       (dx, da1, db1, n["x"], n["w_up"], n["a1"], n["b1"], du)):
        want = E.adapter_backward(x, a, b, sc, g, off, rows, g @ w)
        size = E.adapter_backward(*(np.abs(v) for v in (x, a, b)), sc, np.abs(g), off, rows, np.abs(g) @ np.abs(w))
        close(got, want[0], size[0], 264)
        near(f64(da), want[1], (4 * (m / 8 + 150)) * 2 * U * size[1] + TINY)
        near(f64(db), want[2], (4 * (m / 8 + 150)) * 2 * U * size[2] + TINY)


def test_adapter_beside_8_bit_products(asg):
    # the shared projection in 8 bits, its bf16 output added to in place; fp32 accumulation besides
    say("adapter beside 8 bits")
    torch = torch_()
    s = adapter_state(130, 256, 264, 16, 5, 5)
    off, rows, _ = asg.group_rows(s["ids"], 5)
    x8, w8 = asg.fp8_quantize(s["x"]), asg.fp8_quantize(s["w_up"], block_rows=128)
    for t in (torch.bfloat16, torch.float32):
        base = asg.fp8_linear(x8, w8, out_dtype=t)
        want = E.adapter(f64(s["x"]), f64(s["a1"]), f64(s["b1"]), f64(s["scales"]), off.cpu().numpy(), rows.cpu().numpy(), f64(base))
        y = asg.adapter_forward(s["x"], s["a1"], s["b1"], off, rows=rows, scales=s["scales"], base=base, y=base)
        assert y is base
        near(f64(y), want, (2 * B if t == torch.bfloat16 else 1e-5) * (np.abs(want) + 1))


# ---------------------------------------------------------------- graphs and streams
def bits(t):
    return t.contiguous().view(torch_().uint8).cpu().numpy()


def same(a, b):
    a, b = (list(v.values()) if isinstance(v, dict) else list(v) for v in (a, b))
    assert len(a) == len(b) and all(np.array_equal(bits(p), bits(q)) for p, q in zip(a, b))


def captured(step, s, other):
    """The step in two graphs, replayed with the inputs of s and other in turn, eager work between; every time as eagerly."""
    torch = torch_()
    want = [step(s), step(other)]
    want = [{k: v.clone() for k, v in (w.items() if isinstance(w, dict) else enumerate(w))} for w in want]
    live = {k: v.clone() for k, v in s.items()}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(live)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = step(live)
        graphs.append((graph, out))
    for n in range(6):
        for k, v in ((s, other)[n % 2]).items():
            live[k].copy_(v)
        for graph, _ in graphs:
            graph.replay()
        eager = step(live)
        torch.cuda.synchronize()
        for _, out in graphs:
            same(out, want[n % 2])
        same(eager, want[n % 2])


def test_layer_captured(asg):
    say("layer captured")
    # without the library's product, whose kernels choose their sums by themselves
    def step(s):
        experts = s["w1"].shape[0]
        w, ids, sc = asg.route_forward(s["logits"], 3, bias=s["bias"], scores=True, **ROUTE)
        off, rows, slots = asg.group_rows(ids, experts)
        xg = asg.gather_forward(s["x"], slots)
        y = asg.grouped_forward(xg, s["w1"], off)
        out = asg.combine_forward(y, slots, w)
        dy, dw = asg.combine_backward(y, slots, w, s["dout"])
        dxg, dw1 = asg.grouped_backward(xg, s["w1"], dy, off)
        dx = asg.gather_backward(dxg, slots)
        dl = asg.route_backward(s["logits"], ids, dw, dscores=sc, score=ROUTE["score"], scale=ROUTE["scale"])
        q = asg.gather_forward(s["x"], slots, fp8=True)
        return w, ids, sc, off, rows, slots, xg, y, out, dy, dw, dxg, dw1, dx, dl, q.q, q.scale
    both = []
    for seed in (6, 7):
        s = layer_state(130, 128, 128, 16, seed)
        s["logits"] = s["x"].float() @ s["wr"].float().T
        both.append({k: s[k] for k in ("x", "logits", "bias", "w1", "dout")})
    captured(step, *both)


@pytest.mark.parametrize("m,groups", [(30, 40), (700, 5), (4200, 1)])
def test_adapters_captured(asg, m, groups):
    say("adapters captured", m, groups)
    torch = torch_()
    both = []
    for seed in (8, 9):
        s = adapter_state(m, 136, 264, 16, groups, seed)
        s["one"] = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        both.append(s)
    captured(lambda s: adapter_step(asg, s), *both)


def test_two_streams_at_once(asg):
    say("two streams")
    torch = torch_()
    states = [layer_state(500, 256, 264, 16, 10 + i) for i in range(2)]
    adapters = []
    for i in range(2):
        adapters.append(adapter_state(520 + 100 * i, 136, 264, 32, 4, 12 + i))
        adapters[i]["one"] = torch.tensor([0, 520 + 100 * i], dtype=torch.int32, device="cuda")
    want = [(layer_step(asg, s), adapter_step(asg, a)) for s, a in zip(states, adapters)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = (layer_step(asg, states[i]), adapter_step(asg, adapters[i]))
    torch.cuda.synchronize()
    for (a, b), (c, d) in zip(got, want):
        same({k: v for k, v in a.items() if k not in ("logits",)}, {k: v for k, v in c.items() if k not in ("logits",)})
        same(b, d)


def test_a_stream_by_hand(asg):
    say("stream argument")
    torch = torch_()
    s, a = layer_state(60, 128, 136, 8, 14), adapter_state(60, 136, 264, 16, 4, 15)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    logits = s["x"].float() @ s["wr"].float().T
    torch.cuda.synchronize()
    w, ids, _ = asg.route_forward(logits, 2, stream=st)
    off, rows, slots = asg.group_rows(ids, 8, stream=st)
    xg = asg.gather_forward(s["x"], slots, stream=st)
    out = asg.combine_forward(xg, slots, w, stream=st)
    dy, dw = asg.combine_backward(xg, slots, w, s["dout"], stream=st)
    dx = asg.gather_backward(dy, slots, stream=st)
    dl = asg.route_backward(logits, ids, dw, stream=st)
    aoff, arows, _ = asg.group_rows(a["ids"], 4, stream=st)
    y = asg.adapter_forward(a["x"], a["a1"], a["b1"], aoff, rows=arows, stream=st)
    g = asg.adapter_backward(a["x"], a["a1"], a["b1"], y, aoff, rows=arows, stream=st)
    st.synchronize()
    w2, ids2, _ = asg.route_forward(logits, 2)
    off2, rows2, slots2 = asg.group_rows(ids2, 8)
    xg2 = asg.gather_forward(s["x"], slots2)
    dy2, dw2 = asg.combine_backward(xg2, slots2, w2, s["dout"])
    y2 = asg.adapter_forward(a["x"], a["a1"], a["b1"], aoff, rows=arows)
    same((w, ids, off, rows, slots, xg, out, dy, dw, dx, dl, y, *g),
         (w2, ids2, off2, rows2, slots2, xg2, asg.combine_forward(xg2, slots2, w2), dy2, dw2, asg.gather_backward(dy2, slots2),
          asg.route_backward(logits, ids2, dw2), y2, *asg.adapter_backward(a["x"], a["a1"], a["b1"], y2, aoff, rows=arows)))
    with pytest.raises(ValueError):
        asg.group_rows(a["ids"].cpu(), 4, stream=st)
