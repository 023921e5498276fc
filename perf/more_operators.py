"""Routing to experts, the rows' way to the experts and back, and low-rank adapters beside a shared projection, as cases
to time.

Routing. A token's scores are the softmax or the sigmoid of its logits; experts are chosen by score + bias, first the
best groups of experts (by the sum of a group's one or two best values), then the best experts in them, ties to the lowest
index. An expert whose logit is -inf is never chosen; a slot without an expert has id -1 and weight 0.

Rows. Grouping by expert gives offsets [experts + 1], rows (the entry at every place of the order) and slots (the place of
every entry), entries of an expert in their own order.

Adapters. y = base + scale_e (x A_e^T) B_e^T for the rows of adapter e, base for rows without one.
"""
import math

import torch

own = False

BLOCK = 128
FLOOR = 2.0 ** -100
BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}
SOFTMAX, SIGMOID = "softmax", "sigmoid"


# ---------------------------------------------------------------- cases
def route(**kw):
    return dict(dict(op="route", way="forward", m=1, experts=256, top_k=8, score=SIGMOID, bias=True, groups=8, top_groups=4,
                     best=2, renormalize=True, scale=2.5, scores=False, dtype=F32), **kw)


def dispatch(**kw):
    return dict(dict(op="dispatch", m=8, d=4096, experts=8, top_k=2, dtype=BF16, fp8=False), **kw)


def combine(**kw):
    return dict(dict(op="combine", way="forward", m=8, d=4096, top_k=2, dtype=BF16, weighted=True, residual=False), **kw)


def adapter(**kw):
    return dict(dict(op="adapter", way="forward", m=1, n=14336, k=4096, r=16, adapters=8, idle=0, without=0, ordered=False,
                     base=True, f32=False), **kw)


def listed():
    return [
        # the router of one token in a decode step (latency), and of a prefill block: 256 experts in 8 groups
        route(name="route_1x256"),
        route(name="route_8192x256", m=8192),
        # a training step's router: the gradient of the weights and of a balancing loss on all scores
        route(name="route_backward_4095x64", way="backward", m=4095, experts=64, top_k=6, score=SOFTMAX, bias=False, groups=1,
              top_groups=1, best=1, renormalize=False, scale=1.0, scores=True),
        # rows to eight experts: a decode batch, and a prefill block whose experts read 8-bit blocks
        dispatch(name="dispatch_8x4096_top2"),
        dispatch(name="dispatch_fp8_4096x4096_top2", m=4096, fp8=True),
        # back again: a decode batch with the residual stream, a prefill with many experts a token, a training step
        combine(name="combine_8x4096_top2", residual=True),
        combine(name="combine_4096x4096_top8", m=4096, top_k=8),
        combine(name="combine_backward_4095x2048_top2", way="backward", m=4095, d=2048),
        # adapters beside the up projection: one token, a decode batch of many requests in any order, a prefill, training
        adapter(name="adapter_1x4096x14336"),
        adapter(name="adapter_48x4096x14336", m=48, adapters=32, without=5),
        adapter(name="adapter_8192x4096x14336", m=8192, r=64, ordered=True),
        adapter(name="adapter_backward_4095x2048x8192", way="backward", m=4095, n=8192, k=2048, idle=1, ordered=True),
    ]


def _between(rng, low, high, step):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    return min(high, max(low, step * round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)))


def draw(rng):
    """One more case: other token counts and widths, any way of scoring, direction and type."""
    c = _drawn(rng)
    while work(c)["bytes"] > 5e8:
        c["m"] = max(1, c["m"] // 2)
        if c["op"] == "adapter":
            c["adapters"], c["without"], c["idle"] = -(-c["adapters"] // 2), min(c["without"] // 2, c["m"] - 1), 0
    return c


def _drawn(rng):
    op = rng.choice(["route", "route", "dispatch", "combine", "combine", "adapter", "adapter", "adapter"])
    way = rng.choice(["forward", "backward"])
    dtype = rng.choice([BF16, BF16, F32])
    m = _between(rng, 1, 8192, 1)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _between(rng, max(2, 8 // groups), 256 // groups, 1)
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(8, top_groups * (experts // groups)))
        return route(way=way, m=m, experts=experts, top_k=top_k, score=rng.choice([SOFTMAX, SIGMOID]), bias=rng.random() < 0.5,
                     groups=groups, top_groups=top_groups, best=rng.choice([1, 2]), renormalize=top_k > 1 and rng.random() < 0.6,
                     scale=rng.choice([1.0, 2.5]), scores=rng.random() < 0.4, dtype=rng.choice([BF16, F32]))
    if op == "dispatch":
        experts = _between(rng, 2, 256, 1)
        return dispatch(m=m, d=_between(rng, 64, 8192, 8), experts=experts, top_k=rng.randint(1, min(8, experts)), dtype=dtype,
                        fp8=rng.random() < 0.5)
    if op == "combine":
        return combine(way=way, m=m, d=_between(rng, 64, 8192, 8), top_k=rng.randint(1, 8), dtype=dtype,
                       weighted=way == "backward" or rng.random() < 0.7, residual=way == "forward" and rng.random() < 0.4)
    adapters = rng.choice([1, 3, 8, 32, 100])
    return adapter(way=way, m=m, n=_between(rng, 256, 14336, 8), k=_between(rng, 256, 8192, 8), r=rng.choice([8, 16, 24, 32, 64, 128]),
                   adapters=adapters, idle=min(adapters - 1, rng.choice([0, 1])), without=m // rng.choice([8, 20, 10 ** 6]),
                   ordered=rng.random() < 0.5, base=rng.random() < 0.7, f32=way == "forward" and rng.random() < 0.3)


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _logits(g, m, experts, dtype):
    """A router's logits: some experts liked by most tokens."""
    return (1.5 * _randn(g, m, experts) + _randn(g, experts)).to(dtype)


def _choice(g, m, experts, top_k):
    """top_k different experts for each token, uneven over the experts."""
    return _logits(g, m, experts, torch.float32).argsort(1, descending=True)[:, :top_k].to(torch.int32).contiguous()


def _order(ids, groups):
    """(offsets, rows, slots) of ids in [0, groups); -1 stands behind every group, and has no place."""
    flat = ids.flatten().long()
    key = torch.where(flat < 0, groups, flat)
    rows = torch.sort(key, stable=True).indices
    ends = (key[None, :] <= torch.arange(groups, device=key.device)[:, None]).sum(1)
    offsets = torch.cat([ends.new_zeros(1), ends])
    slots = torch.empty_like(rows)
    slots[rows] = torch.arange(rows.numel(), device=rows.device)
    slots = torch.where(flat < 0, -1, slots)
    return offsets.to(torch.int32), rows.to(torch.int32), slots.to(torch.int32).view(ids.shape)


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = dict(c)
    if c["op"] == "route":
        s["logits"] = _logits(g, c["m"], c["experts"], TYPES[c["dtype"]])
        s["b"] = 0.1 * _randn(g, c["experts"]) if c["bias"] else None
        if c["way"] == "backward":
            with torch.no_grad():                       # the choice that the forward pass made
                s["ids"] = _route_forward(s)[1]
            s["dweights"] = _randn(g, c["m"], c["top_k"])
            s["dscores"] = 0.05 * _randn(g, c["m"], c["experts"]) if c["scores"] else None
    elif c["op"] == "dispatch":
        s["x"] = _randn(g, c["m"], c["d"]).to(TYPES[c["dtype"]])
        s["ids"] = _choice(g, c["m"], c["experts"], c["top_k"])
    elif c["op"] == "combine":
        t = TYPES[c["dtype"]]
        s["slots"] = _order(_choice(g, c["m"], 16, c["top_k"]), 16)[2]
        s["y"] = _randn(g, c["m"] * c["top_k"], c["d"]).to(t)
        s["w"] = torch.rand(c["m"], c["top_k"], generator=g, device="cuda") if c["weighted"] else None
        s["res"] = _randn(g, c["m"], c["d"]).to(t) if c["residual"] else None
        if c["way"] == "backward":
            s["dout"] = _randn(g, c["m"], c["d"]).to(t)
    else:
        e, r, n, k = c["adapters"], c["r"], c["n"], c["k"]
        s["x"] = _randn(g, c["m"], k, dtype=torch.bfloat16)
        s["a"] = _randn(g, e, r, k, dtype=torch.bfloat16) / math.sqrt(k)
        s["b"] = _randn(g, e, n, r, dtype=torch.bfloat16) / math.sqrt(r)
        s["scales"] = 0.5 + torch.rand(e, generator=g, device="cuda")
        ids = torch.randint(0, e - c["idle"], (c["m"],), generator=g, device="cuda", dtype=torch.int32)
        ids[c["m"] - c["without"]:] = -1
        ids = ids[torch.randperm(c["m"], generator=g, device="cuda")]
        if c["ordered"]:                                # sequence after sequence, those without an adapter last
            ids = torch.sort(ids.remainder(e + 1)).values
            ids = torch.where(ids == e, -1, ids).to(torch.int32)
        s["offsets"], rows, _ = _order(ids, e)
        s["rows"] = None if c["ordered"] else rows
        s["most"] = max(1, int(s["offsets"].diff().max()))
        s["base_y"] = _randn(g, c["m"], n if c["way"] == "forward" else k).to(torch.float32 if c["f32"] else torch.bfloat16) if c["base"] else None
        if c["way"] == "backward":
            s["dy"] = _randn(g, c["m"], n, dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------- the plain forms
def _selection(s):
    """What experts are chosen by, in 64 bits: values close to each other are told apart."""
    l = s["logits"].double()
    if s["score"] == SOFTMAX:
        e = torch.exp(l - l.amax(1, keepdim=True))
        v = e / e.sum(1, keepdim=True)
    else:
        v = 1 / (1 + torch.exp(-l))
    if s["b"] is not None:
        v = v + s["b"].double()
    return torch.where(torch.isneginf(l), -math.inf, v)


def _route_forward(s):
    v = _selection(s)
    m, experts, groups = s["m"], s["experts"], s["groups"]
    if s["top_groups"] < groups:
        best = torch.sort(v.view(m, groups, -1), -1, descending=True).values[..., :s["best"]]
        best = torch.where(torch.isneginf(best), 0.0, best).sum(-1) + torch.where(torch.isneginf(best[..., 0]), -math.inf, 0.0)
        chosen = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        keep = torch.zeros(m, groups, dtype=torch.bool, device=v.device).scatter_(1, chosen, True)
        v = torch.where(keep.repeat_interleave(experts // groups, 1), v, -math.inf)
    order = torch.sort(v, dim=1, descending=True, stable=True)
    ids = order.indices[:, :s["top_k"]]
    live = ~torch.isneginf(order.values[:, :s["top_k"]])
    scores = _scores(s)
    w = torch.where(live, scores.gather(1, ids), 0.0)
    if s["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    w = w * s["scale"]
    ids = torch.where(live, ids, -1).to(torch.int32)
    return (w, ids, scores) if s["scores"] else (w, ids)


def _scores(s):
    l = s["logits"].float()
    if s["score"] == SIGMOID:
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route_backward(s):
    scores, ids, dw = _scores(s), s["ids"].long(), s["dweights"]
    p = scores.gather(1, ids.clamp_min(0)) * (ids >= 0)
    if s["renormalize"]:
        total = p.sum(1, keepdim=True)
        of_p = s["scale"] * (dw - (dw * p).sum(1, keepdim=True) / total) / total
    else:
        of_p = s["scale"] * dw
    grad = torch.zeros_like(scores) if s["dscores"] is None else s["dscores"].clone()
    grad.scatter_add_(1, ids.clamp_min(0), of_p * (ids >= 0))
    if s["score"] == SOFTMAX:
        dl = scores * (grad - (grad * scores).sum(1, keepdim=True))
    else:
        dl = grad * scores * (1 - scores)
    return dl.to(s["logits"].dtype)


def _blocks(x):
    """The 8-bit blocks of 1 x 128 of x [m, d] and their scales [d / 128, m]."""
    d = x.shape[1]
    b = torch.nn.functional.pad(x.float(), (0, -d % BLOCK)).unflatten(1, (-1, BLOCK))
    scale = (b.abs().amax(-1) * (1 / 448)).clamp_min(FLOOR)
    q = (b * (1 / scale)[..., None]).to(torch.float8_e4m3fn).flatten(1)[:, :d].contiguous()
    return q, scale.T.contiguous()


def _dispatch(s):
    offsets, rows, slots = _order(s["ids"], s["experts"])
    y = s["x"][rows.long() // s["top_k"]]
    return (offsets, rows, slots, *_blocks(y)) if s["fp8"] else (offsets, rows, slots, y)


def _combine(s):
    at = s["slots"].long()
    if s["way"] == "backward":
        dy = torch.empty(s["y"].shape, device=s["y"].device)
        dy[at.flatten()] = (s["w"][..., None] * s["dout"].float()[:, None]).flatten(0, 1)
        return dy.to(s["y"].dtype), (s["y"].float()[at] * s["dout"].float()[:, None]).sum(-1)
    y = s["y"].float()[at]
    out = (y if s["w"] is None else y * s["w"][..., None]).sum(1)
    if s["res"] is not None:
        out = out + s["res"].float()
    return out.to(s["y"].dtype)


def _adapter(s):
    # every adapter's rows side by side, as many places each as the most of them have; empty places go to a row behind the last
    m, e = s["m"], s["adapters"]
    place = torch.arange(s["most"], device="cuda")[None, :] + s["offsets"][:-1, None].long()
    live = place < s["offsets"][1:, None]
    place = place.clamp_max(m - 1)
    rows = place if s["rows"] is None else s["rows"].long()[place]
    x = torch.where(live[..., None], s["x"][rows].float(), 0.0)
    a, b, scale, to = s["a"].float(), s["b"].float(), s["scales"][:, None, None], torch.where(live, rows, m).flatten()
    h = torch.bmm(x, a.transpose(1, 2))
    out = torch.zeros(m + 1, s["n"] if s["way"] == "forward" else s["k"], device="cuda")
    if s["base_y"] is not None:
        out[:m] = s["base_y"]
    if s["way"] == "forward":
        out.index_add_(0, to, (scale * torch.bmm(h, b.transpose(1, 2))).flatten(0, 1))
        return out[:m].to(torch.float32 if s["f32"] else torch.bfloat16)
    dy = torch.where(live[..., None], s["dy"][rows].float(), 0.0)
    dh = scale * torch.bmm(dy, b)
    out.index_add_(0, to, torch.bmm(dh, a).flatten(0, 1))
    return out[:m].to(torch.bfloat16), torch.bmm(dh.transpose(1, 2), x), scale * torch.bmm(dy.transpose(1, 2), h)


def _plain(s):
    if s["op"] == "route":
        return _route_forward(s) if s["way"] == "forward" else _route_backward(s)
    return {"dispatch": _dispatch, "combine": _combine, "adapter": _adapter}[s["op"]](s)


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import activation_sparse_gated_amd as asg
    if s["op"] == "route":
        if s["way"] == "backward":
            return asg.route_backward(s["logits"], s["ids"], s["dweights"], dscores=s["dscores"], score=s["score"],
                                      renormalize=s["renormalize"], scale=s["scale"])
        out = asg.route_forward(s["logits"], s["top_k"], score=s["score"], bias=s["b"], groups=s["groups"],
                                top_groups=s["top_groups"], group_best=s["best"], renormalize=s["renormalize"],
                                scale=s["scale"], scores=s["scores"])
        return out if s["scores"] else out[:2]
    if s["op"] == "dispatch":
        offsets, rows, slots = asg.group_rows(s["ids"], s["experts"])
        y = asg.gather_forward(s["x"], slots, fp8=s["fp8"])
        return (offsets, rows, slots, y.q, y.scale) if s["fp8"] else (offsets, rows, slots, y)
    if s["op"] == "combine":
        if s["way"] == "backward":
            return asg.combine_backward(s["y"], s["slots"], s["w"], s["dout"])
        if s["w"] is None and s["res"] is None:
            return asg.gather_backward(s["y"], s["slots"])
        return asg.combine_forward(s["y"], s["slots"], s["w"], residual=s["res"])
    if s["way"] == "backward":
        return asg.adapter_backward(s["x"], s["a"], s["b"], s["dy"], s["offsets"], rows=s["rows"], scales=s["scales"], base=s["base_y"])
    return asg.adapter_forward(s["x"], s["a"], s["b"], s["offsets"], rows=s["rows"], scales=s["scales"], base=s["base_y"],
                               out_dtype=torch.float32 if s["f32"] else torch.bfloat16)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    m = c["m"]
    if c["op"] == "route":
        e = 2 if c["dtype"] == BF16 else 4
        n = m * c["experts"]
        if c["way"] == "backward":      # logits, choice, its gradient and the scores' in, the logits' gradient out
            return {"bytes": n * (2 * e + 4 * c["scores"]) + 8 * m * c["top_k"], "flops": 10 * n}
        return {"bytes": n * (e + 4 * c["scores"]) + 4 * c["experts"] * c["bias"] + 8 * m * c["top_k"], "flops": (6 + c["top_k"]) * n}
    if c["op"] == "dispatch":
        e = 2 if c["dtype"] == BF16 else 4
        n, row = m * c["top_k"], c["d"] + 4 * -(-c["d"] // BLOCK) if c["fp8"] else c["d"] * e
        return {"bytes": 12 * n + 4 * (c["experts"] + 1) + m * c["d"] * e + n * row, "flops": (2 if c["fp8"] else 0) * m * c["d"]}
    if c["op"] == "combine":
        e = 2 if c["dtype"] == BF16 else 4
        rows = m * c["top_k"]
        if c["way"] == "backward":      # rows, the output's gradient, slots and weights in, both gradients out
            return {"bytes": c["d"] * e * (2 * rows + m) + 12 * rows, "flops": 3 * rows * c["d"]}
        return {"bytes": c["d"] * e * (rows + m * (1 + c["residual"])) + rows * (4 + 4 * c["weighted"]), "flops": 2 * rows * c["d"]}
    live = min(m - c["without"], max(1, c["adapters"] - c["idle"]))
    weights = live * c["r"] * (c["n"] + c["k"])
    if c["way"] == "forward":
        out = m * c["n"] * (4 if c["f32"] else 2)
        return {"bytes": 2 * m * c["k"] + 2 * weights + out * (1 + c["base"]), "flops": 2 * m * c["r"] * (c["n"] + c["k"])}
    # x and dy, the adapters and the input gradient's base in, dx and every adapter's fp32 gradients out
    return {"bytes": 2 * m * (c["k"] * (2 + c["base"]) + c["n"]) + 2 * weights + 4 * c["adapters"] * c["r"] * (c["n"] + c["k"]),
            "flops": 2 * m * c["r"] * (3 * c["k"] + 2 * c["n"])}


# ---------------------------------------------------------------- in 64 bits
def _softmax64(l):
    return torch.exp(l - torch.logsumexp(l, 1, keepdim=True))


def _exact_route(s):
    l = s["logits"].double()
    p = _softmax64(l) if s["score"] == SOFTMAX else torch.exp(-torch.log1p(torch.exp(-l)))
    if s["way"] == "backward":
        live = s["ids"] >= 0
        hot = torch.zeros(s["m"], s["top_k"], s["experts"], dtype=torch.float64, device=l.device)
        hot.scatter_(2, s["ids"].long().clamp_min(0)[..., None], 1.0)
        hot *= live[..., None]
        g = s["dweights"].double()
        if s["renormalize"]:            # w_j = c p_j / P: dL/dp_j = c (g_j - sum_i g_i p_i / P) / P
            mine = (hot * p[:, None]).sum(2)
            g = (g - (g * mine).sum(1, keepdim=True) / mine.sum(1, keepdim=True)) / mine.sum(1, keepdim=True)
        g = s["scale"] * (hot * g[..., None]).sum(1)
        if s["dscores"] is not None:
            g = g + s["dscores"].double()
        return p * g - p * (p * g).sum(1, keepdim=True) if s["score"] == SOFTMAX else g * (p - p * p)
    ids = _route_forward(dict(s, scores=False))[1]      # whole numbers: chosen in 64 bits there
    w = p.gather(1, ids.long())
    w = s["scale"] * (w / w.sum(1, keepdim=True) if s["renormalize"] else w)
    return (w, ids, p) if s["scores"] else (w, ids)


def _by_adapter(s):
    """[(adapter, its rows)], those that have any."""
    ends = s["offsets"].tolist()
    every = torch.arange(s["m"], device="cuda") if s["rows"] is None else s["rows"].long()
    return [(e, every[ends[e]:ends[e + 1]]) for e in range(s["adapters"]) if ends[e + 1] > ends[e]]


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "route":
        return _exact_route(s)
    if s["op"] == "dispatch":
        flat = s["ids"].flatten().tolist()
        rows = sorted(range(len(flat)), key=lambda i: flat[i])
        slots = [0] * len(flat)
        for place, i in enumerate(rows):
            slots[i] = place
        offsets = [sum(i < e for i in flat) for e in range(s["experts"] + 1)]
        whole = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (offsets, rows, slots)]
        whole[2] = whole[2].view(s["ids"].shape)
        y = s["x"].double().repeat_interleave(s["top_k"], 0)[whole[1].long()]
        if not s["fp8"]:
            return (*whole, y)
        q, scale = torch.empty_like(y), y.new_empty(-(-s["d"] // BLOCK), y.shape[0])
        for j in range(scale.shape[0]):
            cols = slice(j * BLOCK, min(s["d"], (j + 1) * BLOCK))
            scale[j] = (y[:, cols].abs().max(1).values / 448).clamp_min(FLOOR)
            q[:, cols] = y[:, cols] / scale[j][:, None]
        return (*whole, q, scale)
    if s["op"] == "combine":
        if s["way"] == "backward":
            dout = s["dout"].double()
            dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
            dw = torch.zeros(s["m"], s["top_k"], dtype=torch.float64, device="cuda")
            for j in range(s["top_k"]):
                at = s["slots"][:, j].long()
                dy[at] = s["w"][:, j, None].double() * dout
                dw[:, j] = (s["y"][at].double() * dout).sum(1)
            return dy, dw
        out = torch.zeros(s["m"], s["d"], dtype=torch.float64, device="cuda") if s["res"] is None else s["res"].double()
        for j in range(s["top_k"]):
            y = s["y"][s["slots"][:, j].long()].double()
            out = out + (y if s["w"] is None else y * s["w"][:, j, None].double())
        return out
    dims = (s["m"], s["n"]) if s["way"] == "forward" else (s["m"], s["k"])
    out = torch.zeros(dims, dtype=torch.float64, device="cuda") if s["base_y"] is None else s["base_y"].double()
    da, db = (torch.zeros(s[v].shape, dtype=torch.float64, device="cuda") for v in "ab")
    for e, rows in _by_adapter(s):
        x, a, b = s["x"][rows].double(), s["a"][e].double(), s["b"][e].double()
        h = s["scales"][e].double() * (x @ a.T)
        if s["way"] == "forward":
            out[rows] += h @ b.T
            continue
        dy = s["dy"][rows].double()
        dh = s["scales"][e].double() * (dy @ b)
        out[rows] += dh @ a
        da[e], db[e] = dh.T @ x, dy.T @ h
    return out if s["way"] == "forward" else (out, da, db)
