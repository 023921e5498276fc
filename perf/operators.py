"""The operators around the gated FFN, as cases to time: RMS norm with the residual's addition, 8-bit blocks with a
scale each, the matrix product of such blocks, and products grouped by expert.

Layouts. A matrix held in 8 bits is float8_e4m3fn [m, k] with one fp32 scale for each block: of 128 columns of a row
(scale [ceil(k / 128), m]) or of 128 x 128 (scale [ceil(m / 128), ceil(k / 128)], one such matrix for each expert).
A block's scale is max|x| / 448, at least 2^-100; its values are x / scale rounded to nearest even.
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK = 128
FLOOR = 2.0 ** -100
BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}


# ---------------------------------------------------------------- cases
def norm(**kw):
    return dict(dict(op="norm", way="forward", m=1, d=4096, dtype=BF16, residual=True, fp8=True), **kw)


def quantize(**kw):
    return dict(dict(op="quantize", m=1, k=4096, rows=1, experts=1, transposed=True), **kw)


def product(**kw):
    return dict(dict(op="product", m=1, n=14336, k=4096, rows=BLOCK, experts=0, f32=False), **kw)


def grouped(**kw):
    return dict(dict(op="grouped", way="forward", m=16, n=14336, k=4096, experts=8, idle=0, f32=False), **kw)


def listed():
    return [
        # the norm before a quantised FFN: one token of a decode step (latency), and a prefill block
        norm(name="norm_fp8_1x4096"),
        norm(name="norm_fp8_4096x4096", m=4096),
        # the norm's gradients in training, with the residual stream's own gradient; a batch of odd length
        norm(name="norm_backward_4095x2048", way="backward", m=4095, d=2048, fp8=False),
        # a gradient of a training step for both products that take it: along its columns, and along its tokens
        quantize(name="quantize_rows_4091x8192", m=4091, k=8192),
        # a weight after an optimizer step, as the forward product and the input's gradient read it
        quantize(name="quantize_blocks_14336x4096", m=14336, rows=BLOCK),
        # the up projection of one token, the same for the ragged tokens of eight experts, and of a prefill block
        product(name="product_1x4096x14336"),
        product(name="product_experts_74x4096x14336", m=74, experts=8),
        product(name="product_4096x4096x14336", m=4096),
        # a weight's gradient: both sides in blocks of 128 tokens, summed over 4096 tokens
        product(name="product_wgrad_14336x4096x4096", m=14336, n=4096, k=4096, rows=1, f32=True),
        # a mixture-of-experts layer: a decode batch of 8 tokens with two experts each, a prefill, a training step
        grouped(name="grouped_16x4096x14336"),
        grouped(name="grouped_8192x4096x14336", m=8192),
        grouped(name="grouped_backward_4095x2048x8192", way="backward", m=4095, n=8192, k=2048, idle=1),
    ]


def _between(rng, low, high, step):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    return min(high, max(low, step * round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)))


def draw(rng):
    """One more case: another token count, widths other than the workloads', any direction and type."""
    op = rng.choice(["norm", "quantize", "product", "product", "grouped", "grouped"])
    if op == "norm":
        way = rng.choice(["forward", "forward", "backward"])
        return norm(way=way, m=_between(rng, 1, 8192, 1), d=_between(rng, 64, 8192, 8), dtype=rng.choice([BF16, BF16, F32]),
                    residual=rng.random() < 0.7, fp8=way == "forward" and rng.random() < 0.6)
    if op == "quantize":
        rows = rng.choice([1, BLOCK])
        return quantize(m=_between(rng, 1, 8192, 1), k=_between(rng, 256, 14336, 16), rows=rows,
                        experts=rng.choice([1, 1, 5]) if rows == BLOCK else 1, transposed=rng.random() < 0.6)
    m, n, k = _between(rng, 1, 8192, 1), _between(rng, 256, 14336, 8), _between(rng, 512, 14336, 16)
    if op == "product":
        rows = rng.choice([1, BLOCK, BLOCK])
        experts = rng.choice([0, 0, 3, 8]) if rows == BLOCK else 0
        c = product(m=m, n=n, k=k, rows=rows, experts=experts, f32=rows == 1 or rng.random() < 0.3)
    else:
        way = rng.choice(["forward", "backward"])
        c = grouped(way=way, m=m, n=n, k=k, experts=rng.choice([2, 5, 8, 16]), idle=rng.choice([0, 1]),
                    f32=way == "forward" and rng.random() < 0.3)
    while work(c)["flops"] > 4e11 or max(1, c["experts"]) * c["n"] * c["k"] > 3e8:
        c["m"], c["n"], c["k"] = max(1, c["m"] // 2), max(256, c["n"] // 16 * 8), max(512, c["k"] // 32 * 16)
    return c


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _activations(g, m, d, dtype):
    """Unit normal, with one channel in a hundred twenty times as large, as in trained models."""
    large = 1 + 19 * (torch.rand(d, generator=g, device="cuda") < 0.01).float()
    return (_randn(g, m, d) * large).to(dtype)


def _counts(g, m, experts, idle):
    """Tokens of each expert: uneven, the last `idle` of them without any."""
    share = torch.rand(experts - idle, generator=g, device="cuda") + 0.25
    at = torch.rand(m, generator=g, device="cuda")
    edge = (share.cumsum(0) / share.sum())[:-1]
    return torch.bincount(torch.bucketize(at, edge), minlength=experts)


def _offsets(counts):
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = dict(c)
    if c["op"] == "norm":
        t = TYPES[c["dtype"]]
        s["x"] = _activations(g, c["m"], c["d"], t)
        s["res"] = (2 * _randn(g, c["m"], c["d"])).to(t) if c["residual"] else None
        s["w"] = (1 + 0.2 * _randn(g, c["d"])).to(t)
        if c["way"] == "backward":
            s["dy"] = _randn(g, c["m"], c["d"]).to(t)
    elif c["op"] == "quantize":
        shape = (c["experts"], c["m"], c["k"]) if c["experts"] > 1 else (c["m"], c["k"])
        if c["rows"] == 1:
            s["x"] = _activations(g, c["m"], c["k"], torch.bfloat16)
        else:
            s["x"] = (_randn(g, *shape, dtype=torch.bfloat16) / math.sqrt(c["k"])).contiguous()
    elif c["op"] == "product":
        s["xq"], s["xs"] = _quantize(_activations(g, c["m"], c["k"], torch.float32), 1)
        shape = (c["experts"], c["n"], c["k"]) if c["experts"] else (c["n"], c["k"])
        w = _randn(g, *shape, dtype=torch.bfloat16)
        s["wq"], s["ws"] = _quantize(w if c["rows"] == 1 else w / math.sqrt(c["k"]), c["rows"])
        if c["experts"]:
            counts = _counts(g, c["m"], c["experts"], 0)
            s["offsets"], s["counts"] = _offsets(counts), counts.tolist()
    else:
        s["x"] = _activations(g, c["m"], c["k"], torch.bfloat16)
        s["w"] = _randn(g, c["experts"], c["n"], c["k"], dtype=torch.bfloat16) / math.sqrt(c["k"])
        counts = _counts(g, c["m"], c["experts"], c["idle"])
        s["offsets"], s["counts"] = _offsets(counts), counts.tolist()
        if c["way"] == "backward":
            s["dy"] = _randn(g, c["m"], c["n"], dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------- the plain forms
def _padded(x, rows):
    """x [..., m, k] with zeros behind its last row and column, up to whole blocks."""
    m, k = x.shape[-2:]
    return torch.nn.functional.pad(x, (0, -k % BLOCK, 0, -m % rows))


def _quantize(x, rows):
    """The 8-bit blocks of x [..., m, k] and their scales."""
    m, k = x.shape[-2:]
    p = _padded(x, rows).float()
    b = p.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, rows))      # [..., m / rows, rows, k / 128, 128]
    scale = (b.abs().amax((-3, -1), keepdim=True) / 448).clamp_min(FLOOR)
    q = (b * (1 / scale)).to(torch.float8_e4m3fn).flatten(-2).flatten(-3, -2)[..., :m, :k].contiguous()
    scale = scale.squeeze(-1).squeeze(-2)                           # [..., m / rows, k / 128]
    return q, (scale.transpose(-1, -2) if rows == 1 else scale).contiguous()


def _values(q, scale, rows):
    """What the blocks stand for, in 32 bits."""
    m, k = q.shape[-2:]
    s = scale.transpose(-1, -2) if rows == 1 else scale.repeat_interleave(rows, -2)[..., :m, :]
    return q.float() * s.repeat_interleave(BLOCK, -1)[..., :k]


def _transposed(x):
    """x [..., m, k] as [..., k, m], its rows filled with zeros to a multiple of 16."""
    return torch.nn.functional.pad(x.transpose(-1, -2), (0, -x.shape[-2] % 16))


def _norm_forward(s):
    r = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["x"].dtype)
    x = r.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["w"].float()
    return (r, *_quantize(y, 1)) if s["fp8"] else (r, y.to(r.dtype))


def _norm_backward(s):
    # x holds the rows that were normalised, res the residual stream's own gradient
    x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
    inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    h, v = x * inv, dy * w
    dx = inv * (v - h * (v * h).mean(-1, keepdim=True))
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return dx.to(s["x"].dtype), (dy * h).sum(0)


def _plain(s):
    if s["op"] == "norm":
        return _norm_forward(s) if s["way"] == "forward" else _norm_backward(s)
    if s["op"] == "quantize":
        x = s["x"]
        q, scale = _quantize(x, s["rows"])
        if not s["transposed"]:
            return q, scale
        qt, st = _quantize(_transposed(x), s["rows"])
        return q, scale, qt, st
    if s["op"] == "product":
        out = torch.float32 if s["f32"] else torch.bfloat16
        x, w = _values(s["xq"], s["xs"], 1), _values(s["wq"], s["ws"], s["rows"])
        if not s["experts"]:
            return (x @ w.T).to(out)
        return torch.cat([a @ b.T for a, b in zip(x.split(s["counts"]), w)]).to(out)
    x = s["x"].split(s["counts"])
    if s["way"] == "forward":
        return torch.cat([a.float() @ b.float().T for a, b in zip(x, s["w"])]).to(torch.float32 if s["f32"] else torch.bfloat16)
    dy = s["dy"].split(s["counts"])
    dx = torch.cat([a.float() @ b.float() for a, b in zip(dy, s["w"])]).to(torch.bfloat16)
    return dx, torch.stack([a.float().T @ b.float() for a, b in zip(dy, x)])


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import activation_sparse_gated_amd as asg
    if s["op"] == "norm":
        if s["way"] == "backward":
            return asg.rmsnorm_backward(s["x"], s["w"], s["dy"], dr=s["res"], eps=EPS)
        y, r = asg.rmsnorm_forward(s["x"], s["w"], residual=s["res"], eps=EPS, fp8=s["fp8"])
        return (r, y.q, y.scale) if s["fp8"] else (r, y)
    if s["op"] == "quantize":
        y = asg.fp8_quantize(s["x"], block_rows=s["rows"], transposed=s["transposed"])
        return (y[0].q, y[0].scale, y[1].q, y[1].scale) if s["transposed"] else (y.q, y.scale)
    out = torch.float32 if s.get("f32") else torch.bfloat16
    if s["op"] == "product":
        return asg.fp8_linear(asg.Fp8Tensor(s["xq"], s["xs"], 1), asg.Fp8Tensor(s["wq"], s["ws"], s["rows"]),
                              offsets=s.get("offsets"), out_dtype=out)
    if s["way"] == "backward":
        return asg.grouped_backward(s["x"], s["w"], s["dy"], s["offsets"])
    return asg.grouped_forward(s["x"], s["w"], s["offsets"], out_dtype=out)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "norm":
        e = 2 if c["dtype"] == BF16 else 4
        n = c["m"] * c["d"]
        if c["way"] == "backward":      # rows, their gradient and the residual stream's in; the input's and the weight's out
            return {"bytes": n * e * (3 + c["residual"]) + c["d"] * (e + 4), "flops": 10 * n}
        out = n + 4 * c["m"] * -(-c["d"] // BLOCK) if c["fp8"] else n * e
        # without a residual the rows that go on are the input itself
        return {"bytes": n * e * (3 if c["residual"] else 1) + c["d"] * e + out, "flops": 6 * n}
    if c["op"] == "quantize":
        n = c["experts"] * c["m"] * c["k"]
        return {"bytes": n * (3 + c["transposed"]), "flops": (4 if c["transposed"] and c["rows"] == 1 else 2) * n}
    out = c["m"] * c["n"] * (4 if c["f32"] else 2)
    live = min(c["m"], max(1, c["experts"] - c.get("idle", 0)))
    weights, flops = live * c["n"] * c["k"], 2 * c["m"] * c["n"] * c["k"]
    if c["op"] == "product":
        return {"bytes": c["m"] * c["k"] + weights + out, "flops": flops}
    if c["way"] == "forward":
        return {"bytes": 2 * c["m"] * c["k"] + 2 * weights + out, "flops": flops}
    # x, dy and the weights in, dx and every expert's fp32 gradient out
    return {"bytes": 2 * c["m"] * (2 * c["k"] + c["n"]) + 2 * weights + 4 * c["experts"] * c["n"] * c["k"], "flops": 2 * flops}


# ---------------------------------------------------------------- in 64 bits
def _blocks64(x, rows):
    """Each value over its block's scale, unrounded, and the scales: block after block."""
    m, k = x.shape
    q = torch.empty_like(x)
    scale = x.new_empty((-(-m // rows), -(-k // BLOCK)))
    for j in range(scale.shape[1]):
        cols = slice(j * BLOCK, min(k, (j + 1) * BLOCK))
        top = x[:, cols].abs().max(1).values
        if rows > 1:
            top = torch.stack([t.max() for t in top.split(rows)])
        scale[:, j] = torch.maximum(top / 448, torch.full_like(top, FLOOR))
        q[:, cols] = x[:, cols] / scale[:, j].repeat_interleave(rows)[:m, None]
    return q, (scale.T if rows == 1 else scale).contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        x, w = s["x"].double(), s["w"].double()
        if s["way"] == "backward":
            dy, d = s["dy"].double(), x.shape[1]
            size = ((x * x).sum(1, keepdim=True) / d + EPS).sqrt()
            along = (dy * w * x).sum(1, keepdim=True)
            dx = dy * w / size - x * along / (d * size ** 3)
            return dx if s["res"] is None else dx + s["res"].double(), (dy * x / size).sum(0)
        r = x if s["res"] is None else (x + s["res"].double()).to(s["x"].dtype).double()
        y = r / ((r * r).sum(1, keepdim=True) / r.shape[1] + EPS).sqrt() * w
        return (r, *_blocks64(y, 1)) if s["fp8"] else (r, y)
    if s["op"] == "quantize":
        xs = s["x"].double()
        xs = [xs] if xs.dim() == 2 else list(xs)
        one = [_blocks64(x, s["rows"]) for x in xs]
        if s["transposed"]:
            fill = -s["m"] % 16
            one = [a + _blocks64(torch.cat([x, x.new_zeros(fill, x.shape[1])]).T.contiguous(), s["rows"]) for a, x in zip(one, xs)]
        return tuple(one[0]) if s["x"].dim() == 2 else tuple(torch.stack(v) for v in zip(*one))
    if s["op"] == "product":
        ends = s["offsets"].tolist() if s["experts"] else [0, s["m"]]
        wq, ws = (s["wq"], s["ws"]) if s["experts"] else (s["wq"][None], s["ws"][None])
        y = torch.zeros(s["m"], s["n"], dtype=torch.float64, device="cuda")
        for e in range(len(ends) - 1):
            a, b = ends[e], ends[e + 1]
            for j in range(-(-s["k"] // BLOCK)):
                cols = slice(j * BLOCK, (j + 1) * BLOCK)
                part = s["xq"][a:b, cols].double() @ wq[e][:, cols].double().T
                of_w = ws[e][j] if s["rows"] == 1 else ws[e][:, j].repeat_interleave(BLOCK)[:s["n"]]
                y[a:b] += part * s["xs"][j, a:b, None].double() * of_w.double()
        return y
    ends = s["offsets"].tolist()
    y = torch.zeros(s["m"], s["n"], dtype=torch.float64, device="cuda")
    dx = torch.zeros(s["m"], s["k"], dtype=torch.float64, device="cuda")
    dw = []
    for e in range(s["experts"]):
        rows = slice(ends[e], ends[e + 1])
        w, x = s["w"][e].double(), s["x"][rows].double()
        if s["way"] == "forward":
            y[rows] = x @ w.T
        else:
            dy = s["dy"][rows].double()
            dx[rows] = dy @ w
            dw.append(dy.T @ x)
    return y if s["way"] == "forward" else (dx, torch.stack(dw))
