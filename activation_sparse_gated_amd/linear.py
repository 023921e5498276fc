"""Python binding of the operators around the FFN (include/ffn_linear.h).

Argument checks and marshalling only: PyTorch provides device memory and the
current stream of the tensors' device; every step runs in the HIP kernels
behind the C ABI. Function names follow the C entry points. Tensors are
contiguous and on one GPU; what does not fit raises ValueError before anything
is launched. Outputs that are not passed in are allocated.

Every function takes `stream`, a torch.cuda.Stream of the tensors' device: the
call is then made as inside `with torch.cuda.stream(stream)`, its outputs and
scratch memory allocated there. Inputs made on other streams have to be ready
and to stay (torch.Tensor.record_stream), as for any torch operation.
"""
from __future__ import annotations

import functools
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import FFN_BF16, FFN_F32, check

_DTYPES = {torch.bfloat16: FFN_BF16, torch.float32: FFN_F32}
FP8 = torch.float8_e4m3fn
BLOCK = 128


@dataclass
class Fp8Tensor:
    """A matrix in 8-bit blocks, or one for each expert (layout in the C header):
    q float8_e4m3fn [..., m, k]; scale fp32 [..., ceil(k/128), m] (block_rows 1)
    or [..., ceil(m/128), ceil(k/128)] (block_rows 128). A value is q * scale."""
    q: torch.Tensor
    scale: torch.Tensor
    block_rows: int

    def dequantize(self) -> torch.Tensor:
        """The values in fp32 (elementary torch operations, for inspection)."""
        m, k = self.q.shape[-2:]
        s = self.scale.transpose(-1, -2) if self.block_rows == 1 else \
            self.scale.repeat_interleave(BLOCK, -2)[..., :m, :]
        return self.q.float() * s.repeat_interleave(BLOCK, -1)[..., :k]


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _scale_shape(shape, block_rows):
    *lead, m, k = shape
    return (*lead, _blocks(k), m) if block_rows == 1 else (*lead, _blocks(m), _blocks(k))


def _fail(name, t, want):
    got = type(t).__name__ if not isinstance(t, torch.Tensor) else \
        f"{t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}"
    raise ValueError(f"{name}: expected a contiguous {want}, got {got}")


def _check(name, t, dtype, shape, device):
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        _fail(name, t, f"{dtype} {tuple(shape)} on {device}")


def _first(name, t, dtypes, ndims):
    """The tensor that the others are measured by."""
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.dim() in ndims and t.is_cuda and t.is_contiguous()):
        _fail(name, t, f"GPU tensor of {' or '.join(map(str, ndims))} dimensions, {' or '.join(map(str, dtypes))}")
    if t.numel() >> 31 and any(n >> 31 for n in t.shape):
        _no_size(name, *t.shape)
    return t.device


# The C calls take sizes as int32, and ctypes cuts a larger one off without a word: `>> 31` is 0 for what fits.
def _no_size(name, *sizes):
    raise ValueError(f"{name}: sizes are 0 .. 2^31 - 1, got {', '.join(map(str, sizes))}")


def _ptr(t):
    return None if t is None else t.data_ptr()


# The handle of torch.cuda.current_stream(index), without the object around it (2 us a call): an entry that torch keeps
# to itself, so a torch that lacks it goes the long way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(index):
    return torch.cuda.current_stream(index).cuda_stream if _raw_stream is None else _raw_stream(index)


def _call(fn, device, *args):
    """The C call on the tensors' own device, on its current stream."""
    index = device.index
    if torch.cuda.current_device() != index:
        with torch.cuda.device(device):
            return _call(fn, device, *args)
    check(fn(*args, _stream_handle(index)), fn.__name__)


def _on_stream(fn):
    """Adds the `stream` argument (module docstring)."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        tensors = (a.q if isinstance(a, Fp8Tensor) else a for a in (*args, *kw.values()))
        device = next((t.device for t in tensors if isinstance(t, torch.Tensor)), None)
        if device not in (None, stream.device):
            raise ValueError(f"stream: of {stream.device}, the tensors are on {device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _again(fn, given):
    """fn once more with the arguments of its own locals(), inside their `stream`: what _on_stream does, without a
    function around every call (0.7 us each)."""
    stream = given.pop("stream")
    tensors = (a.q if isinstance(a, Fp8Tensor) else a for a in given.values())
    device = next((t.device for t in tensors if isinstance(t, torch.Tensor)), None)
    if device not in (None, stream.device):
        raise ValueError(f"stream: of {stream.device}, the tensors are on {device}")
    with torch.cuda.stream(stream):
        return fn(**given)


def _workspace(workspace, nbytes, device):
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    _check("workspace", workspace, torch.uint8, getattr(workspace, "shape", ()), device)
    return workspace


def _nbytes(t):
    return 0 if t is None else t.numel()


# ---------------------------------------------------------------- RMS norm
@_on_stream
def rmsnorm_forward(x, w, *, residual=None, eps=1e-6, fp8=False, r=None, y=None):
    """RMS norm of the rows of x + residual (ffn_rmsnorm_forward): (y, r).

    x [m, d] bf16 or fp32; w [d]; residual [m, d] or None. r is the sum, which
    the residual stream goes on with (x itself without a residual; it may be
    passed as x or residual to be written in place). y is of x's type, or with
    fp8 an Fp8Tensor of blocks of 1 x 128."""
    dev = _first("x", x, (torch.bfloat16, torch.float32), (2,))
    m, d = x.shape
    _check("w", w, x.dtype, (d,), dev)
    if residual is not None:
        _check("residual", residual, x.dtype, x.shape, dev)
        if r is None:
            r = torch.empty_like(x)
    if r is not None:
        _check("r", r, x.dtype, x.shape, dev)
    if fp8:
        if y is None:
            y = Fp8Tensor(torch.empty(m, d, dtype=FP8, device=dev),
                          torch.empty(_blocks(d), m, dtype=torch.float32, device=dev), 1)
        else:
            _check_fp8("y", y, (m, d), 1, dev)
        out, q, scale = None, y.q, y.scale
    else:
        if y is None:
            y = torch.empty_like(x)
        else:
            _check("y", y, x.dtype, x.shape, dev)
        out, q, scale = y, None, None
    _call(_lib.load().ffn_rmsnorm_forward, dev, _ptr(x), _ptr(residual), _ptr(w), _DTYPES[x.dtype], m, d,
          float(eps), _ptr(r), _ptr(out), _ptr(q), _ptr(scale))
    return y, (x if r is None else r)


@_on_stream
def rmsnorm_backward(r, w, dy, *, dr=None, eps=1e-6, need_dx=True, need_dw=True, dx=None, dw=None, accumulate=False,
                     workspace=None):
    """Gradients of the norm of the rows r (ffn_rmsnorm_backward): (dx, dw).

    dx [m, d] of r's type is the gradient of x and of the residual, dr (the
    gradient that reaches r besides) included; dw [d] is fp32, written, or added
    to with accumulate. One that is not needed (need_dx, need_dw) is not
    computed: None in its place."""
    dev = _first("r", r, (torch.bfloat16, torch.float32), (2,))
    m, d = r.shape
    _check("w", w, r.dtype, (d,), dev)
    _check("dy", dy, r.dtype, r.shape, dev)
    if dr is not None:
        _check("dr", dr, r.dtype, r.shape, dev)
    _needs(need_dx, need_dw, dx, dw, accumulate)
    if need_dx:
        if dx is None:
            dx = torch.empty_like(r)
        else:
            _check("dx", dx, r.dtype, r.shape, dev)
    lib = _lib.load()
    if need_dw:
        dw = _accumulator("dw", dw, accumulate, (d,), dev)
        workspace = _workspace(workspace, lib.ffn_rmsnorm_backward_workspace_bytes(m, d), dev)
    else:
        workspace = None                                # what adds up dw is all that takes one
    _call(lib.ffn_rmsnorm_backward, dev, _ptr(r), _ptr(w), _ptr(dy), _ptr(dr), _DTYPES[r.dtype], m, d,
          float(eps), _ptr(dx), _ptr(dw), int(bool(accumulate)), _ptr(workspace), _nbytes(workspace))
    return dx, dw


def _needs(need_dx, need_dw, dx, dw, accumulate):
    if not (need_dx or need_dw):
        raise ValueError("need_dx, need_dw: one of the gradients at least")
    if not need_dx and dx is not None:
        raise ValueError("dx: given without need_dx")
    if not need_dw and (dw is not None or accumulate):
        raise ValueError("dw, accumulate: given without need_dw")


def _accumulator(name, t, accumulate, shape, dev):
    if t is None:
        if accumulate:
            raise ValueError(f"{name}: accumulate needs the tensor that is added to")
        return torch.empty(*shape, dtype=torch.float32, device=dev)
    _check(name, t, torch.float32, shape, dev)
    return t


# ---------------------------------------------------------------- 8-bit blocks
def _check_fp8(name, t, shape, block_rows, dev):
    if not isinstance(t, Fp8Tensor) or t.block_rows != block_rows:
        raise ValueError(f"{name}: expected an Fp8Tensor of blocks of {block_rows} x {BLOCK}")
    _check(f"{name}.q", t.q, FP8, shape, dev)
    _check(f"{name}.scale", t.scale, torch.float32, _scale_shape(shape, block_rows), dev)


@_on_stream
def fp8_quantize(x, *, block_rows=1, transposed=False, out=None, out_t=None):
    """x [m, k] (or [experts, m, k]), bf16 or fp32, in 8-bit blocks of block_rows
    (1 or 128) x 128 (ffn_fp8_quantize): an Fp8Tensor, or with transposed a pair
    of it and the blocks of the transposed matrices [k, m], their rows filled
    with zeros to a multiple of 16."""
    dev = _first("x", x, (torch.bfloat16, torch.float32), (2, 3))
    if block_rows not in (1, BLOCK):
        raise ValueError(f"block_rows: 1 or {BLOCK}, got {block_rows}")
    *lead, m, k = x.shape
    shape_t = (*lead, k, (m + 15) // 16 * 16)
    if out is None:
        out = Fp8Tensor(torch.empty_like(x, dtype=FP8),
                        torch.empty(*_scale_shape(x.shape, block_rows), dtype=torch.float32, device=dev), block_rows)
    else:
        _check_fp8("out", out, x.shape, block_rows, dev)
    if transposed:
        if out_t is None:
            out_t = Fp8Tensor(torch.empty(*shape_t, dtype=FP8, device=dev),
                              torch.empty(*_scale_shape(shape_t, block_rows), dtype=torch.float32, device=dev),
                              block_rows)
        else:
            _check_fp8("out_t", out_t, shape_t, block_rows, dev)
    elif out_t is not None:
        raise ValueError("out_t: given without transposed")
    groups = lead[0] if lead else 1
    if groups:
        _call(_lib.load().ffn_fp8_quantize, dev, _ptr(x), _DTYPES[x.dtype], groups, m, k, block_rows,
              _ptr(out.q), _ptr(out.scale), _ptr(out_t.q if transposed else None),
              _ptr(out_t.scale if transposed else None))
    return (out, out_t) if transposed else out


@_on_stream
def fp8_linear(x: Fp8Tensor, w: Fp8Tensor, *, offsets=None, y=None, out_dtype=torch.bfloat16, accumulate=False,
               workspace=None):
    """y = x w^T of 8-bit blocks (ffn_fp8_linear), [m, n] in out_dtype (bf16 or fp32).

    x: blocks of 1 x 128, [m, k]. w: [n, k], blocks of 128 x 128 or 1 x 128; with
    offsets (int32 [experts + 1] on the GPU) [experts, n, k], blocks of 128 x 128:
    rows offsets[e] .. offsets[e + 1] - 1 are expert e's. accumulate adds to an
    fp32 y.

    An fp32 output is summed in fp32 from exact products. A bf16 output comes
    from the e4m3 matrix instructions, twice as fast: of every 8 consecutive k,
    products lose what lies 13 bits below the largest one, so that besides its
    rounding an output is off by up to 7 * 2^-13 of the largest product of each
    eight. Where large products cancel that can be all of it: take fp32 there."""
    if not isinstance(x, Fp8Tensor) or not isinstance(w, Fp8Tensor):
        raise ValueError("x, w: expected Fp8Tensors")
    rows = w.block_rows
    if x.block_rows != 1 or (rows != BLOCK and (rows != 1 or offsets is not None)):
        raise ValueError(f"x, w: blocks of {x.block_rows} x {BLOCK} and {rows} x {BLOCK} are not taken here")
    xq, wq = x.q, w.q
    dev = _first("x.q", xq, (FP8,), (2,))
    m, k = xq.shape
    kb = (k + 127) // 128
    _check("x.scale", x.scale, torch.float32, (kb, m), dev)
    if offsets is None:
        _first("w.q", wq, (FP8,), (2,))
        groups, n = 1, wq.shape[0]
        _check("w.q", wq, FP8, (n, k), dev)
        _check("w.scale", w.scale, torch.float32, (kb, n) if rows == 1 else ((n + 127) // 128, kb), dev)
    else:
        _first("w.q", wq, (FP8,), (3,))
        groups, n, _ = wq.shape
        _check("w.q", wq, FP8, (groups, n, k), dev)
        _check("w.scale", w.scale, torch.float32, (groups, (n + 127) // 128, kb), dev)
        _check("offsets", offsets, torch.int32, (groups + 1,), dev)
    y = _product_out(y, (m, n), out_dtype, dev, accumulate)
    lib = _lib.load()
    workspace = _workspace(workspace, lib.ffn_fp8_linear_workspace_bytes(m, n, k, groups), dev)
    _call(lib.ffn_fp8_linear, dev, xq.data_ptr(), x.scale.data_ptr(), wq.data_ptr(), w.scale.data_ptr(), rows, m, n,
          k, _ptr(offsets), groups, _ptr(y), _DTYPES[y.dtype], int(bool(accumulate)), _ptr(workspace), _nbytes(workspace))
    return y


def _product_out(y, shape, out_dtype, dev, accumulate=False):
    if y is None:
        if accumulate:
            raise ValueError("y: accumulate needs the tensor that is added to")
        if out_dtype not in _DTYPES:
            raise ValueError(f"out_dtype: bfloat16 or float32, got {out_dtype}")
        return torch.empty(*shape, dtype=out_dtype, device=dev)
    dtype = getattr(y, "dtype", None)
    if accumulate and dtype != torch.float32:
        raise ValueError("y: accumulate needs fp32")
    _check("y", y, dtype if dtype in _DTYPES else torch.bfloat16, shape, dev)
    return y


# ---------------------------------------------------------------- products by expert
@_on_stream
def grouped_forward(x, w, offsets, *, y=None, out_dtype=torch.bfloat16, workspace=None):
    """y[t] = W_e x[t] for the rows t of each expert e (ffn_grouped_forward).

    x [m, k] bf16, sorted by expert; w [experts, n, k] bf16; offsets int32
    [experts + 1] on the GPU: rows offsets[e] .. offsets[e + 1] - 1 are expert
    e's. y [m, n] in out_dtype (bf16 or fp32); rows of no expert are left as
    they were."""
    dev = _first("x", x, (torch.bfloat16,), (2,))
    _first("w", w, (torch.bfloat16,), (3,))
    m, k = x.shape
    groups, n, _ = w.shape
    _check("w", w, torch.bfloat16, (groups, n, k), dev)
    _check("offsets", offsets, torch.int32, (groups + 1,), dev)
    y = _product_out(y, (m, n), out_dtype, dev)
    lib = _lib.load()
    workspace = _workspace(workspace, lib.ffn_grouped_forward_workspace_bytes(m, n, k, groups), dev)
    _call(lib.ffn_grouped_forward, dev, _ptr(x), _ptr(w), _ptr(offsets), groups, m, n, k, _ptr(y),
          _DTYPES[y.dtype], _ptr(workspace), _nbytes(workspace))
    return y


@_on_stream
def grouped_backward(x, w, dy, offsets, *, need_dx=True, need_dw=True, dx=None, dw=None, accumulate=False,
                     workspace=None):
    """Gradients of grouped_forward (ffn_grouped_backward): (dx, dw).

    dy [m, n] bf16; dx [m, k] bf16, rows of no expert left as they were; dw
    [experts, n, k] fp32, written (zeros for an expert without rows) or added to
    with accumulate. One that is not needed (need_dx, need_dw) is not computed:
    None in its place. Without dw, x may be None, and w without dx."""
    _needs(need_dx, need_dw, dx, dw, accumulate)
    dev = _first("dy", dy, (torch.bfloat16,), (2,))
    if need_dw or x is not None:
        _first("x", x, (torch.bfloat16,), (2,))
    if need_dx or w is not None:
        _first("w", w, (torch.bfloat16,), (3,))
    m, n = dy.shape
    k = x.shape[1] if w is None else w.shape[2]
    if w is None:
        _first("offsets", offsets, (torch.int32,), (1,))
    groups = offsets.shape[0] - 1 if w is None else w.shape[0]
    if x is not None:
        _check("x", x, torch.bfloat16, (m, k), dev)
    if w is not None:
        _check("w", w, torch.bfloat16, (groups, n, k), dev)
    _check("offsets", offsets, torch.int32, (groups + 1,), dev)
    if need_dx:
        if dx is None:
            dx = torch.empty(m, k, dtype=torch.bfloat16, device=dev)
        else:
            _check("dx", dx, torch.bfloat16, (m, k), dev)
    if need_dw:
        dw = _accumulator("dw", dw, accumulate, (groups, n, k), dev)
    lib = _lib.load()
    if need_dx:
        workspace = _workspace(workspace, lib.ffn_grouped_backward_workspace_bytes(m, n, k, groups), dev)
    else:
        workspace = None                                # only dx is ever cut along its contraction
    _call(lib.ffn_grouped_backward, dev, _ptr(x), _ptr(w), _ptr(dy), _ptr(offsets), groups, m, n, k, _ptr(dx),
          _ptr(dw), int(bool(accumulate)), _ptr(workspace), _nbytes(workspace))
    return dx, dw
