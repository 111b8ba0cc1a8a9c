"""8-bit linear layers: their norm, products and gradients.

An RMS norm that adds the residual and writes 8 bits with scales, and its
gradient; products of such tokens with block-FP8 and MXFP8 weights, dense or
grouped by expert; and MXFP8 weight gradients from what ``quantize_colwise_t``
writes.  As in the rest of the package, this module only checks and marshals
arguments; the work is done by the library's kernels on the current stream of
the operands' device.
"""
from __future__ import annotations

import struct

import torch

import block_scaled_precision_mxfp8_amd as _mxq
from .decode import _need, _stream_of

# mxq_matmul_args, mxq_rmsnorm_args and mxq_rmsnorm_backward_args as bytes: packing
# them costs a fraction of filling a ctypes structure field by field
_MATMUL = struct.Struct("@PPqqPPqqqqPqqPqqqiiq")
_RMSNORM = struct.Struct("@PPPPPPPPqqqqfiq")
_RMSNORM_BACKWARD = struct.Struct("@PPPPPPPPNqqqqqii")

_MOST_LD = 1 << 22  # bytes between rows of codes

_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(fn: str, device: torch.device, args: bytes):
    """One library call on the current stream of ``device``, made current where it is not."""
    f = getattr(_mxq._lib or _mxq.load(), fn)
    if device.index == _current_device():
        st = f(args, _stream_of(device))
    else:
        with torch.cuda.device(device):
            st = f(args, _stream_of(device))
    if st:
        raise _mxq.MXQError(fn, st)


def _codes(t, what: str, dims: int, device=None) -> torch.Tensor:
    """E4M3 codes with a unit last stride and 16-byte aligned rows no further apart than the
    kernels' 32-bit offsets reach (a copy if they have none)."""
    if not isinstance(t, torch.Tensor) or (t.dtype is not torch.uint8 and t.dtype is not torch.float8_e4m3fn):
        raise TypeError(f"{what} must be a uint8 or float8_e4m3fn tensor")
    if device is None:
        if not t.is_cuda:
            raise ValueError(f"{what} must live on the GPU (the library has no CPU path)")
    elif t.device != device:
        raise ValueError(f"{what} must be on {device}")
    stride = t.stride()
    if len(stride) != dims:
        raise ValueError(f"{what} must have {dims} dimensions")
    if stride[-1] == 1 and not t.data_ptr() & 15 and not stride[-2] & 15 and t.shape[-1] <= stride[-2] <= _MOST_LD \
            and (dims == 2 or not stride[0] & 15):
        return t
    if t.shape[-1] % 16 == 0:
        return t.clone(memory_format=torch.contiguous_format)
    # rows of their own, apart by a multiple of 16 bytes
    wide = t.new_empty((*t.shape[:-1], (t.shape[-1] + 15) // 16 * 16))[..., :t.shape[-1]]
    return wide.copy_(t)


def _scales(t, what: str, shape: tuple, mx: bool, device) -> torch.Tensor:
    if mx:
        if not isinstance(t, torch.Tensor) or (t.dtype is not torch.uint8 and t.dtype is not torch.float8_e8m0fnu):
            raise TypeError(f"{what} must be a uint8 or float8_e8m0fnu tensor")
        if t.device != device:
            raise ValueError(f"{what} must be on {device}")
    else:
        _need(t, what, torch.float32, device)
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, not {list(t.shape)}")
    stride = t.stride()
    if stride[-1] != 1 or stride[-2] < shape[-1]:
        t = t.clone(memory_format=torch.contiguous_format)
    return t


def _out(out, shape: tuple, dtype, like: torch.Tensor) -> torch.Tensor:
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError("out_dtype must be bfloat16 or float32")
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    _need(out, "out", dtype, like.device)
    if out.shape != shape or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {list(shape)} tensor")
    return out


def _offsets(offsets, device) -> torch.Tensor:
    _need(offsets, "offsets", torch.int32, device)
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be [groups + 1]")
    return offsets.contiguous()


def _launch(fn: str, dev, x, sx, w, sw, y, n: int, k: int, offsets=None, w_stride=0, sw_stride=0, y_stride=0):
    _call(fn, dev, _MATMUL.pack(
        x.data_ptr(), sx.data_ptr(), x.stride(0), sx.stride(0), w.data_ptr(), sw.data_ptr(),
        w.stride(-2), sw.stride(-2), w_stride, sw_stride, y.data_ptr(), n, y_stride,
        0 if offsets is None else offsets.data_ptr(), x.shape[0], n, k,
        0 if offsets is None else offsets.shape[0] - 1, y.dtype is torch.float32, 0))
    return y


def _matmul(fn: str, mx: bool, q, s, wq, ws, out_dtype, out, offsets=None) -> torch.Tensor:
    q = _codes(q, "q", 2)
    dev = q.device
    wq = _codes(wq, "wq", 2 if offsets is None else 3, dev)
    m, k = q.shape
    *lead, n, wk = wq.shape
    if wk != k:
        raise ValueError(f"q has {k} columns, the weights {wk}")
    step, size = (32, 32) if mx else (16, 128)
    if k % step:
        raise ValueError(f"the contraction must be a multiple of {step}, not {k}")
    blocks = -(-k // size)
    s = _scales(s, "scale", (m, blocks), mx, dev)
    ws = _scales(ws, "weight scale", (*lead, n if mx else -(-n // 128), blocks), mx, dev)
    if offsets is None:
        return _launch(fn, dev, q, s, wq, ws, _out(out, (m, n), out_dtype, q), n, k)
    offsets = _offsets(offsets, dev)
    if offsets.shape[0] != lead[0] + 1:
        raise ValueError(f"offsets must be [{lead[0] + 1}], one more than there are weights")
    return _launch(fn, dev, q, s, wq, ws, _out(out, (m, n), out_dtype, q), n, k, offsets, wq.stride(0), ws.stride(0))


def blockfp8_matmul(q: torch.Tensor, S: torch.Tensor, wq: torch.Tensor, wS: torch.Tensor,
                    out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """Tokens times the transpose of block-FP8 weights: q uint8 [m, k] with S
    float32 [m, ceil(k/128)] (``blockfp8_quantize_1x128``, ``rmsnorm_blockfp8``), wq
    uint8 [n, k] with wS float32 [ceil(n/128), ceil(k/128)] (``blockfp8_quantize``):
    [m, n], summed in fp32, bf16 or fp32.  Of 8 neighbouring products bf16 results
    drop what lies below 2^-13 of the largest, far below their rounding unless a sum
    cancels; fp32 results, which with many tokens take about twice the time, drop
    nothing.  k is a multiple of 16; codes may also be float8_e4m3fn.  For the gradient
    of the tokens pass the quantized gradient and wq.t().contiguous(),
    wS.t().contiguous()."""
    return _matmul("blockfp8_matmul", False, q, S, wq, wS, out_dtype, out)


def mxfp8_matmul(q: torch.Tensor, scale: torch.Tensor, wq: torch.Tensor, wscale: torch.Tensor,
                 out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """Tokens times the transpose of MXFP8 weights: q uint8 [m, k] with scale
    uint8 [m, k/32], wq uint8 [n, k] with wscale uint8 [n, k/32] (``quantize_rowwise``,
    or of transposed matrices ``quantize_colwise_t``): [m, n], summed in fp32, bf16 or
    fp32, as blockfp8_matmul has them.  k is a multiple of 32; codes and scales may also
    have their float8 types."""
    return _matmul("mxq_matmul", True, q, scale, wq, wscale, out_dtype, out)


def blockfp8_matmul_grouped(q: torch.Tensor, S: torch.Tensor, wq: torch.Tensor, wS: torch.Tensor,
                            offsets: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                            out: torch.Tensor | None = None) -> torch.Tensor:
    """blockfp8_matmul of tokens sorted by expert: rows offsets[g] ..
    offsets[g+1] - 1 of q (offsets int32 [groups + 1] on the GPU, not decreasing) with
    wq[g] of uint8 [groups, n, k], wS float32 [groups, ceil(n/128), ceil(k/128)].
    Rows that belong to no group are not written."""
    if not isinstance(offsets, torch.Tensor):
        raise TypeError("offsets must be an int32 tensor")
    return _matmul("blockfp8_matmul_grouped", False, q, S, wq, wS, out_dtype, out, offsets)


def mxfp8_matmul_grouped(q: torch.Tensor, scale: torch.Tensor, wq: torch.Tensor, wscale: torch.Tensor,
                         offsets: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                         out: torch.Tensor | None = None) -> torch.Tensor:
    """mxfp8_matmul of tokens sorted by expert, as blockfp8_matmul_grouped: wq
    uint8 [groups, n, k], wscale uint8 [groups, n, k/32]."""
    if not isinstance(offsets, torch.Tensor):
        raise TypeError("offsets must be an int32 tensor")
    return _matmul("mxq_matmul_grouped", True, q, scale, wq, wscale, out_dtype, out, offsets)


def mxfp8_matmul_wgrad(dyt: torch.Tensor, dys: torch.Tensor, xt: torch.Tensor, xs: torch.Tensor,
                       offsets: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                       out: torch.Tensor | None = None) -> torch.Tensor:
    """Weight gradients of layers whose tokens are sorted by expert: dyt uint8
    [n, tokens] with dys uint8 [n, ceil(tokens/32)], xt uint8 [k, tokens] with xs uint8
    [k, ceil(tokens/32)] (q_colT and s_colT of ``quantize_colwise_t``; their row
    stride, ldt, may be larger than tokens): [groups, n, k], group g summed over
    tokens offsets[g] .. offsets[g+1] - 1, zeros for an empty one.  offsets int32
    [groups + 1] on the GPU are multiples of 32, since 32 tokens share a scale (pad
    each expert's tokens with zeros to that), or the number of tokens."""
    dyt = _codes(dyt, "dyt", 2)
    dev = dyt.device
    xt = _codes(xt, "xt", 2, dev)
    n, tokens = dyt.shape
    k = xt.shape[0]
    if xt.shape[1] != tokens:
        raise ValueError(f"dyt has {tokens} tokens, xt {xt.shape[1]}")
    dys = _scales(dys, "dys", (n, -(-tokens // 32)), True, dev)
    xs = _scales(xs, "xs", (k, -(-tokens // 32)), True, dev)
    if not isinstance(offsets, torch.Tensor):
        raise TypeError("offsets must be an int32 tensor")
    offsets = _offsets(offsets, dev)
    y = _out(out, (offsets.shape[0] - 1, n, k), out_dtype, dyt)
    return _launch("mxq_matmul_wgrad", dev, dyt, dys, xt, xs, y, k, tokens, offsets, y_stride=n * k)


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------

def _rows(t, what: str, shape, device=None) -> torch.Tensor:
    """bf16 [..., cols] as 2-D with 16-byte aligned rows (a copy if it has none)."""
    if device is None:
        _mxq._need_bf16_cuda(t, what)
    else:
        _need(t, what, torch.bfloat16, device)
        if t.shape != shape:
            raise ValueError(f"{what} must be {list(shape)}, not {list(t.shape)}")
    stride = t.stride()
    if len(stride) != 2:
        if not stride:
            raise ValueError(f"{what} must be [..., cols]")
        t = t.reshape(t.shape[:-1].numel(), t.shape[-1])
        stride = t.stride()
    if stride[1] != 1 or stride[0] & 7 or stride[0] < t.shape[1] or t.data_ptr() & 15:
        t = t.clone(memory_format=torch.contiguous_format)
    return t


def _norm_weight(weight, cols: int, device) -> torch.Tensor:
    if not isinstance(weight, torch.Tensor) or (weight.dtype is not torch.bfloat16
                                                and weight.dtype is not torch.float32):
        raise TypeError("weight must be a bfloat16 or float32 tensor")
    if weight.device != device:
        raise ValueError(f"weight must be on {device}")
    if weight.shape != (cols,):
        raise ValueError(f"weight must be [{cols}]")
    if weight.stride(0) != 1 or weight.data_ptr() & 15:
        weight = weight.clone(memory_format=torch.contiguous_format)
    return weight


def _rmsnorm(fn: str, mx: bool, x, weight, residual, eps, return_rstd, return_normed):
    x2 = _rows(x, "x", None)
    dev, shape = x2.device, x.shape
    rows, cols = x2.shape
    step = 32 if mx else 8
    if cols % step:
        raise ValueError(f"x must have a multiple of {step} columns, not {cols}")
    weight = _norm_weight(weight, cols, dev)
    q = x2.new_empty((rows, cols), dtype=torch.uint8)
    if mx:
        scale = x2.new_empty((rows, cols // 32), dtype=torch.uint8)
    else:
        scale = x2.new_empty((rows, -(-cols // 128)), dtype=torch.float32)
    got = [q, scale]
    rp = ldr = hp = sp = yp = 0
    if residual is not None:
        residual = _rows(residual, "residual", shape, dev)
        h = x2.new_empty(shape)
        got.append(h)
        rp, ldr, hp = residual.data_ptr(), residual.stride(0), h.data_ptr()
    if return_rstd:
        rstd = x2.new_empty((rows,), dtype=torch.float32)
        got.append(rstd)
        sp = rstd.data_ptr()
        if not cols:
            rstd.fill_(float("nan"))  # the mean of nothing
    if return_normed:
        y = x2.new_empty(shape)
        got.append(y)
        yp = y.data_ptr()
    _call(fn, dev, _RMSNORM.pack(x2.data_ptr(), rp, weight.data_ptr(), q.data_ptr(), scale.data_ptr(), hp, yp, sp,
                                 rows, cols, x2.stride(0), ldr, eps, weight.dtype is torch.float32, 0))
    return tuple(got)


def rmsnorm_blockfp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                     eps: float = 1e-6, return_rstd: bool = False, return_normed: bool = False):
    """RMS norm of x [..., cols] bf16 (any row stride), the residual of its shape
    added first, with 1 x 128 block-FP8 output: (q uint8 [rows, cols], S float32
    [rows, ceil(cols/128)]), then, as asked for, h = bf16(x + residual) (with a
    residual), 1 / rms float32 [rows], and the normed values in bf16.  weight [cols] is
    bf16 or fp32; cols a multiple of 8, at most 16384."""
    return _rmsnorm("blockfp8_rmsnorm", False, x, weight, residual, eps, return_rstd, return_normed)


def rmsnorm_mxfp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                  eps: float = 1e-6, return_rstd: bool = False, return_normed: bool = False):
    """rmsnorm_blockfp8 with row-wise MXFP8 output (q uint8 [rows, cols], scale uint8
    [rows, cols/32]); cols a multiple of 32."""
    return _rmsnorm("mxq_rmsnorm", True, x, weight, residual, eps, return_rstd, return_normed)


def rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     dh: torch.Tensor | None = None):
    """The norm's gradient, the quantizer counted as the identity: dy, h (x, or h as
    the norm returned it) and dh (the gradient that reaches h past the norm) bf16 [...,
    cols], rstd float32 [rows] as returned: (dx bf16 of dy's shape, the gradient of x
    and of the residual alike, dweight float32 [cols])."""
    dy2 = _rows(dy, "dy", None)
    dev, shape = dy2.device, dy.shape
    rows, cols = dy2.shape
    if cols % 8:
        raise ValueError(f"dy must have a multiple of 8 columns, not {cols}")
    h = _rows(h, "h", shape, dev)
    weight = _norm_weight(weight, cols, dev)
    _need(rstd, "rstd", torch.float32, dev)
    if rstd.shape != (rows,):
        raise ValueError(f"rstd must be [{rows}]")
    if rows and rstd.stride(0) != 1:
        rstd = rstd.contiguous()
    gp = ldg = 0
    if dh is not None:
        dh = _rows(dh, "dh", shape, dev)
        gp, ldg = dh.data_ptr(), dh.stride(0)
    dx = dy2.new_empty(shape)
    dweight = dy2.new_empty((cols,), dtype=torch.float32)
    nbytes = (_mxq._lib or _mxq.load()).mxq_rmsnorm_backward_workspace_size(rows, cols)
    ws = dy2.new_empty((nbytes,), dtype=torch.uint8)
    _call("mxq_rmsnorm_backward", dev, _RMSNORM_BACKWARD.pack(
        dy2.data_ptr(), h.data_ptr(), gp, weight.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dweight.data_ptr(),
        ws.data_ptr(), nbytes, rows, cols, dy2.stride(0), h.stride(0), ldg, weight.dtype is torch.float32, 0))
    return dx, dweight
