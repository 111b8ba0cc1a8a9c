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
from .decode import _as_bytes, _need, _stream_of

# mxq_matmul_args as bytes
_MATMUL = struct.Struct("@PPqqPPqqqqPqqPqqqiiq")


def _on(device: torch.device):
    """Makes ``device`` current for a launch where it is not."""
    return torch.cuda.device(device)


def _codes(t, what: str, dims: int, device=None) -> torch.Tensor:
    """E4M3 codes as uint8 with a unit last stride and 16-byte aligned rows (a copy if they have none)."""
    t = _as_bytes(t, what)
    if device is None:
        if not t.is_cuda:
            raise ValueError(f"{what} must live on the GPU (the library has no CPU path)")
    elif t.device != device:
        raise ValueError(f"{what} must be on {device}")
    if t.dim() != dims:
        raise ValueError(f"{what} must have {dims} dimensions")
    *rows, unit = t.stride()
    if unit != 1 or t.data_ptr() % 16 or rows[-1] < t.shape[-1] or any(v % 16 for v in rows):
        if t.shape[-1] % 16 == 0:
            return t.clone(memory_format=torch.contiguous_format)
        # rows of their own, apart by a multiple of 16 bytes
        wide = t.new_empty((*t.shape[:-1], (t.shape[-1] + 15) // 16 * 16))[..., :t.shape[-1]]
        return wide.copy_(t)
    return t


def _scales(t, what: str, shape, mx: bool, device) -> torch.Tensor:
    if mx:
        t = _as_bytes(t, what)
        if t.device != device:
            raise ValueError(f"{what} must be on {device}")
    else:
        _need(t, what, torch.float32, device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must be {list(shape)}, not {list(t.shape)}")
    stride = t.stride()
    if stride[-1] != 1 or stride[-2] < shape[-1]:
        t = t.clone(memory_format=torch.contiguous_format)
    return t


def _out(out, shape, dtype, device) -> torch.Tensor:
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError("out_dtype must be bfloat16 or float32")
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(out, "out", dtype, device)
    if tuple(out.shape) != tuple(shape) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {list(shape)} tensor")
    return out


def _offsets(offsets, device) -> torch.Tensor:
    _need(offsets, "offsets", torch.int32, device)
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be [groups + 1]")
    return offsets.contiguous()


def _launch(fn: str, x, sx, w, sw, y, n: int, k: int, offsets=None, w_stride=0, sw_stride=0, y_stride=0):
    L = _mxq._lib or _mxq.load()
    args = _MATMUL.pack(
        x.data_ptr(), sx.data_ptr(), x.stride(0), sx.stride(0), w.data_ptr(), sw.data_ptr(),
        w.stride(-2), sw.stride(-2), w_stride, sw_stride, y.data_ptr(), n, y_stride,
        0 if offsets is None else offsets.data_ptr(), x.shape[0], n, k,
        0 if offsets is None else offsets.shape[0] - 1, y.dtype is torch.float32, 0)
    dev = x.device
    if dev.index == torch.cuda.current_device():
        st = getattr(L, fn)(args, _stream_of(dev))
    else:
        with _on(dev):
            st = getattr(L, fn)(args, _stream_of(dev))
    if st:
        raise _mxq.MXQError(fn, st)
    return y


def _matmul(fn: str, mx: bool, q, s, wq, ws, out_dtype, out, offsets=None) -> torch.Tensor:
    q = _codes(q, "q", 2)
    dev = q.device
    wq = _codes(wq, "wq", 2 if offsets is None else 3, dev)
    m, k = q.shape
    n = wq.shape[-2]
    if wq.shape[-1] != k:
        raise ValueError(f"q has {k} columns, the weights {wq.shape[-1]}")
    step, size = (32, 32) if mx else (16, 128)
    if k % step:
        raise ValueError(f"the contraction must be a multiple of {step}, not {k}")
    blocks = -(-k // size)
    s = _scales(s, "scale", (m, blocks), mx, dev)
    lead = wq.shape[:-2]
    ws = _scales(ws, "weight scale", (*lead, n if mx else -(-n // 128), blocks), mx, dev)
    if offsets is not None:
        offsets = _offsets(offsets, dev)
        if offsets.shape[0] != lead[0] + 1:
            raise ValueError(f"offsets must be [{lead[0] + 1}], one more than there are weights")
    y = _out(out, (m, n), out_dtype, dev)
    return _launch(fn, q, s, wq, ws, y, n, k, offsets, wq.stride(0) if lead else 0, ws.stride(0) if lead else 0)


def blockfp8_matmul(q: torch.Tensor, S: torch.Tensor, wq: torch.Tensor, wS: torch.Tensor,
                    out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """Tokens times the transpose of block-FP8 weights: q uint8 [m, k] with S
    float32 [m, ceil(k/128)] (``blockfp8_quantize_1x128``, ``rmsnorm_blockfp8``), wq
    uint8 [n, k] with wS float32 [ceil(n/128), ceil(k/128)] (``blockfp8_quantize``):
    [m, n], summed in fp32, bf16 or fp32.  k is a multiple of 16; codes may also be
    float8_e4m3fn.  For the gradient of the tokens pass the quantized gradient and
    wq.t().contiguous(), wS.t().contiguous()."""
    return _matmul("blockfp8_matmul", False, q, S, wq, wS, out_dtype, out)


def mxfp8_matmul(q: torch.Tensor, scale: torch.Tensor, wq: torch.Tensor, wscale: torch.Tensor,
                 out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """Tokens times the transpose of MXFP8 weights: q uint8 [m, k] with scale
    uint8 [m, k/32], wq uint8 [n, k] with wscale uint8 [n, k/32] (``quantize_rowwise``,
    or of transposed matrices ``quantize_colwise_t``): [m, n], summed in fp32, bf16 or
    fp32.  k is a multiple of 32; codes and scales may also have their float8 types."""
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
    y = _out(out, (offsets.shape[0] - 1, n, k), out_dtype, dev)
    return _launch("mxq_matmul_wgrad", dyt, dys, xt, xs, y, k, tokens, offsets, y_stride=n * k)
