"""The operators of a decode step on 4-bit data.

Products of a few tokens with MXFP4 / NVFP4 weights (as ``mxfp4_quantize`` and
``nvfp4_quantize`` write them), and a paged key/value cache held in MXFP4: its
append, attention over it, copies of its pages and the host's bookkeeping of
them.  As in the rest of the package, this module only checks and marshals
arguments; the work is done by the library's kernels on the current stream.

Cache pages are runs of bytes whose layout ``include/mxq.h`` describes.  The
cache of a model is one uint8 tensor [layers, pages, page_bytes]
(``mxfp4_kv_cache``); the per-layer calls take ``cache[layer]``.
"""
from __future__ import annotations

import heapq
import struct

import torch

import block_scaled_precision_mxfp8_amd as _mxq

# mxq_kv_cache and mxq_kv_attention as bytes: packing them costs a fraction of
# filling a ctypes structure field by field
_CACHE = struct.Struct("@Pqqiiii")
_ATTENTION = struct.Struct("@PqqqPqPiiiifiiiPPPN")

_INT32_MAX = (1 << 31) - 1

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device: torch.device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, what: str, dtype: torch.dtype, device: torch.device):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{what} must be a {str(dtype).removeprefix('torch.')} tensor")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}")


def _as_bytes(t: torch.Tensor, what: str) -> torch.Tensor:
    """t as uint8; only types of one byte are codes or scales."""
    if isinstance(t, torch.Tensor):
        if t.dtype is torch.uint8:
            return t
        if t.dtype.itemsize == 1:
            return t.view(torch.uint8)
    raise TypeError(f"{what} must be a tensor of bytes")


def _rows16(x: torch.Tensor) -> torch.Tensor:
    """x with a unit last stride and 16-byte aligned rows (a copy if it has none)."""
    *rows, unit = x.stride()
    if unit != 1 or x.data_ptr() % 16:
        return x.clone(memory_format=torch.contiguous_format)
    for v in rows:
        if v % 8:
            return x.clone(memory_format=torch.contiguous_format)
    return x


# ---------------------------------------------------------------------------
# products with 4-bit weights
# ---------------------------------------------------------------------------

def _matvec(fn: str, x, q, s, g, group: int, out_dtype, out):
    if not isinstance(x, torch.Tensor) or x.dtype is not torch.bfloat16 or not x.is_cuda:
        _mxq._need_bf16_cuda(x)
    dev = x.device
    q, s = _as_bytes(q, "q"), _as_bytes(s, "scale")
    if q.device != dev or s.device != dev:
        raise ValueError(f"q and scale must be on {dev}")
    if q.dim() != 2 or not q.is_contiguous() or not s.is_contiguous():
        raise ValueError("q and scale must be 2-D and contiguous")
    n, half = q.shape
    k = 2 * half
    shape = x.shape
    if not shape or shape[-1] != k:
        raise ValueError(f"x has {shape[-1] if shape else 0} columns, the weights {k}")
    if k % group or s.shape != (n, k // group):
        raise ValueError(f"scale must be [{n}, {k}/{group}]")
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise TypeError("out_dtype must be bfloat16 or float32")
    x2 = x if len(shape) == 2 else x.reshape(shape[:-1].numel(), k)
    ldx, unit = x2.stride()
    xp = x2.data_ptr()
    if unit != 1 or ldx % 8 or ldx < k or xp % 16:
        x2 = x2.clone(memory_format=torch.contiguous_format)
        ldx, xp = k, x2.data_ptr()
    shape = (*shape[:-1], n)
    if out is None:
        out = x.new_empty(shape, dtype=out_dtype)
    else:
        _need(out, "out", out_dtype, dev)
        if tuple(out.shape) != shape or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous {list(shape)} tensor")
    L = _mxq._lib or _mxq.load()
    f32 = out_dtype is torch.float32
    if g is None:
        st = L.mxfp4_matvec(xp, x2.shape[0], ldx, q.data_ptr(), s.data_ptr(), n, k,
                            out.data_ptr(), n, f32, _stream_of(dev))
    else:
        st = L.nvfp4_matvec(xp, x2.shape[0], ldx, q.data_ptr(), s.data_ptr(), g.data_ptr(), n, k,
                            out.data_ptr(), n, f32, _stream_of(dev))
    if st:
        raise _mxq.MXQError(fn, st)
    return out


def mxfp4_matvec(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor,
                 out_dtype: torch.dtype = torch.bfloat16,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """x [..., k] bf16 times the transpose of the MXFP4 weights (q uint8
    [n, k/2], scale uint8 [n, k/32]): [..., n], summed in fp32, bf16 or fp32.
    Made for few rows of x: they are taken in tiles of 16, 32 or 64 (larger
    ones for larger n), each of which reads the weights."""
    return _matvec("mxfp4_matvec", x, q, scale, None, _mxq.MX_GROUP, out_dtype, out)


def nvfp4_matvec(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, g: torch.Tensor,
                 out_dtype: torch.dtype = torch.bfloat16,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """mxfp4_matvec for NVFP4 weights (q uint8 [n, k/2], s uint8 [n, k/16]
    E4M3, g float32 [1])."""
    _need(g, "g", torch.float32, x.device)
    if g.numel() != 1:
        raise ValueError("g must hold one value")
    return _matvec("nvfp4_matvec", x, q, s, g, _mxq.NV_BLOCK, out_dtype, out)


# ---------------------------------------------------------------------------
# the key/value cache
# ---------------------------------------------------------------------------

_page_bytes: dict = {}  # (kv_heads, head_dim, page_size) -> bytes


def mxfp4_kv_page_bytes(kv_heads: int, head_dim: int, page_size: int = 64) -> int:
    """Bytes of one page of one layer: page_size tokens' keys and values."""
    key = (kv_heads, head_dim, page_size)
    n = _page_bytes.get(key)
    if n is None:
        if not all(0 < v <= _INT32_MAX for v in key):  # the library's int32 would take them modulo 2^32
            raise ValueError("heads, head_dim and page_size must be positive 32-bit integers")
        n = _mxq.load().mxfp4_kv_page_bytes(kv_heads, head_dim, page_size)
        if n == 0:
            raise ValueError("the cache has head_dim 64, 96, 128, 192 or 256 and page_size a "
                             f"multiple of 16, not {head_dim} and {page_size} ({kv_heads} heads)")
        _page_bytes[key] = n
    return n


def mxfp4_kv_cache(layers: int, pages: int, kv_heads: int, head_dim: int, page_size: int = 64,
                   device="cuda") -> torch.Tensor:
    """An empty cache: uint8 [layers, pages, page_bytes]."""
    return torch.zeros((layers, pages, mxfp4_kv_page_bytes(kv_heads, head_dim, page_size)),
                       dtype=torch.uint8, device=device)


def _layer(cache: torch.Tensor, dev: torch.device, kv_heads: int, head_dim: int, page_size: int) -> bytes:
    """mxq_kv_cache of one layer."""
    if not isinstance(cache, torch.Tensor) or cache.dtype is not torch.uint8:
        raise TypeError("cache must be a uint8 tensor")
    if cache.device != dev:
        raise ValueError(f"cache must be on {dev}")
    nbytes = _page_bytes.get((kv_heads, head_dim, page_size)) or mxfp4_kv_page_bytes(kv_heads, head_dim, page_size)
    shape = cache.shape
    if len(shape) != 2 or shape[1] != nbytes or cache.stride(1) != 1:
        raise ValueError(f"cache must be one layer, [pages, {nbytes}] bytes for these heads")
    return _CACHE.pack(cache.data_ptr(), shape[0], cache.stride(0), kv_heads, head_dim, page_size, 0)


def mxfp4_kv_append(cache: torch.Tensor, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                    page_size: int = 64, fake_quant: bool = False):
    """Quantizes k and v [tokens, kv_heads, head_dim] bf16 (any token and head
    stride) to MXFP4 and stores token i at slots[i] = page * page_size +
    position (int64 [tokens]) of the layer ``cache`` [pages, page_bytes].
    Tokens whose slot is negative or past the cache are not stored; no two
    may have the same slot.  With fake_quant, returns (k, v) bf16 as the cache
    holds them."""
    _mxq._need_bf16_cuda(k, "k")
    dev = k.device
    _need(v, "v", torch.bfloat16, dev)
    _need(slots, "slots", torch.int64, dev)
    shape = k.shape
    if len(shape) != 3 or v.shape != shape:
        raise ValueError("k and v must be [tokens, kv_heads, head_dim]")
    tokens, heads, dim = shape
    if slots.shape != (tokens,):
        raise ValueError("slots must be [tokens]")
    desc = _layer(cache, dev, heads, dim, page_size)
    k, v, slots = _rows16(k), _rows16(v), slots.contiguous()
    kq = vq = None
    kp = vp = 0
    if fake_quant:
        kq, vq = k.new_empty(shape), k.new_empty(shape)
        kp, vp = kq.data_ptr(), vq.data_ptr()
    ks, vs = k.stride(), v.stride()
    st = (_mxq._lib or _mxq.load()).mxfp4_kv_append(
        desc, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], slots.data_ptr(), tokens, kp,
        vp, _stream_of(dev))
    if st:
        raise _mxq.MXQError("mxfp4_kv_append", st)
    return (kq, vq) if fake_quant else None


def mxfp4_kv_attention(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor,
                       lengths: torch.Tensor, kv_heads: int, page_size: int = 64,
                       scale: float | None = None, causal: bool = True, window: int = 0,
                       return_lse: bool = False):
    """Attention of q [seqs, tokens, q_heads, head_dim] bf16 over the layer
    ``cache`` [pages, page_bytes].

    Sequence b holds lengths[b] tokens (int32 [seqs], the new ones among them),
    token j in page page_table[b, j // page_size] (int32 [seqs, width]; entries
    outside the cache are holes).  Query t stands at lengths[b] - tokens + t; it
    sees cached positions up to its own (causal) and, with window > 0, only
    those less than window before it.  scale defaults to head_dim ** -0.5.
    Returns bf16 of q's shape and, with return_lse, the fp32 log sum of exp of
    the scores [seqs, tokens, q_heads]; a query that sees nothing gets zeros
    and -inf."""
    _mxq._need_bf16_cuda(q, "q")
    dev = q.device
    _need(page_table, "page_table", torch.int32, dev)
    _need(lengths, "lengths", torch.int32, dev)
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [seqs, tokens, q_heads, head_dim]")
    seqs, tokens, heads, dim = shape
    table_shape = page_table.shape
    if len(table_shape) != 2 or table_shape[0] != seqs:
        raise ValueError("page_table must be [seqs, width]")
    if lengths.shape != (seqs,):
        raise ValueError("lengths must be [seqs]")
    if kv_heads < 1 or heads < 1 or heads % kv_heads:
        raise ValueError("q's heads must be a multiple of kv_heads")
    if not 0 <= window <= _INT32_MAX:
        raise ValueError("window must be a 32-bit integer that is not negative")
    desc = _layer(cache, dev, kv_heads, dim, page_size)
    q = _rows16(q)
    width = table_shape[1]
    row, unit = page_table.stride()
    if unit != 1 or row < width:
        page_table = page_table.contiguous()
        row = width
    lengths = lengths.contiguous()
    out = q.new_empty(shape)
    lse = q.new_empty(shape[:3], dtype=torch.float32) if return_lse else None
    L = _mxq._lib or _mxq.load()
    nbytes = L.mxfp4_kv_attention_workspace_size(seqs, tokens, heads, kv_heads, dim, page_size, width, window)
    ws = q.new_empty((nbytes,), dtype=torch.uint8) if nbytes else None
    s0, s1, s2, _ = q.stride()
    st = L.mxfp4_kv_attention(desc, _ATTENTION.pack(
        q.data_ptr(), s0, s1, s2, page_table.data_ptr(), row, lengths.data_ptr(), seqs, tokens, heads,
        width, dim ** -0.5 if scale is None else scale, 1 if causal else 0, window, 0, out.data_ptr(),
        lse.data_ptr() if return_lse else 0, ws.data_ptr() if nbytes else 0, nbytes), _stream_of(dev))
    if st:
        raise _mxq.MXQError("mxfp4_kv_attention", st)
    return (out, lse) if return_lse else out


def mxfp4_kv_copy_pages(cache: torch.Tensor, src: torch.Tensor, dst: torch.Tensor) -> None:
    """cache[:, dst[i]] = cache[:, src[i]] for a cache [layers, pages,
    page_bytes] (or one layer [pages, page_bytes]); src and dst int32 [n].
    Pairs outside the cache are left out.  No page may be in dst twice, nor be
    in dst and, in another pair, in src."""
    if not isinstance(cache, torch.Tensor) or cache.dtype != torch.uint8:
        raise TypeError("cache must be a uint8 tensor")
    if not cache.is_cuda:
        raise ValueError("cache must live on the GPU (the library has no CPU path)")
    dev = cache.device
    _need(src, "src", torch.int32, dev)
    _need(dst, "dst", torch.int32, dev)
    if src.dim() != 1 or src.shape != dst.shape:
        raise ValueError("src and dst must be [n]")
    if cache.dim() == 2:
        layers, pages, nbytes = 1, *cache.shape
        layer_stride, page_stride, last = 0, *cache.stride()
    elif cache.dim() == 3:
        layers, pages, nbytes = cache.shape
        layer_stride, page_stride, last = cache.stride()
    else:
        raise ValueError("cache must be [layers, pages, page_bytes]")
    if last != 1:
        raise ValueError("a page must be contiguous")
    # both held until the launch: a copy let go of early gives its memory to the next one
    src, dst = src.contiguous(), dst.contiguous()
    st = (_mxq._lib or _mxq.load()).mxfp4_kv_copy_pages(
        cache.data_ptr(), layers, layer_stride, pages, page_stride, nbytes, src.data_ptr(),
        dst.data_ptr(), src.shape[0], _stream_of(dev))
    if st:
        raise _mxq.MXQError("mxfp4_kv_copy_pages", st)


class KVPagePool:
    """Which page of a cache holds what: host bookkeeping, no device work.

    Sequences are named by any hashable value and hold pages in order; forks
    share whole pages (reference counts) until compaction or release.  Every
    call hands out the lowest free pages, so the same calls give the same
    tables.  Calls that need page contents moved return (src, dst) lists for
    ``mxfp4_kv_copy_pages``; the caller copies before it uses the new pages.
    """

    def __init__(self, pages: int, page_size: int = 64):
        if pages < 0 or page_size < 1:
            raise ValueError("pages must not be negative, page_size must be positive")
        self.page_size = page_size
        self.refs = [0] * pages
        self._free = list(range(pages))  # a heap; sorted is one
        self._table: dict = {}
        self._length: dict = {}

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def __contains__(self, seq) -> bool:
        return seq in self._table

    def pages(self, seq) -> list:
        return list(self._table[seq])

    def length(self, seq) -> int:
        return self._length[seq]

    def _take(self, n: int) -> list:
        if n > len(self._free):
            raise MemoryError(f"{n} pages wanted, {len(self._free)} free")
        got = [heapq.heappop(self._free) for _ in range(n)]
        for p in got:
            self.refs[p] = 1
        return got

    def _drop(self, page: int):
        self.refs[page] -= 1
        if self.refs[page] == 0:
            heapq.heappush(self._free, page)

    def extend(self, seq, tokens: int):
        """Room for ``tokens`` more tokens of seq (a new one if unknown):
        (slots, src, dst), the slots to append them at and the page to copy
        first when the tokens begin in a page shared with a fork."""
        if tokens < 0:
            raise ValueError("tokens must not be negative")
        have, length = self._table.get(seq, []), self._length.get(seq, 0)
        end = length + tokens
        shared = tokens > 0 and length % self.page_size != 0 and self.refs[have[-1]] > 1
        new = self._take(-(-end // self.page_size) - len(have) + shared)
        src, dst = [], []
        have = list(have)
        if shared:
            src, dst = [have[-1]], [new[0]]
            self._drop(have[-1])
            have[-1] = new.pop(0)
        have += new
        self._table[seq], self._length[seq] = have, end
        size = self.page_size
        return [have[i // size] * size + i % size for i in range(length, end)], src, dst

    def fork(self, seq, new_seq) -> None:
        """new_seq begins as seq stands: all its pages are shared."""
        if new_seq in self._table:
            raise ValueError(f"{new_seq!r} is there already")
        self._table[new_seq], self._length[new_seq] = list(self._table[seq]), self._length[seq]
        for p in self._table[new_seq]:
            self.refs[p] += 1

    def truncate(self, seq, length: int) -> None:
        """Drops seq's tokens from ``length`` on (a rejected draft)."""
        if not 0 <= length <= self._length[seq]:
            raise ValueError(f"length must be 0..{self._length[seq]}")
        keep = -(-length // self.page_size)
        for p in self._table[seq][keep:]:
            self._drop(p)
        del self._table[seq][keep:]
        self._length[seq] = length

    def free(self, seq) -> None:
        self.truncate(seq, 0)
        del self._table[seq], self._length[seq]

    def compact(self):
        """Moves the highest pages in use into the lowest free ones: (src, dst)
        to copy.  Afterwards the pages in use are the first ones."""
        used = sum(r > 0 for r in self.refs)
        src = [p for p in range(used, len(self.refs)) if self.refs[p]]
        dst = [p for p in range(used) if not self.refs[p]]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        for table in self._table.values():
            table[:] = [to.get(p, p) for p in table]
        self._free = list(range(used, len(self.refs)))
        return src, dst

    def table(self, seqs, width: int | None = None, device="cpu"):
        """(page_table int32 [len(seqs), width], lengths int32 [len(seqs)]) for
        mxfp4_kv_attention; unused entries are -1."""
        rows = [self._table[s] for s in seqs]
        need = max((len(r) for r in rows), default=0)
        if width is None:
            width = need
        elif width < need:
            raise ValueError(f"a sequence holds {need} pages, width is {width}")
        table = torch.tensor([r + [-1] * (width - len(r)) for r in rows], dtype=torch.int32)
        lengths = torch.tensor([self._length[s] for s in seqs], dtype=torch.int32)
        return table.view(len(rows), width).to(device), lengths.to(device)
