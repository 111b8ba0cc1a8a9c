"""The decode operators on the GPU: products with 4-bit weights, the paged
MXFP4 key/value cache's append, attention and page copies, against plain 64-bit
forms (decode_ref.py, where the bounds are derived) and, for stored bytes, the
quantizers' oracle."""
import numpy as np
import pytest
import torch

import decode_ref as ref
from gpu_util import announce, bits16, to_dev_bf16, u8

pytestmark = pytest.mark.gpu


def bf16_bits(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)


# -- products -----------------------------------------------------------------

def weights(rng, kind, n, k):
    q = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    if kind == "mx":
        s = rng.integers(110, 134, (n, k // 32), dtype=np.uint8)
        return q, s, None, ref.fp4_values(q) * np.repeat(ref.e8m0_to_f64(s), 32, -1)
    s = rng.integers(0, 0x7F, (n, k // 16), dtype=np.uint8)
    return q, s, np.float32(0.0371), ref.fp4_values(q) * np.repeat(ref.e4m3_to_f64(s), 16, -1)


def product(gpu, kind, x, q, s, g, dtype):
    dev = [torch.from_numpy(a).cuda() for a in (q, s)]
    if kind == "mx":
        return gpu.mxfp4_matvec(x, *dev, out_dtype=dtype)
    return gpu.nvfp4_matvec(x, *dev, torch.tensor([g], device="cuda"), out_dtype=dtype)


@pytest.mark.parametrize("kind", ["mx", "nv"])
@pytest.mark.parametrize("tokens,n,k", [
    (1, 1, 32), (1, 16, 128), (1, 17, 96), (2, 100, 256), (3, 33, 288), (16, 64, 512), (17, 48, 544),
    (31, 40, 2048), (33, 130, 1056), (64, 64, 4096), (65, 20, 160), (130, 33, 96), (1, 257, 7168), (5, 4097, 320),
    (1, 3, 2080), (48, 1000, 2336), (1, 40, 16384), (9, 4100, 2080), (64, 2050, 1184), (4, 40, 8192), (4, 33, 9376), (3, 70, 544),
    (20, 8200, 1184), (7, 8195, 672), (40, 8208, 672), (24, 4160, 288),
])
def test_matvec(gpu, kind, tokens, n, k):
    announce(f"matvec {kind} {tokens}x{n}x{k}")
    rng = np.random.default_rng(tokens * 1000003 + n * 101 + k)
    if kind == "nv":
        k += 16  # rows of NVFP4 end inside a run of 32
    q, s, g, w = weights(rng, kind, n, k)
    xb = bf16_bits(rng.standard_normal((tokens, k)))
    for dtype in (torch.float32, torch.bfloat16):
        got = product(gpu, kind, to_dev_bf16(xb), q, s, g, dtype)
        assert got.dtype == dtype and got.shape == (tokens, n)
        want, bound = ref.matvec(ref.bf16_to_f64(xb), w, 1.0 if g is None else float(g), dtype is torch.float32)
        ref.assert_within(f"{kind} {dtype}", got.float().cpu().numpy(), want, bound)
    again = product(gpu, kind, to_dev_bf16(xb), q, s, g, torch.float32)
    one = product(gpu, kind, to_dev_bf16(xb), q, s, g, torch.float32)
    assert torch.equal(again, one)


@pytest.mark.parametrize("kind", ["mx", "nv"])
@pytest.mark.parametrize("tokens, n, k", [(15, 8207, 416), (17, 2101, 1184), (33, 4000, 416), (50, 8000, 160),
                                          (30, 9001, 416), (70, 9001, 1184)])
def test_matvec_tiles(gpu, kind, tokens, n, k):
    """Enough rows for each size of tile that a workgroup may take."""
    announce(f"matvec tiles {kind} {tokens}x{n}x{k}")
    rng = np.random.default_rng(tokens + n)
    q, s, g, w = weights(rng, kind, n, k)
    xb = bf16_bits(rng.standard_normal((tokens, k)))
    got = product(gpu, kind, to_dev_bf16(xb), q, s, g, torch.float32)
    want, bound = ref.matvec(ref.bf16_to_f64(xb), w, 1.0 if g is None else float(g))
    ref.assert_within(kind, got.cpu().numpy(), want, bound)


@pytest.mark.parametrize("kind", ["mx", "nv"])
def test_matvec_strides_and_shapes(gpu, kind):
    """Leading dimensions, padded and misaligned rows, one row of a batch, no rows, no columns."""
    announce(f"matvec strides {kind}")
    rng = np.random.default_rng(7)
    n, k = 50, 224
    q, s, g, w = weights(rng, kind, n, k)
    wide = torch.from_numpy(rng.standard_normal((2, 3, k + 24)).astype(np.float32)).bfloat16().cuda()
    for x in (wide[..., :k], wide[..., 8:8 + k], wide[..., 3:3 + k], wide[:, 1, :k], wide[0, 0, :k], wide[:1, 2, 1:1 + k],
              wide[..., :k].transpose(0, 1), wide[:, :0, :k], wide[:, 0, :1].expand(2, k)):
        got = product(gpu, kind, x, q, s, g, torch.float32)
        assert got.shape == (*x.shape[:-1], n)
        want, bound = ref.matvec(x.double().cpu().numpy().reshape(-1, k), w, 1.0 if g is None else float(g))
        ref.assert_within(str(tuple(x.stride())), got.cpu().numpy().reshape(-1, n), want, bound)
    x = torch.ones(4, 0, dtype=torch.bfloat16, device="cuda")
    got = product(gpu, kind, x, q[:, :0], s[:, :0], g, torch.bfloat16)
    assert got.shape == (4, n) and not got.any()
    got = product(gpu, kind, wide[0, :, :k], q[:0], s[:0], g, torch.bfloat16)
    assert got.shape == (3, 0)


def test_matvec_writes_only_its_output(gpu):
    announce("matvec guard")
    rng = np.random.default_rng(8)
    for tokens, n in ((3, 21), (40, 70), (64, 33)):
        q, s, _, w = weights(rng, "mx", n, 320)
        xb = bf16_bits(rng.standard_normal((tokens, 320)))
        for dtype in (torch.float32, torch.bfloat16):
            buf = torch.full((tokens + 2, n), 7.0, dtype=dtype, device="cuda")
            out = buf[1:-1]
            got = gpu.mxfp4_matvec(to_dev_bf16(xb), torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), out_dtype=dtype, out=out)
            assert got is out and (buf[0] == 7).all() and (buf[-1] == 7).all()
            want, bound = ref.matvec(ref.bf16_to_f64(xb), w, out_f32=dtype is torch.float32)
            ref.assert_within("out=", out.float().cpu().numpy(), want, bound)


@pytest.mark.parametrize("kind", ["mx", "nv"])
@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_matvec_nan_and_inf(gpu, kind, tokens):
    """A NaN scale spoils its row, NaN and Inf of x their token; nothing spreads."""
    announce(f"matvec nan {kind} {tokens}")
    rng = np.random.default_rng(9)
    n, k = 40, 416
    q, s, g, _ = weights(rng, kind, n, k)
    q |= 0x11  # no zero codes: Inf times 0 is another matter
    q &= 0x77  # and no signs: Inf minus Inf as well
    s[13, 3] = 0xFF if kind == "mx" else 0x7F
    s[39, -1] = 0xFF if kind == "mx" else 0xFF
    if kind == "mx":
        s[2, 1], s[3, :] = 0, 0  # 2^-127
    w = ref.fp4_values(q) * (np.repeat(ref.e8m0_to_f64(s), 32, -1) if kind == "mx" else np.repeat(ref.e4m3_to_f64(s), 16, -1))
    x = np.abs(rng.standard_normal((tokens, k))).astype(np.float32)
    x[0, 411] = np.inf
    if tokens > 1:
        x[2, 7], x[4, 200] = np.nan, -np.inf
    xb = bf16_bits(x)
    got = product(gpu, kind, to_dev_bf16(xb), q, s, g, torch.float32)
    want, bound = ref.matvec(ref.bf16_to_f64(xb), w, 1.0 if g is None else float(g))
    if kind == "mx":  # products with 2^-127 weights may count as zero
        bound = bound + 1e-30
    ref.assert_within("nan", got.cpu().numpy(), want, bound)


def test_matvec_of_quantized_weights(gpu):
    """The quantizers' outputs feed the products as they are, typed views too."""
    announce("matvec of quantizer outputs")
    rng = np.random.default_rng(10)
    w = to_dev_bf16(bf16_bits(0.02 * rng.standard_normal((130, 1024))))
    xb = bf16_bits(rng.standard_normal((6, 1024)))
    x = to_dev_bf16(xb)
    q, s = gpu.mxfp4_quantize(w)
    want, bound = ref.matvec(ref.bf16_to_f64(xb), gpu.mxfp4_dequantize(q, s).double().cpu().numpy())
    ref.assert_within("mx", gpu.mxfp4_matvec(x, q, s, out_dtype=torch.float32).cpu().numpy(), want, bound)
    typed = gpu.mxfp4_matvec(x, q, s.view(torch.float8_e8m0fnu), out_dtype=torch.float32)
    ref.assert_within("mx typed", typed.cpu().numpy(), want, bound)
    q, s, g = gpu.nvfp4_quantize(w)
    values = ref.fp4_values(u8(q)) * np.repeat(ref.e4m3_to_f64(u8(s)), 16, -1)
    want, bound = ref.matvec(ref.bf16_to_f64(xb), values, float(g))
    ref.assert_within("nv", gpu.nvfp4_matvec(x, q, s, g, out_dtype=torch.float32).cpu().numpy(), want, bound)


def test_matvec_past_32_bits(gpu):
    """Rows of weights whose bytes lie past 2^31 and elements past 2^32."""
    announce("matvec past 32 bits")
    n, k = 640000, 8192  # 2.6 GB of codes, 5.2 G weights
    q = torch.zeros((n, k // 2), dtype=torch.uint8, device="cuda")
    s = torch.full((n, k // 32), 127, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(11)
    rows = np.array([0, 1, 524287, 524288, 600001, n - 1])
    part, ps, _, w = weights(rng, "mx", len(rows), k)
    at = torch.from_numpy(rows).cuda()
    q[at], s[at] = torch.from_numpy(part).cuda(), torch.from_numpy(ps).cuda()
    xb = bf16_bits(rng.standard_normal((2, k)))
    got = gpu.mxfp4_matvec(to_dev_bf16(xb), q, s, out_dtype=torch.float32)
    want, bound = ref.matvec(ref.bf16_to_f64(xb), w)
    ref.assert_within("rows", got[:, at].cpu().numpy(), want, bound)
    got[:, at] = 0
    assert not got.any()


# -- the cache ------------------------------------------------------------------

GEOS = [(1, 64, 16), (2, 96, 48), (3, 128, 64), (2, 192, 32), (1, 256, 16)]


@pytest.mark.parametrize("geo", GEOS, ids=str)
@pytest.mark.parametrize("tokens", [1, 15, 16, 70, 200])
def test_append(gpu, orc, geo, tokens):
    """Bytes and values as the MXFP4 quantizer's oracle says, at their places; the rest untouched."""
    heads, dim, page = geo
    announce(f"append {geo} {tokens}")
    rng = np.random.default_rng(tokens + dim)
    pages = 20
    xb = bf16_bits(rng.standard_normal((tokens, (2 * heads + 1) * dim)) * np.exp2(rng.integers(-3, 4, (tokens, 1))))
    xb[0, :32] = 0
    xb[tokens // 2, 40:42] = 0x7FC0, 0xFF80  # NaN and -Inf
    xb[-1, -5] = 0x7F80
    x = to_dev_bf16(xb)
    k, v = x[:, :heads * dim].view(tokens, heads, dim), x[:, heads * dim:2 * heads * dim].view(tokens, heads, dim)
    for kind in ("runs", "scattered"):
        slots = rng.permutation(pages * page)[:tokens] if kind == "scattered" else (np.arange(tokens) + 5)
        slots = slots.astype(np.int64)
        if tokens > 3:
            slots[1], slots[3] = -1, pages * page + 2
        before = rng.integers(0, 256, (pages + 2, ref.page_bytes(heads, dim, page)), dtype=np.uint8)
        buf = torch.from_numpy(before).cuda()
        for fq in (False, True):
            got = gpu.mxfp4_kv_append(buf[1:-1], k, v, torch.from_numpy(slots).cuda(), page, fake_quant=fq)
            want = before.copy()
            kq, ks = orc.mxfp4_quantize(bits16(k).reshape(-1, dim))
            vq, vs = orc.mxfp4_quantize(bits16(v).reshape(-1, dim))
            ref.write_page_tokens(want[1:-1], geo, slots, *(a.reshape(tokens, heads, -1) for a in (kq, ks, vq, vs)))
            assert np.array_equal(u8(buf), want), kind
            if fq:
                for a, c, s in ((got[0], kq, ks), (got[1], vq, vs)):
                    assert np.array_equal(bits16(a).reshape(-1, dim), orc.mxfp4_dequantize(c, s))
            else:
                assert got is None


@pytest.mark.parametrize("geo", [(16, 64, 16), (32, 96, 48), (16, 128, 64), (16, 192, 32), (16, 256, 16)], ids=str)
def test_append_long_runs(gpu, orc, geo):
    """A prompt of several sequences: runs that begin and end inside blocks of 16, with gaps."""
    heads, dim, page = geo
    announce(f"append long runs {geo}")
    rng = np.random.default_rng(dim)
    tokens = 32768 // heads + 37
    pages = tokens // page + 40
    slots, where = [], 0
    order = rng.permutation(pages)
    while len(slots) < tokens:
        run = int(rng.integers(1, 400))
        first = where * page + int(rng.integers(0, page))
        place = np.arange(first, first + run)
        place = order[place // page % pages] * page + place % page
        slots += place.tolist()
        where += -(-(first % page + run) // page)
        if where >= pages - 400 // page - 2:
            where = 0
    slots = np.array(slots[:tokens], np.int64)
    seen, keep = set(), np.ones(tokens, bool)
    for i, v in enumerate(slots.tolist()):
        keep[i] = v not in seen
        seen.add(v)
    slots[~keep] = -1  # a place is used once
    xb = bf16_bits(rng.standard_normal((tokens, 2 * heads, dim)))
    x = to_dev_bf16(xb)
    cache = gpu.mxfp4_kv_cache(1, pages, heads, dim, page)[0]
    gpu.mxfp4_kv_append(cache, x[:, :heads], x[:, heads:], torch.from_numpy(slots).cuda(), page)
    want = np.zeros(cache.shape, np.uint8)
    q, s = orc.mxfp4_quantize(xb.reshape(-1, dim))
    q, s = q.reshape(tokens, 2 * heads, -1), s.reshape(tokens, 2 * heads, -1)
    ref.write_page_tokens(want, geo, slots, q[:, :heads], s[:, :heads], q[:, heads:], s[:, heads:])
    assert np.array_equal(u8(cache), want)


def test_append_nothing_and_strides(gpu, orc):
    announce("append nothing, odd strides")
    heads, dim, page = 2, 64, 16
    cache = gpu.mxfp4_kv_cache(1, 3, heads, dim, page)[0]
    x = torch.randn(4, dim, heads, device="cuda").bfloat16().transpose(1, 2)  # dims not contiguous
    gpu.mxfp4_kv_append(cache, x[:0], x[:0], torch.zeros(0, dtype=torch.int64, device="cuda"), page)
    assert not cache.any()
    gpu.mxfp4_kv_append(cache, x, x, torch.tensor([16, 2, 31, 47], device="cuda"), page)
    want = np.zeros(cache.shape, np.uint8)
    q, s = orc.mxfp4_quantize(bits16(x).reshape(-1, dim))
    q, s = q.reshape(4, heads, -1), s.reshape(4, heads, -1)
    ref.write_page_tokens(want, (heads, dim, page), [16, 2, 31, 47], q, s, q, s)
    assert np.array_equal(u8(cache), want)


def filled_cache(rng, geo, pages, stride_pad=0):
    """Random codes and ordinary scales; (device [pages, page_bytes], host)."""
    heads, dim, page = geo
    host = rng.integers(0, 256, (pages, ref.page_bytes(heads, dim, page)), dtype=np.uint8)
    host[:, heads * page * dim:] = rng.integers(124, 129, (pages, heads * page * dim // 16), dtype=np.uint8)
    wide = torch.zeros((pages, host.shape[1] + stride_pad), dtype=torch.uint8, device="cuda")
    dev = wide[:, :host.shape[1]]
    dev.copy_(torch.from_numpy(host))
    return dev, host


def attend(gpu, geo, cache, host, q, table, lengths, scale=None, causal=True, window=0):
    heads, dim, page = geo
    got, lse = gpu.mxfp4_kv_attention(q, cache, torch.from_numpy(table).cuda(), torch.from_numpy(lengths).cuda(), heads, page,
                                      scale=scale, causal=causal, window=window, return_lse=True)
    assert got.shape == q.shape and got.dtype == torch.bfloat16 and lse.dtype == torch.float32
    want = ref.attention(q.double().cpu().numpy(), host, geo, table, lengths, dim ** -0.5 if scale is None else scale, causal, window)
    name = f"{geo} {tuple(q.shape)} causal={causal} window={window}"
    ref.assert_within(name, got.float().cpu().numpy(), want[0], want[2])
    ref.assert_within(name + " lse", lse.cpu().numpy(), want[1], want[3])
    return got, lse


@pytest.mark.parametrize("geo", GEOS, ids=str)
@pytest.mark.parametrize("tokens,group", [(1, 1), (1, 8), (2, 5), (4, 4), (7, 3), (33, 2), (70, 4)])
def test_attention(gpu, geo, tokens, group):
    """Ragged lengths from none to many tiles, every mask."""
    heads, dim, page = geo
    announce(f"attention {geo} tokens {tokens} group {group}")
    rng = np.random.default_rng(dim * 100 + tokens)
    lengths = np.array([0, 1, tokens - 1, tokens, 15, 16, 17, 63, 64, 65, 333, 700], np.int32)
    if tokens > 64:  # the plain form takes long
        lengths = lengths[[0, 2, 9, 11]]
    width = -(-700 // page)
    cache, host = filled_cache(rng, geo, 40)
    table = rng.integers(0, 40, (len(lengths), width), dtype=np.int32)
    q = to_dev_bf16(bf16_bits(rng.standard_normal((len(lengths), tokens, heads * group, dim))))
    for causal, window in ((True, 0), (False, 0), (True, 1), (True, 37), (False, 100), (True, 5000)):
        attend(gpu, geo, cache, host, q, table, lengths, causal=causal, window=window)


@pytest.mark.parametrize("geo", GEOS, ids=str)
@pytest.mark.parametrize("rows", [53, 190])
def test_attention_many_rows(gpu, geo, rows):
    """So many rows, in enough workgroups, that they share decoded tiles."""
    heads, dim, page = geo
    group = 2 + dim % 3
    tokens = -(-rows // group)
    announce(f"attention {geo} rows {tokens * group}")
    rng = np.random.default_rng(dim * 10 + rows)
    lengths = np.array([0, 1, tokens - 1, tokens, 15, 16, 17, 63, 64, 65, 333, 700], np.int32)
    while len(lengths) * heads * (rows // 16) <= 128:
        lengths = np.concatenate([lengths, rng.integers(0, 200, 7).astype(np.int32)])
    cache, host = filled_cache(rng, geo, 40)
    table = rng.integers(0, 40, (len(lengths), -(-700 // page)), dtype=np.int32)
    q = to_dev_bf16(bf16_bits(rng.standard_normal((len(lengths), tokens, heads * group, dim))))
    for causal, window in ((True, 0), (False, 0), (True, 29), (False, 100)):
        attend(gpu, geo, cache, host, q, table, lengths, causal=causal, window=window)


@pytest.mark.parametrize("seqs,geo", [(100, (8, 64, 16)), (130, (7, 96, 48)), (100, (8, 128, 32)), (40, (8, 128, 32)), (40, (8, 192, 32)),
                                      (128, (3, 256, 16))], ids=str)
def test_attention_many_sequences(gpu, seqs, geo):
    """More workgroups than CUs: sequences are started by length, ties among them."""
    heads, dim, page = geo
    announce(f"attention {seqs} sequences {geo}")
    rng = np.random.default_rng(seqs + dim)
    cache, host = filled_cache(rng, geo, 50)
    lengths = rng.integers(0, 180, seqs).astype(np.int32)
    lengths[: seqs // 4] = 77
    table = rng.integers(0, 50, (seqs, -(-180 // page)), dtype=np.int32)
    q = to_dev_bf16(bf16_bits(rng.standard_normal((seqs, 1, heads * 2, dim))))
    attend(gpu, geo, cache, host, q, table, lengths)
    attend(gpu, geo, cache, host, q, table, lengths, window=40)


@pytest.mark.parametrize("width,lengths", [(3, [500, 48, -5]), (0, [4, 0, 9]), (40, [1, 640, 639])])
def test_attention_lengths_and_holes(gpu, width, lengths):
    """Lengths past the table or below zero, an empty table, holes in it, no pages at all."""
    announce(f"attention holes {width}")
    geo = (2, 64, 16)
    rng = np.random.default_rng(width)
    cache, host = filled_cache(rng, geo, 9, stride_pad=64)
    table = rng.integers(-2, 11, (3, width), dtype=np.int32)
    lengths = np.array(lengths, np.int32)
    q = to_dev_bf16(bf16_bits(rng.standard_normal((3, 2, 4, 64))))
    attend(gpu, geo, cache, host, q, table, lengths)
    attend(gpu, geo, cache, host, q, table, lengths, causal=False, window=20)
    attend(gpu, geo, cache[:0], host[:0], q, table, lengths)
    attend(gpu, geo, cache, host, q[:0], table[:0], lengths[:0])
    attend(gpu, geo, cache, host, q[:, :0], table, lengths)


def test_attention_strides_and_scales(gpu):
    """q as a view of a fused projection, a strided table, negative, zero and large scales."""
    announce("attention strides, scales")
    geo = (2, 128, 32)
    rng = np.random.default_rng(3)
    cache, host = filled_cache(rng, geo, 12, stride_pad=4096)
    lengths = np.array([200, 33, 96], np.int32)
    wide = rng.integers(0, 12, (3, 20), dtype=np.int32)
    qkv = to_dev_bf16(bf16_bits(rng.standard_normal((3, 3, 14, 128))))
    q = qkv[:, :, 2:10]
    for scale in (None, -0.3, 0.0, 2.5):
        attend(gpu, geo, cache, host, q, wide[:, :7], lengths, scale=scale)
    got = gpu.mxfp4_kv_attention(q, cache, torch.from_numpy(wide).cuda()[:, :7], torch.from_numpy(lengths).cuda(), 2, 32)
    again = gpu.mxfp4_kv_attention(q.contiguous(), cache, torch.from_numpy(wide[:, :7].copy()).cuda(),
                                   torch.from_numpy(lengths).cuda(), 2, 32)
    assert torch.equal(got, again)
    odd = torch.empty(qkv.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(qkv.shape)
    odd.copy_(qkv)
    got = gpu.mxfp4_kv_attention(odd[:, :, 2:10], cache, torch.from_numpy(wide).cuda()[:, :7], torch.from_numpy(lengths).cuda(), 2, 32)
    assert torch.equal(got, again)


@pytest.mark.parametrize("tokens,lengths", [(1, [300, 77]), (40, [300, 77]), (300, [310, 64])])
def test_attention_masked_places_hold_anything(gpu, tokens, lengths):
    """NaN scales, the largest scales and random bytes past the length, outside
    the window and in the causal future change nothing; visible ones do."""
    announce(f"attention garbage {tokens}")
    geo = (2, 128, 32)
    heads, dim, page = geo
    rng = np.random.default_rng(tokens)
    cache, host = filled_cache(rng, geo, 24)
    table = rng.permutation(24).astype(np.int32).reshape(2, 12)
    lengths = np.array(lengths, np.int32)
    q = to_dev_bf16(bf16_bits(rng.standard_normal((2, tokens, 8, dim))))
    a, c = heads * page * dim // 2, heads * page * dim // 32

    def scales(which, b, t):
        sect = host[table[b, t // page], 2 * a + which * c:2 * a + (which + 1) * c]
        return sect.reshape(heads, page // 16, dim // 32, 16)[:, t % page // 16, :, t % 16]

    for b in range(2):
        for t in range(int(lengths[b]), 12 * page):
            for which in (0, 1):
                scales(which, b, t)[:] = rng.choice([255, 254, 253, 0], scales(which, b, t).shape)
    # a NaN group of a new token: seen by some rows of a causal tile only
    scales(1, 0, int(lengths[0]) - 1)[0, 1] = 255
    if tokens > 1:
        scales(1, 0, int(lengths[0]) - tokens // 2)[1, 2] = 255
        scales(0, 1, max(0, int(lengths[1]) - 3))[0, 0] = 255
    scales(1, 0, 5)[1, 3] = 255  # seen unless outside a window
    cache.copy_(torch.from_numpy(host))
    for causal, window in ((True, 0), (True, 50), (False, 0), (True, 3)):
        attend(gpu, geo, cache, host, q, table, lengths, causal=causal, window=window)


def test_attention_nan_and_inf_queries(gpu):
    announce("attention nan queries")
    geo = (1, 64, 16)
    rng = np.random.default_rng(4)
    cache, host = filled_cache(rng, geo, 8)
    host[:, :16 * 32] &= 0x77  # keys without sign, nor zeros: Inf scores of one sign
    host[:, :16 * 32] |= 0x11
    cache.copy_(torch.from_numpy(host))
    x = rng.standard_normal((2, 3, 2, 64))
    x[0, 1, 0, 5] = np.nan
    x[1, 2, 1, 0] = -np.inf  # every score -inf
    q = to_dev_bf16(bf16_bits(x))
    lengths = np.array([100, 128], np.int32)
    table = np.arange(16, dtype=np.int32).reshape(2, 8) % 8
    got, lse = gpu.mxfp4_kv_attention(q, cache, torch.from_numpy(table).cuda(), torch.from_numpy(lengths).cuda(), 1, 16, return_lse=True)
    assert got[0, 1, 0].isnan().all() and lse[0, 1, 0].isnan()
    assert not got[1, 2, 1].any() and lse[1, 2, 1] == -np.inf
    good = torch.ones(2, 3, 2, dtype=torch.bool, device="cuda")
    good[0, 1, 0] = good[1, 2, 1] = False
    assert got[good].isfinite().all() and lse[good].isfinite().all()


def test_attention_long_context(gpu):
    """One long sequence: many splits, joined."""
    announce("attention long context")
    geo = (1, 128, 64)
    rng = np.random.default_rng(5)
    cache, host = filled_cache(rng, geo, 640)
    table = rng.permutation(640).astype(np.int32).reshape(1, 640)
    for tokens, length in ((1, 40960), (3, 40000), (20, 33333)):
        q = to_dev_bf16(bf16_bits(rng.standard_normal((1, tokens, 4, 128))))
        attend(gpu, geo, cache, host, q, table, np.array([length], np.int32))


@pytest.mark.parametrize("geo", [(2, 64, 16), (4, 96, 48), (2, 128, 64), (2, 192, 32), (2, 256, 16)], ids=str)
def test_attention_many_rows_split(gpu, geo):
    """Thousands of rows over split contexts."""
    heads, dim, page = geo
    announce(f"attention many rows split {geo}")
    rng = np.random.default_rng(dim)
    cache, host = filled_cache(rng, geo, 30)
    width = -(-2000 // page)
    table = rng.integers(0, 30, (1, width), dtype=np.int32)
    tokens = 4100 // (2 * heads)
    q = to_dev_bf16(bf16_bits(rng.standard_normal((1, tokens, 2 * heads, dim))))
    attend(gpu, geo, cache, host, q, table, np.array([1900], np.int32))


def test_cache_past_32_bits(gpu, orc):
    """Append, attend and copy in pages past 2^31 and 2^32 bytes of a layer."""
    announce("cache past 32 bits")
    geo = (8, 128, 128)
    heads, dim, page = geo
    pages = -(-(5 << 30) // ref.page_bytes(*geo))
    cache = torch.zeros((pages, ref.page_bytes(*geo)), dtype=torch.uint8, device="cuda")
    used = [pages - 1, 0, pages * 9 // 20, pages * 17 // 20]
    n = 4 * page - 3
    rng = np.random.default_rng(6)
    xb = bf16_bits(rng.standard_normal((n, 2 * heads, dim)))
    x = to_dev_bf16(xb)
    slots = np.array([used[i // page] * page + i % page for i in range(n)], np.int64)
    gpu.mxfp4_kv_append(cache, x[:, :heads], x[:, heads:], torch.from_numpy(slots).cuda(), page)
    q = to_dev_bf16(bf16_bits(rng.standard_normal((1, 2, 16, dim))))
    small = np.zeros((4, cache.shape[1]), np.uint8)
    for i, p in enumerate(used):
        small[i] = u8(cache[p])
    kq, ks = orc.mxfp4_quantize(np.ascontiguousarray(xb[:, :heads]).reshape(-1, dim))
    vq, vs = orc.mxfp4_quantize(np.ascontiguousarray(xb[:, heads:]).reshape(-1, dim))
    want = np.zeros_like(small)
    ref.write_page_tokens(want, geo, np.arange(n), *(a.reshape(n, heads, -1) for a in (kq, ks, vq, vs)))
    assert np.array_equal(small, want)
    lengths = np.array([n], np.int32)
    got = gpu.mxfp4_kv_attention(q, cache, torch.tensor([used], dtype=torch.int32, device="cuda"),
                                 torch.from_numpy(lengths).cuda(), heads, page)
    o, _, ob, _ = ref.attention(q.double().cpu().numpy(), small, geo, np.arange(4, dtype=np.int32)[None], lengths, dim ** -0.5, True, 0)
    ref.assert_within("attention", got.float().cpu().numpy(), o, ob)
    free = [pages - 2, 1, pages // 2, pages * 4 // 5]
    gpu.mxfp4_kv_copy_pages(cache, torch.tensor(used, dtype=torch.int32, device="cuda"), torch.tensor(free, dtype=torch.int32, device="cuda"))
    for a, b in zip(used, free):
        assert torch.equal(cache[a], cache[b])


@pytest.mark.parametrize("layers,geo", [(1, (1, 64, 16)), (3, (2, 96, 48)), (5, (8, 128, 64))])
def test_copy_pages(gpu, layers, geo):
    announce(f"copy pages {layers} {geo}")
    rng = np.random.default_rng(layers)
    host = rng.integers(0, 256, (layers, 30, ref.page_bytes(*geo)), dtype=np.uint8)
    order = rng.permutation(30).astype(np.int32)
    for n in (0, 1, 7, 15):
        src, dst = order[:n].copy(), order[15:15 + n].copy()
        if n == 7:
            src[2], dst[4], dst[5], src[0] = -1, 30, -3, 1 << 30
        want = host.copy()
        fine = (src >= 0) & (src < 30) & (dst >= 0) & (dst < 30)
        want[:, dst[fine]] = host[:, src[fine]]
        padded = torch.full((layers, 31, host.shape[2] + 32), 9, dtype=torch.uint8, device="cuda")
        view = padded[:, :30, :host.shape[2]]
        view.copy_(torch.from_numpy(host))
        gpu.mxfp4_kv_copy_pages(view, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda())
        assert np.array_equal(u8(view), want)
        assert (padded[:, 30] == 9).all() and (padded[:, :, host.shape[2]:] == 9).all()
        one = torch.from_numpy(host[0]).cuda()
        gpu.mxfp4_kv_copy_pages(one, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda())
        assert np.array_equal(u8(one), want[0])


@pytest.mark.parametrize("n", [1, 7, 512])
def test_copy_pages_with_strided_indices(gpu, n):
    """Index tensors as columns of pairs, as even and odd elements, as one of each."""
    announce(f"copy pages, strided indices {n}")
    geo = (1, 64, 16)
    pages = 2 * n + 3
    rng = np.random.default_rng(n)
    host = rng.integers(0, 256, (2, pages, ref.page_bytes(*geo)), dtype=np.uint8)
    pairs = rng.permutation(pages)[:2 * n].reshape(n, 2).astype(np.int32)
    dev = torch.from_numpy(pairs).cuda()
    want = host.copy()
    want[:, pairs[:, 1]] = host[:, pairs[:, 0]]
    turned = dev.t().contiguous()
    for src, dst in ((dev[:, 0], dev[:, 1]), (dev.flatten()[0::2], dev.flatten()[1::2]), (turned[0], dev[:, 1]), (dev[:, 0], turned[1])):
        cache = torch.from_numpy(host).cuda()
        gpu.mxfp4_kv_copy_pages(cache, src, dst)
        assert np.array_equal(u8(cache), want)


# -- streams and graphs ----------------------------------------------------------

def test_decode_step_on_a_side_stream_and_in_a_graph(gpu):
    """The operators run on the current stream and can be captured: replays
    with new inputs equal eager calls."""
    announce("decode step in a graph")
    rng = np.random.default_rng(12)
    heads, dim, page, hidden = 2, 64, 16, 256
    w = to_dev_bf16(bf16_bits(0.05 * rng.standard_normal((6 * dim + 2 * dim, hidden))))
    qw, sw = gpu.mxfp4_quantize(w)
    cache = gpu.mxfp4_kv_cache(1, 64, heads, dim, page)
    x = torch.zeros(3, hidden, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    lengths = torch.zeros(3, dtype=torch.int32, device="cuda")
    table = torch.arange(60, dtype=torch.int32, device="cuda").view(3, 20)
    src, dst = torch.tensor([0], dtype=torch.int32, device="cuda"), torch.tensor([63], dtype=torch.int32, device="cuda")

    def step():
        qkv = gpu.mxfp4_matvec(x, qw, sw).view(3, 8, dim)
        gpu.mxfp4_kv_append(cache[0], qkv[:, 4:6], qkv[:, 6:], slots, page)
        out = gpu.mxfp4_kv_attention(qkv[:, None, :4], cache[0], table, lengths, heads, page)
        gpu.mxfp4_kv_copy_pages(cache, src, dst)
        return qkv, out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    twin = torch.zeros_like(cache)
    cache.zero_()
    for i in range(5):
        x.copy_(to_dev_bf16(bf16_bits(rng.standard_normal((3, hidden)))))
        lengths.fill_(i + 1)
        slots.copy_(torch.arange(3, device="cuda") * 20 * page + i)
        graph.replay()
        torch.cuda.synchronize()
        got, held = [t.clone() for t in captured], cache.clone()
        cache.copy_(twin)
        want = step()
        assert torch.equal(held, cache) and all(torch.equal(a, b) for a, b in zip(got, want))
        twin.copy_(cache)
        assert torch.equal(cache[:, 0], cache[:, 63]) and cache.any()
