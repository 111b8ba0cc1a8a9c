"""The decode operators on the GPU where they can go wrong most easily: every
scale byte beside any other, values past bf16's range, masks that leave some
rows a token and others not, and every form of the attention kernels."""
import numpy as np
import pytest
import torch

import decode_ref as ref
from gpu_util import announce, to_dev_bf16, u8

pytestmark = pytest.mark.gpu


def bf16_bits(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)


def sections(host, geo):
    """Views of the pages' K codes [pages, heads, page, dim/2], V codes and K and
    V scales [pages, heads, page/16, dim/2 or dim/32, 16]."""
    heads, dim, page = geo
    a, c = heads * page * dim // 2, heads * page * dim // 32
    blocks = (len(host), heads, page // 16, -1, 16)
    return (host[:, :a].reshape(len(host), heads, page, dim // 2), host[:, a:2 * a].reshape(blocks),
            host[:, 2 * a:2 * a + c].reshape(blocks), host[:, 2 * a + c:].reshape(blocks))


def filled_cache(rng, geo, pages):
    """Random codes and ordinary scales of ``pages`` pages (host)."""
    heads, dim, page = geo
    host = rng.integers(0, 256, (pages, ref.page_bytes(*geo)), dtype=np.uint8)
    host[:, heads * page * dim:] = rng.integers(124, 129, (pages, heads * page * dim // 16), dtype=np.uint8)
    return host


def attend(gpu, geo, cache, q, table, lengths, **kw):
    out, lse = gpu.mxfp4_kv_attention(q, cache, torch.from_numpy(table).cuda(), torch.from_numpy(lengths).cuda(), geo[0], geo[2],
                                      return_lse=True, **kw)
    return out.float().cpu().numpy(), lse.cpu().numpy()


def check(gpu, geo, host, q, table, lengths, causal=True, window=0):
    got = attend(gpu, geo, torch.from_numpy(host).cuda(), q, table, lengths, causal=causal, window=window)
    want = ref.attention(q.double().cpu().numpy(), host, geo, table, lengths, geo[1] ** -0.5, causal, window)
    name = f"{geo} {tuple(q.shape)} causal={causal} window={window}"
    ref.assert_within(name, got[0], want[0], want[2])
    ref.assert_within(name + " lse", got[1], want[1], want[3])


def wild_case(gpu, geo, tokens, group, seqs, context, masks):
    """V scales of 253 and 254: with small codes ordinary values, with large
    ones past bf16's range, where the result may be infinite, NaN or what real
    numbers give.  On tokens that only some rows of a tile see (causal, window)
    they count for those rows alone."""
    heads, dim, page = geo
    announce(f"values past bf16 {geo} {tokens}x{group}, {seqs} sequences of {context}")
    rng = np.random.default_rng(dim + tokens)
    width = -(-context // page)
    host = filled_cache(rng, geo, seqs * width)
    table = rng.permutation(seqs * width).astype(np.int32).reshape(seqs, width)
    lengths = rng.integers(tokens, width * page + 1, seqs).astype(np.int32)
    _, vc, _, vs = sections(host, geo)
    wild = []  # (sequence, token, head, group of 32)
    for b in range(seqs):
        for h in range(heads):
            for g in range(dim // 32):  # one such token a group: sums of more would overflow
                t = int(lengths[b]) - int(rng.integers(1, tokens + 1))
                p, i = table[b, t // page], t % page
                byte, big = int(rng.choice([253, 254])), rng.random() < 0.5
                codes = vc[p, h, i // 16, 16 * g:16 * g + 16, i % 16]
                if not big:  # magnitudes up to 3 times 2^126 and 1.5 times 2^127 are in range
                    codes[:] = rng.integers(0, 6 if byte == 253 else 4, 16) | rng.integers(0, 6 if byte == 253 else 4, 16) << 4 | 0x80
                vs[p, h, i // 16, g, i % 16] = byte
                wild.append((b, t, h, g))
    q = to_dev_bf16(bf16_bits(0.5 * rng.standard_normal((seqs, tokens, heads * group, dim))))
    cache = torch.from_numpy(host).cuda()
    for causal, window in masks:
        got, lse = attend(gpu, geo, cache, q, table, lengths, causal=causal, window=window)
        o, want_lse, ob, lb = ref.attention(q.double().cpu().numpy(), host, geo, table, lengths, dim ** -0.5, causal, window)
        ref.assert_within("lse", lse, want_lse, lb)
        far = np.zeros(o.shape, bool)  # outputs of a value past the range
        for b, t, h, g in wild:
            _, v = ref.read_pages(host, geo, table[b, t // page:t // page + 1])
            over = np.abs(v[h, t % page, 32 * g:32 * g + 32]) >= 2.0 ** 128
            at = lengths[b] - tokens + np.arange(tokens)
            sees = np.ones(tokens, bool)
            if causal:
                sees &= t <= at
            if window:
                sees &= t > at - window
            far[b, :, h * group:(h + 1) * group, 32 * g:32 * g + 32] |= (sees[:, None] & over)[:, None]
        gone = far & ~np.isfinite(got)
        ref.assert_within(f"{causal} {window}", np.where(gone, 0, got), np.where(gone, 0, o), ob)


# (tokens, query heads): one and two strips of 16 rows; rows that share decoded tiles
@pytest.mark.parametrize("tokens,group", [(5, 2), (20, 1), (50, 2), (150, 2)])
@pytest.mark.parametrize("geo", [(2, 64, 16), (1, 96, 48), (2, 128, 64), (1, 192, 192), (1, 256, 16)], ids=str)
def test_values_past_bf16_where_some_rows_see_them(gpu, geo, tokens, group):
    seqs = max(2, -(-130 // geo[0] // -(-tokens * group // 16)))  # enough workgroups to share tiles from 49 rows on
    wild_case(gpu, geo, tokens, group, seqs, 400, ((True, 0), (True, 3), (True, 40), (False, tokens + 9)))


@pytest.mark.parametrize("geo,tokens,seqs,context", [((2, 64, 16), 3, 2, 3000), ((1, 128, 64), 20, 2, 2600), ((2, 64, 64), 150, 4, 1600),
                                                     ((4, 192, 32), 70, 4, 1100)], ids=str)
def test_values_past_bf16_in_split_contexts(gpu, geo, tokens, seqs, context):
    need = gpu.load().mxfp4_kv_attention_workspace_size(seqs, tokens, 2 * geo[0], *geo, -(-context // geo[2]), 0)
    assert need > 0  # it is split
    wild_case(gpu, geo, tokens, 2, seqs, context, ((True, 0),))


@pytest.mark.parametrize("group", [1, 64])
@pytest.mark.parametrize("page", [16, 64])
def test_weights_are_not_rounded_to_bf16(gpu, page, group):
    """Values of both signs and one magnitude: o is their weights' difference,
    and an error of the weights stands out.

    Scores are exact (four products of a few bits), so each exponent is off by
    at most 2^-22 |s| and each weight by twice that, as e^x and the largest
    score are, plus 2^-20 for exp2.  The product takes a weight as two bf16
    numbers, off by 2^-8 of 2^-8.  Up to 2 n + 64 additions in fp32:
    |err| <= (2^-16 + 2^-19 + 8 * 2^-22 max |s| + (2 n + 64) 2^-23) sum p |v| + 2^-8 |o|.
    Weights rounded to bf16 alone would be off by up to 2^-8 of that sum."""
    announce(f"weights' precision, page {page}, {group} heads")
    dim, n, seqs = 64, 24, 140
    geo = (1, dim, page)
    rng = np.random.default_rng(page + group)
    width = -(-n // page)
    host = np.zeros((seqs * width, ref.page_bytes(*geo)), np.uint8)
    kc, vc, ks, vs = sections(host, geo)
    kc[:] = rng.integers(0, 256, kc.shape)
    vc[:] = 0x22 | rng.integers(0, 2, vc.shape) << 3 | rng.integers(0, 2, vc.shape) << 7  # +-1
    ks[:] = vs[:] = 127
    table = np.arange(seqs * width, dtype=np.int32).reshape(seqs, width)
    x = np.zeros((seqs, 1, group, dim))
    for _ in range(4):
        x[..., rng.integers(0, dim)] = rng.integers(-8, 9, x.shape[:-1]) / 8
    lengths = rng.integers(2, n + 1, seqs).astype(np.int32)
    got, lse = attend(gpu, geo, torch.from_numpy(host).cuda(), to_dev_bf16(bf16_bits(x)), table, lengths, scale=0.125)
    worst = 0.0
    for b in range(seqs):
        k, v = ref.read_pages(host, geo, table[b])
        k, v = k[0, :lengths[b]], v[0, :lengths[b]]
        s = 0.125 * (x[b, 0] @ k.T)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        o = p @ v
        bound = (2.0 ** -16 + 2.0 ** -19 + 2.0 ** -19 * np.abs(s).max() + (2 * n + 64) * 2.0 ** -23) + 2.0 ** -8 * np.abs(o)
        ref.assert_within(f"sequence {b}", got[b, 0], o, bound)


def as_float32(v):
    with np.errstate(over="ignore"):
        return np.asarray(v, np.float64).astype(np.float32)


def assert_values(name, got, want):
    """Equal, NaN and infinities too; magnitudes below 2^-126 may be zero."""
    small = np.abs(want) < 2.0 ** -126
    same = (got == want) | (np.isnan(got) & np.isnan(want)) | (small & (got == 0))
    assert same.all(), f"{name}: {(~same).sum()} of {same.size}, first at {tuple(np.argwhere(~same)[0])}: " \
                       f"{got[~same][0]!r} for {want[~same][0]!r}"


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("group", [1, 64])
def test_attention_every_scale_and_code(gpu, dim, page, group):
    """One visible token, whose V comes back as it is and whose score is the
    lse; its block's other scales are anything.  Then 64 equal tokens."""
    announce(f"attention, every scale and code {dim} {page} {group}")
    rng = np.random.default_rng(dim + page + group)
    geo = (1, dim, page)
    full = -(-64 // page)  # pages of 64 tokens
    host = rng.integers(0, 256, (256 * full, ref.page_bytes(*geo)), dtype=np.uint8)
    kc, vc, ks, vs = sections(host, geo)
    first = host.reshape(256, full, -1)[:, 0]  # page of token 0
    kc1, vc1, ks1, vs1 = sections(first, geo)
    byte = np.arange(256)
    for g in range(dim // 32):
        vs1[:, 0, 0, g, 0] = rng.permutation(256)
    vs1[:, 0, 0, rng.integers(0, dim // 32), 0] = byte
    kc1[:, 0, 0] = 0  # one code of K is not zero
    at = rng.integers(0, dim, 256)
    code = rng.integers(1, 8, 256)
    kc1[byte, 0, 0, at // 2] = code << 4 * (at % 2)
    ks1[:, 0, 0, :, 0] = rng.integers(0, 253, (256, dim // 32))
    ks1[byte, 0, 0, at // 32, 0] = byte
    table = np.arange(256 * full, dtype=np.int32).reshape(256, full)
    q = torch.ones(256, 1, group, dim, dtype=torch.bfloat16, device="cuda")
    got, lse = attend(gpu, geo, torch.from_numpy(host).cuda(), q, table, np.ones(256, np.int32), scale=1.0)
    _, v = ref.read_pages(first, geo, range(256))
    v = v.reshape(256, page, dim)[:, 0]
    # scores past fp32's range have no weight
    score = as_float32(ref.LEVELS[code] * ref.e8m0_to_f64(byte))
    fine = byte < 250
    wide = np.broadcast_to(score[:, None, None], lse.shape)
    assert (np.abs(lse[fine] - wide[fine]) <= 2.0 ** -21 * wide[fine] + 2.0 ** -120).all()
    assert np.isnan(lse[255]).all() and np.isnan(got[255]).all()
    assert_values("one token", got[fine], np.broadcast_to(as_float32(v)[:, None, None], got.shape)[fine])
    # the same token 64 times, so that the tile is full
    for block in (vc, vs):
        whole = block.reshape(256, full, page // 16, -1, 16)
        whole[:] = whole[:, :1, :1, :, :1]
    kc[:], ks[:] = 0, 127
    got, lse = attend(gpu, geo, torch.from_numpy(host).cuda(), q, table, np.full(256, 64, np.int32), scale=1.0)
    scale = np.repeat(sections(first, geo)[3][:, 0, 0, :, 0], 32, -1)  # of each dim
    # 64 values are added before the division: past 2^121 that may overflow
    fine = np.broadcast_to(((scale < 246) | (scale == 255))[:, None, None], got.shape)
    want = np.broadcast_to(as_float32(v)[:, None, None], got.shape)
    assert_values("64 tokens", got[fine], want[fine])
    assert (np.abs(lse - np.log(64)) < 2.0 ** -18).all()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("group", [1, 64])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("power", [22, 33, 90, 120])
def test_vast_scores(gpu, power, page, group, sign):
    """Scores of +-{0, .. 6} 2^power, exact: the largest share all the weight, o
    is the mean of their values and lse their score plus log of their number.
    Each weight is 1 but for exp2, the joins and bf16 (2^-16 and 2^-19 as
    below 2^-8 |o| of the output), lse off by two roundings and log's."""
    announce(f"vast scores 2^{power} {page} {group} {sign}")
    dim, seqs = 64, 140
    geo = (1, dim, page)
    rng = np.random.default_rng(power + page + group + sign)
    width = -(-700 // page)
    pages = 60
    host = filled_cache(rng, geo, pages)
    kc, _, ks, _ = sections(host, geo)
    kc[:] &= 0x77  # keys without signs
    ks[:] = 127
    x = np.zeros((seqs, 1, group, dim))
    at = rng.integers(0, dim, (seqs, group))
    x[np.arange(seqs)[:, None], 0, np.arange(group), at] = sign * 2.0 ** (power - 3)
    table = rng.integers(0, pages, (seqs, width)).astype(np.int32)
    lengths = rng.integers(1, 701, seqs).astype(np.int32)
    lengths[:100] = rng.integers(1, 9, 100)
    got, lse = attend(gpu, geo, torch.from_numpy(host).cuda(), to_dev_bf16(bf16_bits(x)), table, lengths, scale=8.0)
    for b in range(seqs):
        k, v = ref.read_pages(host, geo, table[b])
        k, v = k[0, :lengths[b]], v[0, :lengths[b]]
        s = sign * k[:, at[b]].T * 2.0 ** power  # [group, tokens]
        top = s.max(-1, keepdims=True)
        p = (s == top) / (s == top).sum(-1, keepdims=True)
        o = p @ v
        bound = (2.0 ** -15 + (lengths[b] + 64) * 2.0 ** -23) * (p @ np.abs(v)) + 2.0 ** -8 * np.abs(o)
        ref.assert_within(f"sequence {b}", got[b, 0], o, bound)
        want = top[:, 0] + np.log((s == top).sum(-1))
        ref.assert_within(f"lse {b}", lse[b, 0], want, 2.0 ** -21 * np.abs(want) + 2.0 ** -18)


@pytest.mark.parametrize("tokens,group", [(1, 2), (50, 2)])
@pytest.mark.parametrize("scale", [0.0, -0.0])
def test_zero_scale_of_vast_products(gpu, tokens, group, scale):
    """With a scale of zero every score is 0 however large q.k is, and NaN
    where q or k has no finite product."""
    announce(f"zero scale {tokens}")
    geo = (1, 64, 16)
    rng = np.random.default_rng(tokens)
    seqs, width = 40, 5
    host = filled_cache(rng, geo, seqs * width)
    kc, _, ks, _ = sections(host, geo)
    ks[:] = rng.integers(120, 161, ks.shape)
    table = rng.permutation(seqs * width).astype(np.int32).reshape(seqs, width)
    x = rng.standard_normal((seqs, tokens, group, 64)) * np.exp2(rng.integers(60, 120, (seqs, tokens, group, 1)))
    q = to_dev_bf16(bf16_bits(x))
    lengths = rng.integers(tokens, 81, seqs).astype(np.int32)
    cache = torch.from_numpy(host).cuda()
    got, lse = attend(gpu, geo, cache, q, table, lengths, scale=scale)
    want = ref.attention(q.double().cpu().numpy(), host, geo, table, lengths, 0.0, True, 0)
    ref.assert_within("zero", got, want[0], want[2])
    ref.assert_within("zero lse", lse, want[1], want[3])
    q[0, 0, 0, 3], q[1, 0, 1, 5] = float("nan"), float("inf")
    got, lse = attend(gpu, geo, cache, q, table, lengths, scale=scale)
    assert np.isnan(got[0, 0, 0]).all() and np.isnan(lse[0, 0, 0]) and np.isnan(got[1, 0, 1]).all() and np.isnan(lse[1, 0, 1])
    got[0, 0, 0] = got[1, 0, 1] = 0
    assert np.isfinite(got).all()


@pytest.mark.parametrize("tokens", [1, 5, 70])
@pytest.mark.parametrize("g", [1.0, float("nan"), float("inf")])
def test_products_over_no_columns_are_zero(gpu, tokens, g):
    """An empty sum is 0 whatever the weights' scale is; rows in any shape."""
    announce(f"no columns {tokens} {g}")
    x = torch.ones(tokens, 0, dtype=torch.bfloat16, device="cuda")
    q, s = (torch.zeros(33, 0, dtype=torch.uint8, device="cuda") for _ in range(2))
    for dtype in (torch.bfloat16, torch.float32):
        for rows in (x, x.view(tokens, 1, 0), x.view(1, tokens, 0)):
            out = torch.full((*rows.shape[:-1], 33), 7.0, dtype=dtype, device="cuda")
            gpu.nvfp4_matvec(rows, q, s, torch.tensor([g], device="cuda"), out_dtype=dtype, out=out)
            assert not out.any()
            assert not gpu.mxfp4_matvec(rows, q, s, out_dtype=dtype).any()


@pytest.mark.parametrize("kind", ["mx", "nv"])
def test_matvec_of_millions_of_tokens(gpu, kind):
    """More token tiles than one launch holds."""
    announce(f"matvec of millions of tokens {kind}")
    tokens, n, k = 65535 * 64 + 77, 3, 32
    x = torch.randn(tokens, k, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    rng = np.random.default_rng(2)
    q = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    if kind == "mx":
        s = rng.integers(124, 130, (n, 1), dtype=np.uint8)
        w = ref.fp4_values(q) * np.repeat(ref.e8m0_to_f64(s), 32, -1)
        call = lambda **kw: gpu.mxfp4_matvec(x, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), **kw)  # noqa: E731
    else:
        s = rng.integers(0x30, 0x50, (n, 2), dtype=np.uint8)
        w = ref.fp4_values(q) * np.repeat(ref.e4m3_to_f64(s), 16, -1)
        call = lambda **kw: gpu.nvfp4_matvec(x, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(),  # noqa: E731
                                             torch.ones(1, device="cuda"), **kw)
    w = torch.from_numpy(w).cuda()
    want = torch.mm(x.double(), w.t().contiguous())
    bound = (k + 16) * 2.0 ** -23 * torch.mm(x.double().abs(), w.abs().t().contiguous()) + 2.0 ** -24 * want.abs()
    got = call(out_dtype=torch.float32)
    assert ((got.double() - want).abs() <= bound).all()
    got = call()
    assert ((got.double() - want).abs() <= bound + 2.0 ** -8 * want.abs()).all()


@pytest.mark.parametrize("tokens,group", [(1, 2), (50, 2)])
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_scales_that_are_not_finite(gpu, tokens, group, scale):
    """Queries that see something get NaN; those that see nothing zeros and -inf."""
    announce(f"scale {scale} {tokens}")
    geo = (1, 64, 16)
    rng = np.random.default_rng(tokens)
    seqs, width = 40, 5
    host = filled_cache(rng, geo, seqs * width)
    table = rng.permutation(seqs * width).astype(np.int32).reshape(seqs, width)
    table[3, :2] = -1
    lengths = rng.integers(0, 81, seqs).astype(np.int32)
    lengths[:4] = 0, 1, tokens, 17
    q = to_dev_bf16(bf16_bits(rng.standard_normal((seqs, tokens, group, 64))))
    got, lse = attend(gpu, geo, torch.from_numpy(host).cuda(), q, table, lengths, scale=scale)
    sees = np.zeros((seqs, tokens, group), bool)
    for b in range(seqs):
        at = lengths[b] - tokens + np.arange(tokens)
        sees[b] = (at >= (32 if b == 3 else 0))[:, None]
    assert np.isnan(got[sees]).all() and np.isnan(lse[sees]).all()
    assert not got[~sees].any() and (lse[~sees] == -np.inf).all()


@pytest.mark.parametrize("kind", ["mx", "nv"])
@pytest.mark.parametrize("tokens", [1, 3, 64])
@pytest.mark.parametrize("k", [288, 2336])
def test_matvec_every_scale_and_code(gpu, kind, tokens, k):
    """One weight a row that is not zero, with every scale byte and code, at any
    column and beside any scales: the product with ones is the weight itself."""
    announce(f"every scale and code {kind} {tokens} {k}")
    rng = np.random.default_rng(tokens + k)
    group = 32 if kind == "mx" else 16
    byte, code = np.repeat(np.arange(256), 16), np.tile(np.arange(16), 256)
    n = len(byte)
    at = rng.integers(0, k, n)
    q = np.zeros((n, k // 2), np.uint8)
    q[np.arange(n), at // 2] = code << 4 * (at % 2)
    # beside it anything but NaN
    s = rng.integers(0, 255, (n, k // group), dtype=np.uint8)
    s[s % 128 == 127] -= 1
    s[np.arange(n), at // group] = byte
    value = ref.e8m0_to_f64(byte) if kind == "mx" else ref.e4m3_to_f64(byte)
    want = as_float32(ref.LEVELS[code] * value)
    want = np.where(code % 8 == 0, np.where(np.isnan(value), np.nan, 0), want)
    x = torch.ones(tokens, k, dtype=torch.bfloat16, device="cuda")
    dev = [torch.from_numpy(a).cuda() for a in (q, s)]
    got = gpu.mxfp4_matvec(x, *dev, out_dtype=torch.float32) if kind == "mx" else \
        gpu.nvfp4_matvec(x, *dev, torch.ones(1, device="cuda"), out_dtype=torch.float32)
    assert_values(kind, got.cpu().numpy(), np.broadcast_to(want, (tokens, n)))


def holes(rng, table, pages):
    """A tenth of the entries outside the cache."""
    table = table.copy()
    table[rng.random(table.shape) < 0.1] = rng.choice([-1, pages, -7])
    return table


@pytest.mark.parametrize("page", [64, 128, 192])
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_attention_of_a_large_batch_in_wide_pages(gpu, dim, page):
    """Enough workgroups for four waves each, pages of a multiple of 64 tokens,
    contexts of several tiles a wave."""
    announce(f"large batch, wide pages {dim} {page}")
    geo = (8, dim, page)
    rng = np.random.default_rng(dim + page)
    pages, seqs = 24, 100
    host = filled_cache(rng, geo, pages)
    lengths = rng.integers(0, 1200, seqs).astype(np.int32)
    lengths[:4] = 0, 1, 1200, 1025
    table = rng.integers(0, pages, (seqs, -(-1200 // page)), dtype=np.int32)
    q = to_dev_bf16(bf16_bits(rng.standard_normal((seqs, 1, 8, dim))))
    check(gpu, geo, host, q, table, lengths)
    check(gpu, geo, host, q, holes(rng, table, pages), lengths, window=500)


@pytest.mark.parametrize("page", [64, 192, 320])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_attention_of_a_small_batch_in_wide_pages(gpu, dim, page):
    """Eight waves a workgroup, contexts of several tiles a wave, holes and windows."""
    announce(f"small batch, wide pages {dim} {page}")
    geo = (2, dim, page)
    rng = np.random.default_rng(dim + page)
    pages, seqs = 13, 5
    host = filled_cache(rng, geo, pages)
    lengths = np.array([0, 2000, 1537, 64, 1999], np.int32)
    table = rng.integers(0, pages, (seqs, -(-2000 // page)), dtype=np.int32)
    for tokens, group in ((1, 3), (9, 2)):
        q = to_dev_bf16(bf16_bits(rng.standard_normal((seqs, tokens, 2 * group, dim))))
        check(gpu, geo, host, q, table, lengths)
        check(gpu, geo, host, q, holes(rng, table, pages), lengths)
        check(gpu, geo, host, q, holes(rng, table, pages), lengths, causal=False, window=700)
