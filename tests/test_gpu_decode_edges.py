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


# (tokens, query heads): one and two strips of 16 rows; rows that share decoded tiles
@pytest.mark.parametrize("tokens,group", [(5, 2), (20, 1), (50, 2), (150, 2)])
@pytest.mark.parametrize("geo", [(2, 64, 16), (1, 96, 48), (2, 128, 64), (1, 192, 192), (1, 256, 16)], ids=str)
def test_values_past_bf16_where_some_rows_see_them(gpu, geo, tokens, group):
    """V scales of 253 and 254: with small codes ordinary values, with large
    ones past bf16's range, where the result may be infinite, NaN or what real
    numbers give.  On tokens that only some rows of a tile see (causal, window)
    they count for those rows alone."""
    heads, dim, page = geo
    announce(f"values past bf16 {geo} {tokens}x{group}")
    rng = np.random.default_rng(dim + tokens)
    seqs = max(2, -(-130 // heads // -(-tokens * group // 16)))  # enough workgroups to share tiles from 49 rows on
    width = -(-400 // page)
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
    for causal, window in ((True, 0), (True, 3), (True, 40), (False, tokens + 9)):
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
