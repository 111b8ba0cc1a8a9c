"""Plain 64-bit forms of the decode operators (numpy, CPU), for their tests.

The error bounds are derived, not fitted:

matvec.  Every one of the k products is exact in fp32 (bf16 times a weight of
at most 6 significant bits), and each of the at most k + 16 additions is off by
at most 2^-23 of the largest partial sum, which is at most S = sum |x w|:
|err| <= (k + 16) 2^-23 S, plus g's product (2^-24) and the rounding of a bf16
output, 2^-8 |y| (half a unit of 8 significant bits: values in [1, 2) are 2^-7
apart).

attention.  A score is off by at most e = |scale| (d + 16) 2^-23 sum |q k| +
2^-22 |score| (its scaling and the change of base), so each weight is off by a
factor of at most exp(2 e) (its own score and the maximum), times 1 + 2^-20 for
exp2 and the rescaling by running maxima (at most 2^-22 a step over the few
dozen steps of these sizes), times 1 + 2^-8 for the weight's rounding to bf16.
The sum of weights comes from the unrounded ones.  With A = sum p |v|:
|err| <= (2^-8 + 2^-19 + 8 max e + (n + 64) 2^-23) A + 2^-8 |o|, the n term for
the additions over n visible tokens and the joins.  lse is off by at most
max e + 2^-19 + (n + 64) 2^-23 + 2^-22 |lse|.
"""
import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def bf16_to_f64(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3_to_f64(b):
    b = np.asarray(b, np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, np.ldexp(m / 8.0, -6), np.ldexp(1 + m / 8.0, e - 7))
    v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    return np.where(b & 0x80, -v, v)


def e8m0_to_f64(b):
    b = np.asarray(b, np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))


def fp4_values(packed):
    """uint8 [..., n/2] -> float64 [..., n]."""
    out = np.empty((*packed.shape[:-1], 2 * packed.shape[-1]))
    out[..., 0::2], out[..., 1::2] = LEVELS[packed & 15], LEVELS[packed >> 4]
    return out


def matvec(x, w, g=1.0, out_f32=True):
    """(y, bound) of float64 x [t, k], w [n, k] and the scale g."""
    with np.errstate(all="ignore"):
        y = g * (x @ w.T)
        s = abs(g) * (np.abs(x) @ np.abs(w.T))
        bound = (x.shape[1] + 16) * 2.0 ** -23 * s + 2.0 ** -24 * np.abs(y) + 1e-44
        if not out_f32:
            bound = bound + 2.0 ** -8 * np.abs(y) + 2.0 ** -134
    return y, bound


def page_bytes(heads, dim, page):
    return heads * page * (dim + dim // 16)


def write_page_tokens(cache, geo, slots, kc, ks, vc, vs):
    """Puts codes [n, heads, dim/2] and scales [n, heads, dim/32] of K and V at
    their places of uint8 cache [pages, page_bytes]."""
    heads, dim, page = geo
    a = heads * page * dim // 2
    c = heads * page * dim // 32
    for i, slot in enumerate(slots):
        if slot < 0 or slot // page >= cache.shape[0]:
            continue
        row, t = cache[slot // page], slot % page
        row[:a].reshape(heads, page, dim // 2)[:, t] = kc[i]
        row[a:2 * a].reshape(heads, page // 16, dim // 2, 16)[:, t // 16, :, t % 16] = vc[i]
        row[2 * a:2 * a + c].reshape(heads, page // 16, dim // 32, 16)[:, t // 16, :, t % 16] = ks[i]
        row[2 * a + c:2 * (a + c)].reshape(heads, page // 16, dim // 32, 16)[:, t // 16, :, t % 16] = vs[i]


def read_pages(cache, geo, pages):
    """float64 K and V [heads, len(pages) * page, dim] of the pages, in order."""
    heads, dim, page = geo
    a = heads * page * dim // 2
    c = heads * page * dim // 32
    ks_, vs_ = [], []
    for p in pages:
        row = cache[p]
        kc = row[:a].reshape(heads, page, dim // 2)
        vc = row[a:2 * a].reshape(heads, page // 16, dim // 2, 16).swapaxes(2, 3).reshape(heads, page, dim // 2)
        ks = row[2 * a:2 * a + c].reshape(heads, page // 16, dim // 32, 16).swapaxes(2, 3).reshape(heads, page, dim // 32)
        vs = row[2 * a + c:2 * (a + c)].reshape(heads, page // 16, dim // 32, 16).swapaxes(2, 3).reshape(heads, page, dim // 32)
        ks_.append(fp4_values(kc) * np.repeat(e8m0_to_f64(ks), 32, -1))
        vs_.append(fp4_values(vc) * np.repeat(e8m0_to_f64(vs), 32, -1))
    if not ks_:
        return np.zeros((heads, 0, dim)), np.zeros((heads, 0, dim))
    return np.concatenate(ks_, 1), np.concatenate(vs_, 1)


def attention(q, cache, geo, table, lengths, scale, causal, window):
    """(o, lse, o_bound, lse_bound) of float64 q [seqs, tokens, q_heads, dim]."""
    heads, dim, page = geo
    seqs, tokens, q_heads, _ = q.shape
    o = np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    ob, lb = np.zeros(q.shape), np.zeros(q.shape[:3])
    for b in range(seqs):
        n = int(min(max(lengths[b], 0), table.shape[1] * page))
        pages = table[b, :-(-n // page)]
        held = (pages >= 0) & (pages < cache.shape[0])
        k, v = read_pages(cache, geo, np.where(held, pages, 0)) if cache.shape[0] else (np.zeros((heads, 0, dim)),) * 2
        there = np.repeat(held, page)[:n]
        k, v = k[:, :n], v[:, :n]
        for t in range(tokens):
            pos = n - tokens + t
            j = np.arange(n)
            seen = there.copy()
            if causal:
                seen &= j <= pos
            if window > 0:
                seen &= j > pos - window
            if not cache.shape[0] or not seen.any():
                continue
            m = seen.sum()
            for h in range(q_heads):
                kk, vv = k[h * heads // q_heads][seen], v[h * heads // q_heads][seen]
                with np.errstate(all="ignore"):
                    s = scale * (kk @ q[b, t, h])
                    e = (abs(scale) * (dim + 16) * 2.0 ** -23 * (np.abs(kk) @ np.abs(q[b, t, h])) + 2.0 ** -22 * np.abs(s)).max()
                    top = s.max()
                    if np.isnan(top):
                        o[b, t, h], lse[b, t, h] = np.nan, np.nan
                        continue
                    p = np.exp(s - top)
                    lse[b, t, h] = top + np.log(p.sum())
                    p /= p.sum()
                    o[b, t, h] = p @ vv
                    lb[b, t, h] = e + 2.0 ** -19 + (m + 64) * 2.0 ** -23 + 2.0 ** -22 * abs(lse[b, t, h])
                    ob[b, t, h] = ((2.0 ** -8 + 2.0 ** -19 + 8 * e + (m + 64) * 2.0 ** -23) * (p @ np.abs(vv))
                                   + 2.0 ** -8 * np.abs(o[b, t, h]) + 2.0 ** -120)
    return o, lse, ob, lb


def assert_within(name, got, want, bound):
    """|got - want| <= bound, NaN and infinities in the same places."""
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, f"{name}: shape {got.shape} != {want.shape}"
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{name}: NaN in other places"
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), f"{name}: other infinities"
    off = np.abs(got[fine] - want[fine]) - bound[fine]
    if off.size and off.max() > 0:
        at = np.argwhere(fine)[off.argmax()]
        raise AssertionError(f"{name}: {(off > 0).sum()} of {off.size} outside; worst at {tuple(at)}: "
                             f"got {got[tuple(at)]!r}, want {want[tuple(at)]!r}, bound {bound[tuple(at)]!r}")
