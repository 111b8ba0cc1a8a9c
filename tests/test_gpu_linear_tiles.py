"""The kernel of products of many tokens: what the tests of test_gpu_linear.py hold for few
tokens (dense products with at most 16384 tiles of 64 rows by one column are the other
kernel's), and contractions long enough that the scales' places in LDS are used in turn."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
BOTH = pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
KINDS = pytest.mark.parametrize("kind", ["block", "mx"])
# tiles of 128 x 128, and (bf16 results) of 256 x 256; the last ones short both ways
SMALL, LARGE = (647, 2100), (4000, 3300)
SIZES = pytest.mark.parametrize("m,n", [SMALL, LARGE], ids=["small", "large"])


def many(m, n):
    """Whether a dense product is this kernel's."""
    return m > 64 and -(-m // 64) * n > 16384


def operands(kind, g, m, n, k, lead=()):
    return (ref.block_operands if kind == "block" else ref.mx_operands)(g, m, n, k, lead)


def values(kind, q, s, w, ws):
    return (ref.x_block(q, s), ref.w_block(w, ws)) if kind == "block" else (ref.mx(q, s), ref.mx(w, ws))


def call(mxq, kind, grouped=False):
    return getattr(mxq, ("blockfp8" if kind == "block" else "mxfp8") + "_matmul" + ("_grouped" if grouped else ""))


def some(n):
    """Indexes at the first and last tile and around a border between tiles."""
    at = torch.cat([torch.arange(0, 20), torch.arange(122, 134), torch.arange(250, 262), torch.arange(n - 20, n)])
    return at[(at >= 0) & (at < n)].unique().cuda()


def check_some(y, kind, q, s, w, ws):
    rows, cols = some(y.shape[0]), some(y.shape[1])
    if kind == "block":
        x = ref.x_block(q[rows], s[rows])
        n, k = w.shape
        v = ref.e4m3_values(w[cols]) * ws[cols // 128].double().repeat_interleave(128, -1)[:, :k]
    else:
        x, v = ref.mx(q[rows], s[rows]), ref.mx(w[cols], ws[cols])
    ref.check(y[rows][:, cols], x, v)


def turns(kind, g, m, n, k, lead=()):
    """Operands whose scales change from each four steps of 128 to the next, x's against
    w's: every step counts alike, and a scale of another step is off by 8 or more."""
    q, s, w, ws = operands(kind, g, m, n, k, lead)
    per = 4 if kind == "block" else 16
    e = (torch.arange(s.shape[-1], device="cuda") // per * 3 + torch.arange(s.shape[-1], device="cuda") % per // (per // 4)) % 7 * 3 - 9
    if kind == "block":
        return q, s.clamp(0.5, 2) * torch.exp2(e.float()), w, ws.clamp(0.5, 2) * torch.exp2(-e.float())
    return q, (s.int() % 3 + 126 + e).to(torch.uint8), w, (ws.int() % 3 + 126 - e).to(torch.uint8)


@BOTH
@KINDS
@pytest.mark.parametrize("k", [1024, 1056, 1536, 1568, 2080, 7168])
def test_contractions_of_many_steps(gpu, kind, k, out):
    """8, 9, 12, 13, 17 and 56 steps: two to fourteen groups of four with scales of their own."""
    m, n = SMALL
    q, s, w, ws = turns(kind, ref.generator(k), m, n, k)
    check_some(call(gpu, kind)(q, s, w, ws, out_dtype=out), kind, q, s, w, ws)


@KINDS
@pytest.mark.parametrize("k", [1056, 1536, 7168])
def test_contractions_of_many_steps_large_tiles(gpu, kind, k):
    m, n = LARGE
    q, s, w, ws = turns(kind, ref.generator(k + 1), m, n, k)
    check_some(call(gpu, kind)(q, s, w, ws), kind, q, s, w, ws)


@BOTH
@KINDS
@pytest.mark.parametrize("off,n,k", [([0, 290, 290, 700], 640, 1568), ([5, 133, 900], 300, 4128), ([0, 1500, 2700], 4400, 1056)])
def test_grouped_contractions_of_many_steps(gpu, kind, off, n, k, out):
    m, groups = off[-1] + 3, len(off) - 1
    q, s, w, ws = turns(kind, ref.generator(n), m, n, k, (groups,))
    y = torch.full((m, n), -5.0, dtype=out, device="cuda")
    call(gpu, kind, True)(q, s, w, ws, torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=out, out=y)
    for e in range(groups):
        r = slice(off[e], off[e + 1])
        if r.stop > r.start:
            check_some(y[r], kind, q[r], s[r], w[e], ws[e])
    assert (y[:off[0]] == -5).all() and (y[off[-1]:] == -5).all()


@BOTH
@pytest.mark.parametrize("off,tokens,n,k", [([0, 96, 1664, 3300], 3300, 140, 200), ([32, 64, 2592, 2607], 2607, 260, 130),
                                            ([0, 1600, 3216], 3216, 2500, 2600)])
def test_wgrad_of_many_steps(gpu, off, tokens, n, k, out):
    """Groups of more than 1024 tokens that begin anywhere, the last ending inside a scale's 32."""
    dyt, dys, xt, xs = turns("mx", ref.generator(tokens), n, k, tokens)
    pad = -(-tokens // 16) * 16
    wide = [torch.full((r, pad), 0x7F, dtype=torch.uint8, device="cuda") for r in (n, k)]
    wide[0][:, :tokens], wide[1][:, :tokens] = dyt, xt
    y = gpu.mxfp8_matmul_wgrad(wide[0][:, :tokens], dys, wide[1][:, :tokens], xs,
                               torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=out)
    for e, (i, j) in enumerate(zip(off, off[1:])):
        part = [t[:, i:j].contiguous() for t in (dyt, xt)]
        scales = [t[:, i // 32:-(-j // 32)].contiguous() for t in (dys, xs)]
        check_some(y[e], "mx", part[0], scales[0], part[1], scales[1])


@BOTH
@SIZES
@KINDS
def test_nan_stays_in_its_sums(gpu, kind, m, n, out):
    k = 288
    q, s, w, ws = operands(kind, ref.generator(2), m, n, k)
    clean = call(gpu, kind)(q, s, w, ws, out_dtype=out)
    assert torch.isfinite(clean).all()
    q, s, w, ws = q.clone(), s.clone(), w.clone(), ws.clone()
    q[130, 40] = 0x7F
    w[300, 100] = 0xFF
    s[m - 1, -1] = 255 if kind == "mx" else float("nan")
    ws[-1, 0] = 255 if kind == "mx" else float("nan")
    y = call(gpu, kind)(q, s, w, ws, out_dtype=out)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[[130, m - 1]] = True
    bad[:, 300] = True
    bad[:, n - 1 if kind == "mx" else (n - 1) // 128 * 128:] = True
    assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], clean[~bad])


@SIZES
def test_mx_scales_of_every_size(gpu, m, n):
    """Scale bytes that meet their counterpart: products near 1 whatever the bytes."""
    g = ref.generator(5)
    b, c = (torch.arange(r, device="cuda") % 255 for r in (m, n))
    q, w = ref.codes(g, m, 64), ref.codes(g, n, 64)
    s, ws = b.to(torch.uint8)[:, None].repeat(1, 2), (254 - c).to(torch.uint8)[:, None].repeat(1, 2)
    y = gpu.mxfp8_matmul(q, s, w, ws)
    i = torch.cat([torch.arange(r, min(m, n), 255) for r in (0, 1, 2, 100, 127, 252, 253, 254)]).cuda()
    # the same byte in every column of a row, so places off the diagonal of equal bytes overflow or vanish
    d = i[i < min(m, n)]
    x, v = ref.mx(q[d], s[d]), ref.mx(w[d], ws[d])
    e = (x * v).sum(1)
    lim = ref.bound(e, (x * v).abs().sum(1), (x * v).abs().view(len(d), 8, 8).amax(-1).sum(1), 64, False)
    assert ((y[d, d].double() - e).abs() <= lim).all()


@BOTH
@SIZES
def test_block_scales_zero_and_large(gpu, m, n, out):
    q, s, w, ws = ref.block_operands(ref.generator(8), m, n, 256)
    s[0] = 0
    s[1] = 1e-30
    s[2] = 1e30
    s[4:6, 0] *= 1e12
    y = gpu.blockfp8_matmul(q, s, w, ws, out_dtype=out)
    assert (y[0] == 0).all()
    check_some(y, "block", q, s, w, ws)


@BOTH
@SIZES
@KINDS
def test_strides_types_and_out(gpu, kind, m, n, out):
    k = 288
    q, s, w, ws = operands(kind, ref.generator(11), m, n, k)
    want = call(gpu, kind)(q, s, w, ws, out_dtype=out)
    wide = torch.full((m, k + 64), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:, 16:16 + k] = q
    odd = torch.zeros(n * k + 1, dtype=torch.uint8, device="cuda")
    odd[1:] = w.flatten()
    s_wide = torch.full((m, s.shape[1] + 3), 99, dtype=s.dtype, device="cuda")
    s_wide[:, 1:1 + s.shape[1]] = s
    e8 = torch.float8_e8m0fnu if kind == "mx" else torch.float32
    guard = torch.full((m * n + 9,), 3.0, dtype=out, device="cuda")
    y = guard[1:1 + m * n].view(m, n)  # not 16-byte aligned: stored by elements
    got = call(gpu, kind)(wide[:, 16:16 + k].view(torch.float8_e4m3fn), s_wide[:, 1:1 + s.shape[1]].view(e8),
                          odd[1:].view(n, k), ws.t().contiguous().t(), out_dtype=out, out=y)
    assert got is y and torch.equal(y, want) and guard[0] == 3 and (guard[1 + m * n:] == 3).all()


@BOTH
@SIZES
def test_block_odd_contraction(gpu, m, n, out):
    """Multiples of 16 that are none of 32."""
    for k in (16, 144, 1072):
        q, s, w, ws = ref.block_operands(ref.generator(k), m, n, k)
        check_some(gpu.blockfp8_matmul(q, s, w, ws, out_dtype=out), "block", q, s, w, ws)


@BOTH
@SIZES
@KINDS
def test_no_contraction(gpu, kind, m, n, out):
    q, s, w, ws = operands(kind, ref.generator(3), m, n, 0)
    y = torch.full((m, n), 7.0, dtype=out, device="cuda")
    assert (call(gpu, kind)(q, s, w, ws, out_dtype=out, out=y) == 0).all()


@BOTH
@SIZES
@KINDS
def test_equal_calls_give_equal_bytes(gpu, kind, m, n, out):
    q, s, w, ws = operands(kind, ref.generator(9), m, n, 1568)
    first = call(gpu, kind)(q, s, w, ws, out_dtype=out)
    for _ in range(3):
        assert torch.equal(call(gpu, kind)(q, s, w, ws, out_dtype=out), first)
