"""The 8-bit products on the GPU against 64 bits: sizes where a tile, a workgroup or a
step ends, both formats and results, ragged groups, strides, scales of every size."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def operands(kind, g, m, n, k, lead=()):
    return (ref.block_operands if kind == "block" else ref.mx_operands)(g, m, n, k, lead)


def values(kind, q, s, w, ws):
    return (ref.x_block(q, s), ref.w_block(w, ws)) if kind == "block" else (ref.mx(q, s), ref.mx(w, ws))


def call(mxq, kind, grouped=False):
    name = ("blockfp8" if kind == "block" else "mxfp8") + "_matmul" + ("_grouped" if grouped else "")
    return getattr(mxq, name)


SHAPES = [(1, 1, 32), (1, 64, 128), (2, 17, 160), (3, 130, 416), (15, 300, 544), (16, 33, 2080), (17, 513, 96), (31, 4100, 64),
          (33, 129, 1056), (48, 8200, 128), (49, 100, 7168), (64, 257, 288), (65, 31, 4128), (130, 640, 160), (200, 129, 224),
          (257, 1000, 32), (300, 2050, 352), (520, 520, 512), (1030, 130, 96), (640, 3000, 672)]


@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["block", "mx"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul(gpu, kind, m, n, k, out):
    g = ref.generator(m * 7 + n + k)
    q, s, w, ws = operands(kind, g, m, n, k)
    y = call(gpu, kind)(q, s, w, ws, out_dtype=out)
    assert y.shape == (m, n) and y.dtype == out
    ref.check(y, *values(kind, q, s, w, ws))


@pytest.mark.parametrize("m,n,k", [(5, 70, 16), (70, 200, 48), (300, 300, 144), (9, 40, 2064)])
def test_matmul_block_odd_contraction(gpu, m, n, k):
    """Contractions that are no multiple of 32 end inside a piece of a line."""
    g = ref.generator(k)
    q, s, w, ws = ref.block_operands(g, m, n, k)
    for out in (BF16, F32):
        ref.check(gpu.blockfp8_matmul(q, s, w, ws, out_dtype=out), ref.x_block(q, s), ref.w_block(w, ws))


@pytest.mark.parametrize("kind", ["block", "mx"])
def test_matmul_large_tiles(gpu, kind):
    """Enough tiles for the largest ones, the last of them short both ways."""
    m, n, k = 4000, 3300, 416
    g = ref.generator(1)
    q, s, w, ws = operands(kind, g, m, n, k)
    y = call(gpu, kind)(q, s, w, ws)
    rows = torch.cat([torch.arange(0, 40), torch.arange(250, 262), torch.arange(3960, 4000)])
    cols = torch.cat([torch.arange(0, 40), torch.arange(250, 262), torch.arange(3260, 3300)])
    x, wv = values(kind, q, s, w, ws)
    ref.check(y[rows][:, cols], x[rows], wv[cols])
    full = x @ wv.t().contiguous()
    assert ((y.double() - full).norm() / full.norm()).item() < 2.0 ** -8


@pytest.mark.parametrize("kind", ["block", "mx"])
@pytest.mark.parametrize("m", [5, 70, 300])
def test_matmul_no_contraction_or_nothing(gpu, kind, m):
    g = ref.generator(3)
    q, s, w, ws = operands(kind, g, m, 40, 0)
    for out in (BF16, F32):
        y = torch.full((m, 40), 7.0, dtype=out, device="cuda")
        assert (call(gpu, kind)(q, s, w, ws, out_dtype=out, out=y) == 0).all()
    q, s, w, ws = operands(kind, g, 0, 40, 64)
    assert call(gpu, kind)(q, s, w, ws).shape == (0, 40)
    q, s, w, ws = operands(kind, g, m, 0, 64)
    assert call(gpu, kind)(q, s, w, ws).shape == (m, 0)


@pytest.mark.parametrize("kind", ["block", "mx"])
@pytest.mark.parametrize("m", [9, 300])
def test_matmul_strides_types_and_out(gpu, kind, m):
    n, k = 150, 288
    g = ref.generator(11)
    q, s, w, ws = operands(kind, g, m, n, k)
    want = call(gpu, kind)(q, s, w, ws)
    wide = torch.zeros(m, k + 64, dtype=torch.uint8, device="cuda")
    wide[:, 16:16 + k] = q
    odd = torch.zeros(n * k + 1, dtype=torch.uint8, device="cuda")
    odd[1:] = w.flatten()
    s_wide = torch.zeros(m, s.shape[1] + 3, dtype=s.dtype, device="cuda")
    s_wide[:, 1:1 + s.shape[1]] = s
    ws_t = ws.t().contiguous().t()
    e8 = torch.float8_e8m0fnu if kind == "mx" else torch.float32
    out = torch.full((m, n), 3.0, dtype=BF16, device="cuda")
    got = call(gpu, kind)(wide[:, 16:16 + k].view(torch.float8_e4m3fn), s_wide[:, 1:1 + s.shape[1]].view(e8),
                          odd[1:].view(n, k), ws_t, out=out)
    assert got is out and torch.equal(out, want)


def test_mx_scales_of_every_size(gpu):
    """Scale bytes that meet their counterpart: products near 1 whatever the bytes."""
    g = ref.generator(5)
    for m in (200, 40):  # the tiles, the few-token kernel
        b = torch.arange(m, device="cuda").clamp(max=254).to(torch.uint8)[:, None].repeat(1, 2)
        if m < 100:
            b = (b.int() * 6).to(torch.uint8)
        q, w = ref.codes(g, m, 64), ref.codes(g, m, 64)
        y = gpu.mxfp8_matmul(q, b, w, 254 - b)
        d = torch.arange(m, device="cuda")
        x, v = ref.mx(q, b), ref.mx(w, 254 - b)
        e = (x * v).sum(1)
        lim = ref.bound(e, (x * v).abs().sum(1), (x * v).abs().view(m, 8, 8).amax(-1).sum(1), 64, False)
        assert ((y[d, d].double() - e).abs() <= lim).all()
        # fp32 results: bf16 operands, scales that bf16 numbers can have
        keep = (b[:, 0] >= 12) & (b[:, 0] <= 242)
        y = gpu.mxfp8_matmul(q, b, w, 254 - b, out_dtype=F32)
        lim = ref.bound(e, (x * v).abs().sum(1), e, 64, True)
        assert ((y[d, d].double() - e).abs() <= lim)[keep].all()


@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["block", "mx"])
@pytest.mark.parametrize("m", [20, 300])
def test_nan_stays_in_its_sums(gpu, kind, m, out):
    n, k = 260, 288
    g = ref.generator(2)
    q, s, w, ws = operands(kind, g, m, n, k)
    clean = call(gpu, kind)(q, s, w, ws, out_dtype=out)
    q2, s2, w2, ws2 = q.clone(), s.clone(), w.clone(), ws.clone()
    q2[3, 40] = 0x7F                                     # a token's code
    w2[9, 100] = 0xFF                                    # a weight's code
    if kind == "mx":
        s2[11, 8] = 255                                  # a token's last scale
        ws2[259, 0] = 255
        cols = [259]
    else:
        s2[11, 2] = float("nan")
        ws2[2, 0] = float("nan")
        cols = list(range(256, 260))
    y = call(gpu, kind)(q2, s2, w2, ws2, out_dtype=out)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[[3, 11]] = True
    bad[:, [9] + cols] = True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], clean[~bad])


def test_block_scales_zero_and_large(gpu):
    g = ref.generator(8)
    for m in (6, 140):
        q, s, w, ws = ref.block_operands(g, m, 130, 256)
        s[0] = 0
        s[1] = 1e-30
        s[2] = 1e30
        s[4:6, 0] *= 1e12
        for out in (BF16, F32):
            y = gpu.blockfp8_matmul(q, s, w, ws, out_dtype=out)
            assert (y[0] == 0).all()
            ref.check(y, ref.x_block(q, s), ref.w_block(w, ws))


def test_bf16_results_keep_what_the_instruction_holds(gpu):
    """One large product beside 7 small ones: fp32 results have all of them, bf16
    results at least down to 2^-13 of the large one."""
    q = torch.zeros(1, 128, dtype=torch.uint8, device="cuda")
    w = torch.full((1, 128), 0x38, dtype=torch.uint8, device="cuda")
    s = torch.full((1, 4), 127, dtype=torch.uint8, device="cuda")
    q[0, :8] = torch.tensor([0x7E] + [0x01] * 7)
    want = 448 + 7 * 2.0 ** -9
    assert gpu.mxfp8_matmul(q, s, w, s, out_dtype=F32).item() == want
    assert abs(gpu.mxfp8_matmul(q, s, w, s).item() - want) <= 448 * 2.0 ** -8


# -- grouped ------------------------------------------------------------------------


GROUPS = {"one": [0, 40], "empty ones": [0, 0, 13, 13, 13, 90, 90], "singles": list(range(0, 9)), "uneven": [0, 300, 301, 333, 600],
          "gaps at both ends": [7, 20, 20, 61, 77], "many": [min(3 * i, 190) for i in range(71)], "all empty": [5, 5, 5]}


@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["block", "mx"])
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("spare", [0, 30, 2500])
def test_grouped(gpu, kind, name, spare, out):
    """Few rows a group, many, and rows that no group has, which keep what they hold."""
    off = GROUPS[name]
    m, groups, n, k = off[-1] + spare, len(off) - 1, 270, 224
    g = ref.generator(len(name) + spare)
    q, s, w, ws = operands(kind, g, m, n, k, (groups,))
    y = torch.full((m, n), -5.0, dtype=out, device="cuda")
    call(gpu, kind, True)(q, s, w, ws, torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=out, out=y)
    assert (y[:off[0]] == -5).all() and (y[off[-1]:] == -5).all()
    for e in range(groups):
        r = slice(off[e], off[e + 1])
        if off[e + 1] > off[e]:
            ref.check(y[r], *values(kind, q[r], s[r], w[e], ws[e]))


def test_grouped_equals_one_by_one_at_full_size(gpu):
    """The largest tiles, and weights that lie apart."""
    off = [0, 900, 900, 2100, 4100]
    n, k = 3300, 288
    g = ref.generator(4)
    q, s, w, ws = ref.mx_operands(g, 4100, n, k, (4,))
    apart = torch.zeros(4, 2, n, k, dtype=torch.uint8, device="cuda")
    apart[:, 1] = w
    y = gpu.mxfp8_matmul_grouped(q, s, apart[:, 1], ws, torch.tensor(off, dtype=torch.int32, device="cuda"))
    for e in range(4):
        r = slice(off[e], off[e + 1])
        x, v = ref.mx(q[r], s[r]), ref.mx(w[e], ws[e])
        full = x @ v.t().contiguous()
        if r.stop > r.start:
            assert ((y[r].double() - full).norm() / full.norm()).item() < 2.0 ** -8
            ref.check(y[r][:30, :30], x[:30], v[:30])
            ref.check(y[r][-30:, -30:], x[-30:], v[-30:])


@pytest.mark.parametrize("m", [60, 1200])
def test_grouped_offsets_outside_stay_inside(gpu, m):
    g = ref.generator(6)
    q, s, w, ws = ref.block_operands(g, m, 40, 128, (3,))
    off = torch.tensor([-7, 10, 10, m + 99], dtype=torch.int32, device="cuda")
    guard = torch.full((m + 8, 40), 9.0, dtype=BF16, device="cuda")
    y = guard[4:4 + m]
    gpu.blockfp8_matmul_grouped(q, s, w, ws, off, out=y)
    assert (guard[:4] == 9).all() and (guard[-4:] == 9).all()
    ref.check(y[:10], ref.x_block(q[:10], s[:10]), ref.w_block(w[0], ws[0]))
    ref.check(y[10:], ref.x_block(q[10:], s[10:]), ref.w_block(w[2], ws[2]))


def test_grouped_keeps_groups_apart(gpu):
    g = ref.generator(12)
    q, s, w, ws = ref.mx_operands(g, 50, 64, 64, (3,))
    off = torch.tensor([0, 20, 30, 50], dtype=torch.int32, device="cuda")
    clean = gpu.mxfp8_matmul_grouped(q, s, w, ws, off)
    w[1] = 0x7F
    y = gpu.mxfp8_matmul_grouped(q, s, w, ws, off)
    assert torch.isnan(y[20:30]).all() and torch.equal(y[:20], clean[:20]) and torch.equal(y[30:], clean[30:])


# -- weight gradients ------------------------------------------------------------------


def wgrad_reference(dyt, dys, xt, xs, off, tokens):
    a, b = ref.mx(dyt, dys), ref.mx(xt, xs)
    edge = [tokens if v >= tokens else max(v, 0) // 32 * 32 for v in off]
    return [(a[:, i:max(i, j)], b[:, i:max(i, j)]) for i, j in zip(edge, edge[1:])]


@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(40, 70), (130, 300)])
@pytest.mark.parametrize("off,tokens", [([0, 64], 64), ([0, 32, 32, 224, 352], 352), ([0, 100], 100), ([0, 96, 128, 207], 207),
                                        ([32, 64, 160], 256), ([0, 0, 0], 64), ([0, 40, 100], 128), ([0, 640, 1312], 1312),
                                        ([32 * i for i in range(20)], 32 * 19), ([-5, 64, 999], 130)])
def test_wgrad(gpu, off, tokens, n, k, out):
    g = ref.generator(tokens + n)
    dyt, dys, xt, xs = ref.mx_operands(g, n, k, tokens)
    pad = -(-tokens // 16) * 16 + 16  # rows of their own, as quantize_colwise_t leaves them, with anything behind
    wide = [torch.full((r, pad), 0x7F, dtype=torch.uint8, device="cuda") for r in (n, k)]
    wide[0][:, :tokens], wide[1][:, :tokens] = dyt, xt
    y = gpu.mxfp8_matmul_wgrad(wide[0][:, :tokens], dys, wide[1][:, :tokens], xs,
                               torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=out)
    assert y.shape == (len(off) - 1, n, k)
    for e, (a, b) in enumerate(wgrad_reference(dyt, dys, xt, xs, off, tokens)):
        if a.shape[1] == 0:
            assert (y[e] == 0).all()
        else:
            ref.check(y[e], a, b)


def test_wgrad_large_tiles(gpu):
    """Enough tiles for the largest ones, groups of very different lengths."""
    off = [0, 32, 32, 1056, 1184, 1280, 1297]
    n, k, tokens = 1300, 1700, 1297
    g = ref.generator(31)
    dyt, dys, xt, xs = ref.mx_operands(g, n, k, tokens)
    y = gpu.mxfp8_matmul_wgrad(dyt, dys, xt, xs, torch.tensor(off, dtype=torch.int32, device="cuda"))
    for e, (a, b) in enumerate(wgrad_reference(dyt, dys, xt, xs, off, tokens)):
        full = a @ b.t().contiguous()
        if a.shape[1]:
            assert ((y[e].double() - full).norm() / full.norm()).item() < 2.0 ** -8
            ref.check(y[e][-40:, -40:], a[-40:], b[-40:])
            ref.check(y[e][250:262, 250:262], a[250:262], b[250:262])
        else:
            assert (y[e] == 0).all()


def test_wgrad_of_quantized_columns(gpu):
    """From bf16 to the gradient: both operands by quantize_colwise_t."""
    g = ref.generator(17)
    tokens, n, k = 150, 96, 160
    dy = torch.randn(tokens, n, generator=g, device="cuda").bfloat16()
    x = torch.randn(tokens, k, generator=g, device="cuda").bfloat16()
    a = gpu.quantize_colwise_t(dy, rowwise=False, fake_quant=False)
    b = gpu.quantize_colwise_t(x, rowwise=False, fake_quant=False, ldt=256)
    y = gpu.mxfp8_matmul_wgrad(a["q_colT"], a["s_colT"], b["q_colT"], b["s_colT"],
                               torch.tensor([0, tokens], dtype=torch.int32, device="cuda"), out_dtype=F32)[0]
    dq = [ref.mx(t["q_colT"].contiguous(), t["s_colT"]) for t in (a, b)]
    ref.check(y, *dq)
    exact = dy.double().t() @ x.double()
    # two roundings to E4M3, of at most 2^-4 each, off in random directions
    assert ((y.double() - exact).norm() / exact.norm()).item() < 2 * 2.0 ** -4


# -- calls -------------------------------------------------------------------------------


def test_refusals(gpu):
    g = ref.generator(0)
    q, s, w, ws = ref.mx_operands(g, 4, 8, 64)
    bq, bs, bw, bws = ref.block_operands(g, 4, 8, 64)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        gpu.mxfp8_matmul(q.int(), s, w, ws)
    with pytest.raises(TypeError):
        gpu.mxfp8_matmul(q.view(torch.float8_e5m2), s, w, ws)
    with pytest.raises(TypeError):
        gpu.mxfp8_matmul(q, s.float(), w, ws)
    with pytest.raises(TypeError):
        gpu.blockfp8_matmul(bq, bs.bfloat16(), bw, bws)
    with pytest.raises(TypeError):
        gpu.mxfp8_matmul(q, s, w, ws, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        gpu.mxfp8_matmul_grouped(q, s, w[None], ws[None], [0, 4])
    with pytest.raises(TypeError):
        gpu.mxfp8_matmul_grouped(q, s, w[None], ws[None], off.long())
    for bad in (lambda: gpu.mxfp8_matmul(q[0], s, w, ws), lambda: gpu.mxfp8_matmul(q, s[:, :1], w, ws),
                lambda: gpu.mxfp8_matmul(q, s, w[:, :32], ws), lambda: gpu.mxfp8_matmul(q, s, w, ws[:4]),
                lambda: gpu.mxfp8_matmul(q[:, :48], s, w[:, :48], ws), lambda: gpu.mxfp8_matmul(q, s, w.cpu(), ws),
                lambda: gpu.mxfp8_matmul(q, s.cpu(), w, ws), lambda: gpu.mxfp8_matmul(q.cpu(), s, w, ws),
                lambda: gpu.mxfp8_matmul(q, s, w, ws, out=torch.empty(8, 4, dtype=BF16, device="cuda")),
                lambda: gpu.mxfp8_matmul(q, s, w, ws, out=torch.empty(4, 16, dtype=BF16, device="cuda")[:, ::2]),
                lambda: gpu.blockfp8_matmul(bq[:, :40], bs, bw[:, :40], bws), lambda: gpu.blockfp8_matmul(bq, bs, bw, bws[:, :0]),
                lambda: gpu.mxfp8_matmul_grouped(q, s, w, ws, off), lambda: gpu.mxfp8_matmul_grouped(q, s, w[None], ws[None], off[:1]),
                lambda: gpu.mxfp8_matmul_grouped(q, s, w[None], ws[None], off.cpu()),
                lambda: gpu.mxfp8_matmul_wgrad(q, s, w[:, :32], ws, off), lambda: gpu.mxfp8_matmul_wgrad(q, s, w, ws, off[:0]),
                lambda: gpu.mxfp8_matmul_wgrad(q, s[:, :1], w, ws, off)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gpu.MXQError):  # rows further apart than 32-bit offsets reach
        gpu.mxfp8_matmul(*ref.mx_operands(g, 1, 1, (1 << 22) + 32))


def test_equal_calls_give_equal_bytes(gpu):
    g = ref.generator(9)
    for m in (3, 60, 400):
        q, s, w, ws = ref.block_operands(g, m, 300, 544)
        first = gpu.blockfp8_matmul(q, s, w, ws, out_dtype=F32)
        for _ in range(3):
            assert torch.equal(gpu.blockfp8_matmul(q, s, w, ws, out_dtype=F32), first)


def test_offsets_past_32_bits(gpu):
    """Weights whose last expert lies past 2^32 bytes, and results past 2^31 elements."""
    n, k, groups = 8192, 8192, 66
    w = torch.zeros(groups, n, k, dtype=torch.uint8, device="cuda")
    ws = torch.full((groups, n, k // 32), 127, dtype=torch.uint8, device="cuda")
    g = ref.generator(41)
    w[-1, -40:] = ref.codes(g, 40, k)
    q, s, _, _ = ref.mx_operands(g, 70, 1, k)
    off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    off[-1] = 70
    y = gpu.mxfp8_matmul_grouped(q, s, w, ws, off)
    assert (y[:, :-40] == 0).all()
    ref.check(y[:, -40:], ref.mx(q, s), ref.mx(w[-1, -40:], ws[-1, -40:]))
    del w, ws
    m, n = 300000, 7500
    q, s, w, ws = ref.mx_operands(g, m, n, 32)
    y = gpu.mxfp8_matmul(q, s, w, ws)
    ref.check(y[-40:, -40:], ref.mx(q[-40:], s[-40:]), ref.mx(w[-40:], ws[-40:]))


def test_streams_and_graphs(gpu):
    """Calls on a stream of their own, and captured beside each other with workspaces
    of their own, replayed on new inputs with other work between."""
    g = ref.generator(13)
    few, many = ref.block_operands(g, 5, 300, 256), ref.mx_operands(g, 300, 200, 288)
    dyt = ref.mx_operands(g, 60, 90, 128)
    off = torch.tensor([0, 64, 128], dtype=torch.int32, device="cuda")
    x = torch.randn(37, 512, generator=g, device="cuda").bfloat16()
    weight = torch.rand(512, generator=g, device="cuda").bfloat16()
    rstd = torch.rand(37, generator=g, device="cuda")

    def run():
        return [gpu.blockfp8_matmul(*few), gpu.mxfp8_matmul(*many, out_dtype=F32), gpu.mxfp8_matmul_wgrad(*dyt, off),
                *gpu.rmsnorm_blockfp8(x, weight, x, return_rstd=True), *gpu.rmsnorm_backward(x, x, weight, rstd),
                *gpu.rmsnorm_backward(x, x, weight, rstd, dh=x)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.synchronize()
    for a, b in zip(got, run()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(4):
        few[0].copy_(ref.codes(g, 5, 256))
        many[2].copy_(ref.codes(g, 200, 288))
        x.copy_(torch.randn(37, 512, generator=g, device="cuda"))
        graph.replay()
        eager = run()
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("groups", [65534, 65535])
@pytest.mark.parametrize("m", [1, 40])
def test_grouped_most_groups(gpu, groups, m):
    g = ref.generator(groups + m)
    q, s, w, ws = ref.block_operands(g, m, 8, 16, (groups,))
    of = torch.randint(0, groups, (m,), generator=g, device="cuda").sort().values
    of[-1] = groups - 1
    off = torch.searchsorted(of, torch.arange(groups + 1, device="cuda")).int()
    y = gpu.blockfp8_matmul_grouped(q, s, w, ws, off, out_dtype=F32)
    for i in range(m):
        ref.check(y[i:i + 1], ref.x_block(q[i:i + 1], s[i:i + 1]), ref.w_block(w[of[i]], ws[of[i]]))
