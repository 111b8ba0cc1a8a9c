"""The RMS norm with 8-bit output and its gradient on the GPU against 64 bits."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def half_step(t):
    """Half of E4M3's step at t (64 bits)."""
    low = torch.clamp(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -20))), min=-6.0, max=8.0)
    return 0.5 * 2.0 ** (low - 3)


def check_codes(kind, q, s, y, slack=2.0 ** -21):
    """Scales and codes of y (64 bits): y, its scale and their quotient are each off by a
    few 2^-24; a scale near a power of two may be the next one."""
    size = 128 if kind == "block" else 32
    d = y.shape[1]
    full = torch.nn.functional.pad(y, (0, -d % size)).unflatten(-1, (-1, size))
    amax = full.abs().amax(-1)
    if kind == "block":
        S = s.double()
        assert ((S - amax / 448).abs() <= slack * amax / 448 + 2.0 ** -149).all()
        unit = torch.where(S == 0, torch.ones_like(S), S)
    else:
        def byte(a):
            return torch.where(a > 0, torch.floor(torch.log2(a.clamp(min=2.0 ** -140))) - 8 + 127, 0 * a).clamp(0, 254)
        b = s.double()
        assert ((b == byte(amax * (1 - slack))) | (b == byte(amax * (1 + slack)))).all()
        unit = torch.exp2(b - 127)
    t = (full / unit[..., None]).flatten(-2)[:, :d].clamp(-448, 448)
    got = ref.e4m3_values(q)
    lim = half_step(t) + slack * t.abs() + 1e-12
    assert torch.isfinite(got).all() and ((got - t).abs() <= lim).all()


COLS = [32, 64, 96, 128, 160, 480, 512, 544, 2048, 2080, 4096, 4128, 7168, 8192, 8224, 16384]


@pytest.mark.parametrize("kind", ["block", "mx"])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 3, 37])
def test_norm(gpu, kind, rows, cols):
    g = ref.generator(rows + cols)
    x = (torch.randn(rows, cols, generator=g, device="cuda") * 3).bfloat16()
    res = torch.randn(rows, cols, generator=g, device="cuda").bfloat16() if cols % 64 else None
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(F32 if cols % 96 == 0 else BF16)
    call = gpu.rmsnorm_blockfp8 if kind == "block" else gpu.rmsnorm_mxfp8
    q, s, *rest, rstd, y16 = call(x, w, res, eps=1e-5, return_rstd=True, return_normed=True)
    h, r, y = ref.norm(x, res, w, 1e-5)
    if res is not None:
        assert torch.equal(rest[0].double(), h)
    else:
        assert not rest
    assert ((rstd.double() - r).abs() <= 2.0 ** -22 * r).all()
    assert ((y16.double() - y).abs() <= (2.0 ** -8 + 2.0 ** -20) * y.abs()).all()
    check_codes(kind, q, s, y)


@pytest.mark.parametrize("cols", [8, 24, 136, 1000, 5000])
def test_norm_block_odd_columns(gpu, cols):
    g = ref.generator(cols)
    x = torch.randn(5, cols, generator=g, device="cuda").bfloat16()
    w = torch.rand(cols, generator=g, device="cuda").bfloat16()
    q, s = gpu.rmsnorm_blockfp8(x, w)
    assert s.shape == (5, -(-cols // 128))
    check_codes("block", q, s, ref.norm(x, None, w, 1e-6)[2])


@pytest.mark.parametrize("kind", ["block", "mx"])
def test_norm_shapes_and_strides(gpu, kind):
    g = ref.generator(3)
    call = gpu.rmsnorm_blockfp8 if kind == "block" else gpu.rmsnorm_mxfp8
    big = torch.randn(2, 5, 800, generator=g, device="cuda").bfloat16()
    w = torch.rand(1280, generator=g, device="cuda").bfloat16()[::2][:256]
    x, res = big[:, :, 8:264], big[:, :, 400:656]
    q, s, h = call(x, w, res)
    assert h.shape == x.shape and q.shape == (10, 256)
    a = call(x.contiguous().view(10, 256), w.contiguous(), res.contiguous().view(10, 256))
    assert torch.equal(q, a[0]) and torch.equal(s, a[1]) and torch.equal(h.view(10, 256), a[2])
    rows = big[0][:, 8:264]  # 2-D, rows apart: read in place
    assert torch.equal(call(rows, w)[0], call(rows.contiguous(), w)[0])
    assert torch.equal(call(big[0][:, 4:260], w)[0], call(big[0][:, 4:260].contiguous(), w)[0])
    one = call(x[0, 0], w)
    assert one[0].shape == (1, 256)
    q, s, h = call(x[:0], w, res[:0])
    assert q.shape == (0, 256) and h.shape == (0, 5, 256)


@pytest.mark.parametrize("kind", ["block", "mx"])
def test_norm_rows_that_are_zero_or_not_finite(gpu, kind):
    call = gpu.rmsnorm_blockfp8 if kind == "block" else gpu.rmsnorm_mxfp8
    g = ref.generator(4)
    x = torch.randn(8, 512, generator=g, device="cuda").bfloat16()
    clean = call(x, torch.ones(512, device="cuda"))
    x2 = x.clone()
    x2[1] = 0
    x2[2, 7] = float("nan")
    x2[3, 9] = float("inf")
    w = torch.ones(512, device="cuda")
    q, s = call(x2, w)
    keep = [0, 4, 5, 6, 7]
    assert torch.equal(q[keep], clean[0][keep]) and torch.equal(s[keep], clean[1][keep])
    assert ((q[1] & 127) == 0).all() and (s[1] == 0).all()
    nan = torch.isnan(s[2]) if kind == "block" else s[2] == 255
    assert nan.all() and ((q[2] & 127) == 127).all()
    group = 0
    assert (torch.isnan(s[3, group]) if kind == "block" else s[3, group] == 255)
    # one weight that is not finite reaches its group alone
    w[200] = float("inf")
    q, s = call(x, w)
    bad = torch.isnan(s) if kind == "block" else s == 255
    assert bad[:, 1 if kind == "block" else 6].all() and bad.sum() == 8
    # a zero row without eps is 0 / 0
    q, s = call(torch.zeros(1, 512, dtype=BF16, device="cuda"), torch.ones(512, device="cuda"), eps=0.0)
    assert ((q & 127) == 127).all()


def test_norm_of_small_and_large_values(gpu):
    g = ref.generator(5)
    for scale in (2.0 ** -60, 2.0 ** -40, 2.0 ** 40, 2.0 ** 55):
        x = (torch.randn(3, 1024, generator=g, device="cuda") * scale).bfloat16()
        w = torch.rand(1024, generator=g, device="cuda").bfloat16()
        for kind, call in (("block", gpu.rmsnorm_blockfp8), ("mx", gpu.rmsnorm_mxfp8)):
            q, s = call(x, w, eps=0.0)
            check_codes(kind, q, s, ref.norm(x, None, w, 0.0)[2])


@pytest.mark.parametrize("kind", ["block", "mx"])
def test_norm_weights_of_any_size(gpu, kind):
    """Scales far from 1: codes as good as anywhere else."""
    g = ref.generator(6)
    x = torch.randn(4, 640, generator=g, device="cuda").bfloat16()
    w = torch.exp2(torch.randint(-100, 100, (640,), generator=g, device="cuda").float()).repeat(1)
    w = w.view(5, 128)[:, :1].repeat(1, 128).flatten().contiguous()
    q, s = (gpu.rmsnorm_blockfp8 if kind == "block" else gpu.rmsnorm_mxfp8)(x, w)
    check_codes(kind, q, s, ref.norm(x, None, w, 1e-6)[2])


# -- the gradient --------------------------------------------------------------------------


@pytest.mark.parametrize("rows,cols", [(1, 8), (2, 64), (5, 520), (37, 2048), (300, 96), (1030, 160), (700, 4104), (600, 8200), (3, 16384)])
@pytest.mark.parametrize("joined", [False, True])
def test_backward(gpu, rows, cols, joined):
    g = ref.generator(rows + cols)
    h = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
    dy = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
    dh = torch.randn(rows, cols, generator=g, device="cuda").bfloat16() if joined else None
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(BF16 if cols % 16 else F32)
    r = (1 / (h.double().square().mean(-1) + 1e-6).sqrt()).float()
    dx, dw = gpu.rmsnorm_backward(dy, h, w, r, dh=dh)
    ex, ew = ref.norm_backward(dy, h, w, r, dh)
    # fp32 sums of cols, then rows, terms: at most their number of additions in a row in
    # a lane, 8 values a piece, and in the tree above
    gu = (dy.double() * w.double() * h.double() * r.double()[:, None]).abs()
    size = r.double()[:, None] * ((dy.double() * w.double()).abs() + (h.double() * r.double()[:, None]).abs() * gu.mean(-1, keepdim=True))
    if joined:
        size = size + dh.double().abs()
    assert ((dx.double() - ex).abs() <= 2.0 ** -8 * ex.abs() * (1 + 2.0 ** -8) + 64 * ref.EPS32 * size).all()
    each = (dy.double() * h.double() * r.double()[:, None]).abs().sum(0)
    assert ((dw.double() - ew).abs() <= (rows / 64 + 64) * 2 * ref.EPS32 * each).all()
    again = gpu.rmsnorm_backward(dy, h, w, r, dh=dh)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_backward_against_differences(gpu):
    """Central differences of the 64-bit norm, along random directions."""
    g = ref.generator(8)
    rows, cols = 6, 96
    x = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).bfloat16()
    dy = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
    rstd = gpu.rmsnorm_blockfp8(x, w, return_rstd=True)[2]
    dx, dw = gpu.rmsnorm_backward(dy, x, w, rstd)

    def loss(x, w):
        return (ref.norm(x, None, w, 1e-6)[2] * dy.double()).sum()

    for _ in range(4):
        v = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.float64)
        u = torch.randn(cols, generator=g, device="cuda", dtype=torch.float64)
        e = 1e-5
        by = (loss(x.double() + e * v, w) - loss(x.double() - e * v, w)) / (2 * e)
        # dx is rounded to bf16: off by half a step in each place
        assert (by - (dx.double() * v).sum()).abs() <= (2.0 ** -8 * (dx.double() * v).abs()).sum() + 1e-6
        by = (loss(x.double(), w.double() + e * u) - loss(x.double(), w.double() - e * u)) / (2 * e)
        assert (by - (dw.double() * u).sum()).abs() <= 1e-5 * (dw.double() * u).abs().sum() + 1e-6


def test_backward_shapes_strides_and_nothing(gpu):
    g = ref.generator(9)
    big = torch.randn(3, 4, 900, generator=g, device="cuda").bfloat16()
    w = torch.rand(256, generator=g, device="cuda").bfloat16()
    r = torch.rand(24, generator=g, device="cuda")[::2]
    dy, h, dh = big[..., 0:256], big[..., 304:560], big[..., 601:857]
    dx, dw = gpu.rmsnorm_backward(dy, h, w, r, dh=dh)
    flat = [t.contiguous().view(12, 256) for t in (dy, h, dh)]
    ex, ew = gpu.rmsnorm_backward(flat[0], flat[1], w, r.contiguous(), dh=flat[2])
    assert dx.shape == dy.shape and torch.equal(dx.view(12, 256), ex) and torch.equal(dw, ew)
    dx, dw = gpu.rmsnorm_backward(dy[:0], h[:0], w, r[:0])
    assert dx.shape == (0, 4, 256) and (dw == 0).all()


def test_refusals(gpu):
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    r = torch.ones(4, device="cuda")
    for bad in (lambda: gpu.rmsnorm_mxfp8(x.float(), w), lambda: gpu.rmsnorm_mxfp8(x, w.half()), lambda: gpu.rmsnorm_mxfp8(x, w, x.float()),
                lambda: gpu.rmsnorm_backward(x, x.float(), w, r), lambda: gpu.rmsnorm_backward(x, x, w, r.double())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: gpu.rmsnorm_mxfp8(x[:, :48], w[:48]), lambda: gpu.rmsnorm_blockfp8(x[:, :4], w[:4]), lambda: gpu.rmsnorm_mxfp8(x, w[:32]),
                lambda: gpu.rmsnorm_mxfp8(x, w, x[:2]), lambda: gpu.rmsnorm_mxfp8(x.cpu(), w), lambda: gpu.rmsnorm_mxfp8(x, w.cpu()),
                lambda: gpu.rmsnorm_mxfp8(x, w, x.cpu()), lambda: gpu.rmsnorm_backward(x, x[:2], w, r), lambda: gpu.rmsnorm_backward(x, x, w, r[:2]),
                lambda: gpu.rmsnorm_backward(x, x, w, r, dh=x[:, :32]), lambda: gpu.rmsnorm_backward(x, x, w, r.cpu())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gpu.MXQError):
        gpu.rmsnorm_mxfp8(torch.zeros(1, 16416, dtype=BF16, device="cuda"), torch.ones(16416, device="cuda"))
    with pytest.raises(gpu.MXQError):
        gpu.rmsnorm_backward(*[torch.zeros(1, 16416, dtype=BF16, device="cuda")] * 2, torch.ones(16416, device="cuda"), r[:1])


def test_offsets_past_32_bits(gpu):
    rows, cols = 600000, 7168
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    g = ref.generator(10)
    x[-3:] = torch.randn(3, cols, generator=g, device="cuda").bfloat16()
    w = torch.rand(cols, generator=g, device="cuda").bfloat16()
    q, s, r = gpu.rmsnorm_blockfp8(x, w, return_rstd=True)
    check_codes("block", q[-3:], s[-3:], ref.norm(x[-3:], None, w, 1e-6)[2])
    del q, s
    dx, dw = gpu.rmsnorm_backward(x, x, w, r)
    ex, ew = ref.norm_backward(x[-3:], x[-3:], w, r[-3:], None)
    assert ((dx[-3:].double() - ex).abs() <= 2.0 ** -7 * ex.abs() + 1e-5).all()
    assert ((dw.double() - ew).abs() <= 1e-4 * ew.abs() + 1e-4).all()


def test_more_rows_than_one_launch_has(gpu):
    """Rows of one wave, four to a workgroup of 256 threads: 2^31 threads are 2^25 rows."""
    rows = (1 << 25) + 9
    g = ref.generator(12)
    x = torch.ones(rows, 8, dtype=BF16, device="cuda")
    at = torch.tensor([0, 1, (1 << 25) - 1, 1 << 25, (1 << 25) + 1, rows - 1], device="cuda")
    x[at] = torch.randn(6, 8, generator=g, device="cuda").bfloat16()
    w = torch.rand(8, generator=g, device="cuda").bfloat16()
    q, s, h, r, y16 = gpu.rmsnorm_blockfp8(x, w, x, return_rstd=True, return_normed=True)
    assert torch.equal(h, x + x)
    _, er, ey = ref.norm(x[at], x[at], w, 1e-6)
    check_codes("block", q[at], s[at], ey)
    assert ((r[at].double() - er).abs() <= 2.0 ** -22 * er).all()
    assert ((y16[at].double() - ey).abs() <= (2.0 ** -8 + 2.0 ** -20) * ey.abs()).all()
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (r[rest] == r[2]).all() and (s[rest] == s[2]).all() and (q[rest] == q[2]).all()


def test_no_columns(gpu):
    x = torch.zeros(3, 0, dtype=BF16, device="cuda")
    w = torch.zeros(0, device="cuda")
    for call in (gpu.rmsnorm_blockfp8, gpu.rmsnorm_mxfp8):
        q, s, r = call(x, w, return_rstd=True)
        assert q.shape == s.shape == (3, 0) and torch.isnan(r).all()
    dx, dw = gpu.rmsnorm_backward(x, x, w, r)
    assert dx.shape == (3, 0) and dw.shape == (0,)


@pytest.mark.parametrize("cols", [96, 5120])
def test_outputs_in_place(gpu, cols):
    """h over x or the residual, dx over dy, dh or h: as into memory of their own."""
    from block_scaled_precision_mxfp8_amd import linear
    g = ref.generator(13)
    x, res, dh = (torch.randn(30, cols, generator=g, device="cuda").bfloat16() for _ in range(3))
    w = torch.rand(cols, generator=g, device="cuda")
    q, s, h, r = gpu.rmsnorm_mxfp8(x, w, res, return_rstd=True)
    for over in (0, 1):
        a = [x.clone(), res.clone()]
        q2, s2 = torch.empty_like(q), torch.empty_like(s)
        linear._call("mxq_rmsnorm", x.device, linear._RMSNORM.pack(
            a[0].data_ptr(), a[1].data_ptr(), w.data_ptr(), q2.data_ptr(), s2.data_ptr(), a[over].data_ptr(), 0, 0,
            30, cols, cols, cols, 1e-6, 1, 0))
        assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(h, a[over])
    dx, dw = gpu.rmsnorm_backward(x, h, w, r, dh=dh)
    for over in range(3):
        a = [x.clone(), h.clone(), dh.clone()]
        dw2 = torch.empty_like(dw)
        n = gpu.load().mxq_rmsnorm_backward_workspace_size(30, cols)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        linear._call("mxq_rmsnorm_backward", x.device, linear._RMSNORM_BACKWARD.pack(
            *(t.data_ptr() for t in a), w.data_ptr(), r.data_ptr(), a[over].data_ptr(), dw2.data_ptr(),
            ws.data_ptr(), n, 30, cols, cols, cols, cols, 1, 0))
        assert torch.equal(dx, a[over]) and torch.equal(dw, dw2)
