"""Block-FP8 products whose two scales leave the range of fp32 when they are multiplied,
although the result does not."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
BOTH = pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
# few tokens in each form of rows to a workgroup; many in tiles of 128 and of 256
SIZES = pytest.mark.parametrize("m,n", [(5, 260), (40, 260), (12, 4200), (40, 8300), (647, 2100), (4000, 3300)])


@BOTH
@SIZES
def test_scales_of_every_pair_of_sizes(gpu, m, n, out):
    """Exponents of -148 to 127 on either side, the same in both blocks of a row."""
    k = 256
    g = ref.generator(m + n)
    q, w = ref.codes(g, m, k), ref.codes(g, n, k)
    S = torch.exp2(torch.randint(-148, 128, (m, 1), generator=g, device="cuda").double())
    wS = torch.exp2(torch.randint(-148, 128, (-(-n // 128), 1), generator=g, device="cuda").double())
    S[:2, 0] = torch.tensor([2.0 ** 100, 2.0 ** -140])
    wS[0], wS[-1] = 2.0 ** -45, 2.0 ** 60
    S = (S * (1 + torch.rand(m, 2, generator=g, device="cuda", dtype=torch.float64))).float().clamp(max=2.0 ** 127)
    wS = (wS * (1 + torch.rand(wS.shape[0], 2, generator=g, device="cuda", dtype=torch.float64))).float().clamp(max=2.0 ** 127)
    y = gpu.blockfp8_matmul(q, S, w, wS, out_dtype=out)
    rows = torch.arange(min(m, 60), device="cuda")
    cols = torch.cat([torch.arange(0, 10), torch.arange(124, 132), torch.arange(n - 10, n)]).cuda()
    x = ref.x_block(q[rows], S[rows])
    v = ref.e4m3_values(w[cols]) * wS[cols // 128].double().repeat_interleave(128, -1)
    want, total, largest = ref.product(x, v)
    # where the terms are numbers of fp32; a block's term below 2^-124 may be lost (as a
    # subnormal number, times up to four)
    fits = total < 2.0 ** 127
    assert (want.abs() > 2.0 ** -100)[fits].any()
    lim = ref.bound(want, total, largest, k, out == F32) + 2 * 2.0 ** -124
    assert ((y[rows][:, cols].double() - want).abs() <= lim)[fits].all()


@BOTH
@SIZES
def test_no_codes_under_large_scales_are_zero(gpu, m, n, out):
    """0 times scales whose product is past fp32."""
    g = ref.generator(1)
    q, w = ref.codes(g, m, 272), ref.codes(g, n, 272)
    S = torch.full((m, 3), 2.0 ** 120, device="cuda")
    wS = torch.full((-(-n // 128), 3), 2.0 ** 120, device="cuda")
    q[:] = 0
    q[1::2] = 0x80  # minus zero
    assert (gpu.blockfp8_matmul(q, S, w, wS, out_dtype=out) == 0).all()


@BOTH
@SIZES
def test_smallest_products_under_large_scales(gpu, m, n, out):
    """2^-18 times 1.5 * 2^128."""
    q = torch.zeros(m, 144, dtype=torch.uint8, device="cuda")
    w = torch.zeros(n, 144, dtype=torch.uint8, device="cuda")
    q[:, 5], w[:, 5], w[:, 130] = 1, 1, 0x7E
    S = torch.full((m, 2), 2.0 ** 100, device="cuda")
    wS = torch.full((-(-n // 128), 2), 1.5 * 2.0 ** 28, device="cuda")
    y = gpu.blockfp8_matmul(q, S, w, wS, out_dtype=out)
    assert (y.double() == 1.5 * 2.0 ** 110).all()


@BOTH
@SIZES
def test_scales_whose_product_is_subnormal(gpu, m, n, out):
    """2.2 * 2^-141, of which fp32 keeps nine bits, times 2^24: a result near 2^-115 with all its bits."""
    q = torch.full((m, 128), 0x7E, dtype=torch.uint8, device="cuda")
    w = torch.full((n, 128), 0x7E, dtype=torch.uint8, device="cuda")
    S = torch.full((m, 1), 1.37 * 2.0 ** -100, device="cuda") * (1 + torch.arange(m, device="cuda")[:, None] / m / 8)
    wS = torch.full((-(-n // 128), 1), 1.61 * 2.0 ** -41, device="cuda")
    y = gpu.blockfp8_matmul(q, S, w, wS, out_dtype=out).double()
    want = 128 * 448.0 ** 2 * S.double() * wS[0].double()
    # a sum of 128 in fp32, the product of the scales and the last product: as ref.bound has it
    assert ((y - want).abs() <= ((128 / 16 + 64) * 2.0 ** -23 + (0 if out == F32 else 2.0 ** -8 + 2.0 ** -10)) * want).all()


@BOTH
@SIZES
def test_scales_that_are_not_finite(gpu, m, n, out):
    """An infinite scale times what is not 0 is infinite; a scale of NaN gives NaN; no others are touched."""
    g = ref.generator(4)
    q, S, w, wS = ref.block_operands(g, m, n, 256)
    clean = gpu.blockfp8_matmul(q, S, w, wS, out_dtype=out)
    q[2:4] = q[2:4] & 0x7F
    q[2:4, :128] = 0x38
    w[7:9] = w[7:9] & 0x7F
    w[7:9, :128] = 0x30
    before = gpu.blockfp8_matmul(q, S, w, wS, out_dtype=out)
    S[2, 0] = float("inf")
    S[4, 1] = float("nan")
    y = gpu.blockfp8_matmul(q, S, w, wS, out_dtype=out)
    assert torch.isposinf(y[2, 7:9]).all() and torch.isnan(y[4]).all()
    assert not torch.isfinite(y[2]).any()
    keep = [i for i in range(m) if i not in (2, 4)]
    assert torch.equal(y[keep], before[keep]) and torch.isfinite(clean).all()


@BOTH
def test_grouped(gpu, out):
    """Few and many rows a group."""
    for m in (30, 900):
        g = ref.generator(m)
        q, S, w, wS = ref.block_operands(g, m, 260, 256, (2,))
        S, wS = S * 2.0 ** 90, wS * 2.0 ** 90
        S[::2] *= 2.0 ** -180
        q[1::2] = 0
        wS[1] *= 2.0 ** -120
        off = torch.tensor([0, m // 3, m], dtype=torch.int32, device="cuda")
        y = gpu.blockfp8_matmul_grouped(q, S, w, wS, off, out_dtype=out)
        assert (y[1::2] == 0).all()
        for e, (i, j) in enumerate(((0, m // 3), (m // 3, m))):
            rows = torch.arange(i, min(j, i + 20), device="cuda")
            x, v = ref.x_block(q[rows], S[rows]), ref.w_block(w[e], wS[e])
            want, total, largest = ref.product(x, v)
            lim = ref.bound(want, total, largest, 256, out == F32) + 2.0 ** -123
            assert ((y[rows].double() - want).abs() <= lim).all()
