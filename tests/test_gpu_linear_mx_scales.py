"""MXFP8 products under scales of every size: fp32 results, whose operands pass through
bf16, and bf16 results."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
BOTH = pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
# few tokens in several forms, and many
SIZES = pytest.mark.parametrize("m,n", [(7, 300), (40, 300), (20, 4200), (64, 8300), (647, 2100)])


def meeting(g, m, n, groups):
    """Scale bytes [m, groups] and [n, groups] of every size that, in rows i and i, add up
    to 254 in every group: all groups' products are of size 1 there."""
    rows = torch.randint(0, 255, (max(m, n), groups), generator=g, device="cuda")
    rows[:, 0] = torch.arange(max(m, n), device="cuda") * (37 if m < 255 else 1) % 255
    rows[::3, 1] = torch.arange(len(rows[::3]), device="cuda") % 10          # and the ends more often
    rows[1::3, 2] = 254 - torch.arange(len(rows[1::3]), device="cuda") % 10
    return rows[:m].to(torch.uint8), (254 - rows[:n]).to(torch.uint8)


def check_diagonal(y, q, s, w, ws):
    d = torch.arange(min(y.shape), device="cuda")
    x, v = ref.mx(q[d], s[d]), ref.mx(w[d], ws[d])
    terms = x * v
    total, want = terms.abs().sum(1), terms.sum(1)
    largest = terms.abs().view(len(d), -1, 8).amax(-1).sum(1)
    lim = ref.bound(want, total, largest, q.shape[1], y.dtype == F32)
    off = (y[d, d].double() - want).abs()
    assert (off <= lim).all(), f"{(~(off <= lim)).sum().item()} of {len(d)} are off"


@BOTH
@SIZES
def test_scales_that_meet(gpu, m, n, out):
    for k in (128, 416):
        g = ref.generator(m + k)
        q, w = ref.codes(g, m, k), ref.codes(g, n, k)
        s, ws = meeting(g, m, n, k // 32)
        check_diagonal(gpu.mxfp8_matmul(q, s, w, ws, out_dtype=out), q, s, w, ws)


@BOTH
@pytest.mark.parametrize("off,n,k", [([0, 9, 30], 300, 160), ([0, 0, 130, 700], 640, 160)])
def test_scales_that_meet_grouped(gpu, off, n, k, out):
    g = ref.generator(n)
    groups, m = len(off) - 1, off[-1]
    q, w = ref.codes(g, m, k), ref.codes(g, groups, n, k)
    s, ws = torch.zeros(m, k // 32, dtype=torch.uint8, device="cuda"), torch.zeros(groups, n, k // 32, dtype=torch.uint8, device="cuda")
    for e in range(groups):
        s[off[e]:off[e + 1]], ws[e] = meeting(g, off[e + 1] - off[e], n, k // 32)
    y = gpu.mxfp8_matmul_grouped(q, s, w, ws, torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=out)
    for e in range(groups):
        r = slice(off[e], off[e + 1])
        if r.stop > r.start:
            check_diagonal(y[r], q[r], s[r], w[e], ws[e])


@BOTH
def test_scales_that_meet_in_weight_gradients(gpu, out):
    n, k, off = 140, 200, [0, 96, 416, 427]
    g = ref.generator(3)
    a, b = ref.codes(g, n, off[-1]), ref.codes(g, k, off[-1])
    s, t = meeting(g, n, k, -(-off[-1] // 32))
    y = gpu.mxfp8_matmul_wgrad(a, s, b, t, torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=out)
    for e, (i, j) in enumerate(zip(off, off[1:])):
        part = slice(i // 32, -(-j // 32))
        pad = -(j - i) % 8
        cut = [torch.nn.functional.pad(v[:, i:j], (0, pad)) for v in (a, b)]
        check_diagonal(y[e], cut[0], s[:, part], cut[1], t[:, part])


@BOTH
@SIZES
def test_no_codes_under_large_and_small_scales(gpu, m, n, out):
    """0 times anything but NaN is 0, also in rows whose other group is not.  Against 64
    bits: a result is summed either by the matrix cores or, under such scales, again, so two
    results of equal terms are not equal bits, but each is within what ref.bound allows."""
    g = ref.generator(7)
    q, w = ref.codes(g, m, 64), ref.codes(g, n, 64)
    s = torch.full((m, 2), 127, dtype=torch.uint8, device="cuda")
    ws = torch.full((n, 2), 127, dtype=torch.uint8, device="cuda")
    x, v = ref.mx(q[:, :32].contiguous(), s[:, :1]), ref.mx(w[:, :32].contiguous(), ws[:, :1])
    q[:, 32:] = 0
    for bx, bw in ((254, 254), (254, 127), (0, 254), (0, 0)):
        s[:, 1], ws[:, 1] = bx, bw
        rows = torch.arange(min(m, 70), device="cuda")
        ref.check(gpu.mxfp8_matmul(q, s, w, ws, out_dtype=out)[rows], x[rows], v)


@BOTH
@SIZES
@pytest.mark.parametrize("codes", [(0x38, 0x38), (0, 0x38), (0x38, 0), (0, 0)])
def test_nan_scales_with_codes_of_one_sign_and_none(gpu, codes, m, n, out):
    """No infinities that cancel: a scale of NaN alone makes its row NaN."""
    q, w = (torch.full((r, 96), c, dtype=torch.uint8, device="cuda") for r, c in zip((m, n), codes))
    s, ws = (torch.full((r, 3), 127, dtype=torch.uint8, device="cuda") for r in (m, n))
    s[3, 0] = s[5, 2] = ws[9, 1] = ws[n - 1, 2] = 255
    y = gpu.mxfp8_matmul(q, s, w, ws, out_dtype=out)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[[3, 5]] = True
    bad[:, [9, n - 1]] = True
    assert torch.equal(torch.isnan(y), bad)
    assert (y[~bad] == (96 if 0 not in codes else 0)).all()


@BOTH
@SIZES
def test_large_results(gpu, m, n, out):
    """Sums of 2^100 to 2^124, which in fp32 lie past what the lifted operands hold."""
    g = ref.generator(m)
    q, w = ref.codes(g, m, 96), ref.codes(g, n, 96)
    s = torch.randint(160, 185, (m, 3), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.randint(160, 170, (n, 3), generator=g, device="cuda", dtype=torch.uint8)
    y = gpu.mxfp8_matmul(q, s, w, ws, out_dtype=out)
    rows = torch.arange(min(m, 70), device="cuda")
    ref.check(y[rows], ref.mx(q[rows], s[rows]), ref.mx(w, ws))
    assert y.abs().max() > 2.0 ** 108
