"""The RMS norm of values whose squares leave fp32."""
import pytest
import torch

import linear_ref as ref
from test_gpu_rmsnorm import check_codes

pytestmark = pytest.mark.gpu

KINDS = pytest.mark.parametrize("kind", ["block", "mx"])


def check(gpu, kind, x, w, eps, residual=None):
    """Codes, scales, 1 / rms and the sum with the residual against 64 bits."""
    q, s, *rest = (gpu.rmsnorm_blockfp8 if kind == "block" else gpu.rmsnorm_mxfp8)(x, w, residual, eps=eps, return_rstd=True)
    h, r, y = ref.norm(x, residual, w, eps)
    check_codes(kind, q, s, y)
    # a rounding, and of a subnormal number half a step of 2^-149
    assert ((rest[-1].double() - r).abs() <= 2.0 ** -22 * r + 2.0 ** -150).all()
    if residual is not None:
        assert torch.equal(rest[0].double(), h)


@KINDS
@pytest.mark.parametrize("cols", [64, 544, 4128, 7168, 16384])
@pytest.mark.parametrize("power", [-120, -90, -76, -70, -64, 60, 63, 64, 80, 100])
def test_small_and_large_values(gpu, kind, cols, power):
    g = ref.generator(cols + power)
    x = (torch.randn(5, cols, generator=g, device="cuda", dtype=torch.float64) * 2.0 ** power).bfloat16()
    w = (1 + 0.2 * torch.rand(cols, generator=g, device="cuda")).bfloat16()
    check(gpu, kind, x, w, 0.0)


@KINDS
@pytest.mark.parametrize("cols", [96, 2080, 7168])
def test_one_value_unlike_the_others(gpu, kind, cols):
    """Rows of ordinary, tiny, huge and no values, and rows with one such value, side by side."""
    g = ref.generator(cols)
    x = torch.randn(12, cols, generator=g, device="cuda", dtype=torch.float64)
    x[1] *= 2.0 ** -110
    x[2] *= 2.0 ** 90
    x[4, 7] = 2.0 ** 80
    x[5, cols - 1] = -2.0 ** 100
    x[6] = 0
    x[6, 33] = 2.0 ** -100
    x[7] *= 2.0 ** -90
    x[7, 40] = 1.0
    x[8, 9] = 2.0 ** -120
    x = x.bfloat16()
    res = torch.randn(12, cols, generator=g, device="cuda").bfloat16()
    res[1:3] = 0
    res[6:8] = 0
    w = (1 + 0.2 * torch.rand(cols, generator=g, device="cuda"))
    check(gpu, kind, x, w, 0.0, res)
    check(gpu, kind, x[[0, 2, 3, 4, 5, 8, 9]], w, 1e-6, res[[0, 2, 3, 4, 5, 8, 9]])
