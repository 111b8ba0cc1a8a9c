"""Codes in layouts that the binding copies."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1, 3, 70])
def test_rows_further_apart_than_offsets_reach(gpu, m):
    """Columns of a wide matrix, whose rows are 2^22 + 16 bytes and more apart: as rows of their own."""
    g = ref.generator(m)
    q, s, w, ws = ref.mx_operands(g, m, 40, 96)
    bq, bs, bw, bws = ref.block_operands(g, m, 40, 80)
    off = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    for apart in ((1 << 22) + 16, (1 << 23) + 1):
        def far(t):
            wide = torch.empty(t.shape[0], apart, dtype=torch.uint8, device="cuda")
            wide[:, 16:16 + t.shape[1]] = t
            return wide[:, 16:16 + t.shape[1]]
        assert torch.equal(gpu.mxfp8_matmul(far(q), s, far(w), ws), gpu.mxfp8_matmul(q, s, w, ws))
        assert torch.equal(gpu.blockfp8_matmul(far(bq), bs, far(bw), bws), gpu.blockfp8_matmul(bq, bs, bw, bws))
        assert torch.equal(gpu.mxfp8_matmul_grouped(far(q), s, far(w)[None], ws[None], off),
                           gpu.mxfp8_matmul_grouped(q, s, w[None], ws[None], off))
        t = torch.tensor([0, 96], dtype=torch.int32, device="cuda")
        assert torch.equal(gpu.mxfp8_matmul_wgrad(far(q), s, far(w), ws, t), gpu.mxfp8_matmul_wgrad(q, s, w, ws, t))


def test_rows_that_are_too_long_are_refused(gpu):
    g = ref.generator(1)
    for call, operands in ((gpu.mxfp8_matmul, ref.mx_operands), (gpu.blockfp8_matmul, ref.block_operands)):
        call(*operands(g, 2, 2, 1 << 22))
        with pytest.raises(gpu.MXQError):
            call(*operands(g, 2, 2, (1 << 22) + 32))
