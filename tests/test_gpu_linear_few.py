"""The kernel of products of few tokens: every number of token tiles with every number of
weight rows to a workgroup, and contractions whose scales a wave loads more than once."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
BOTH = pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
KINDS = pytest.mark.parametrize("kind", ["block", "mx"])


def run(gpu, kind, m, n, k, out):
    g = ref.generator(m + n + k)
    q, s, w, ws = (ref.block_operands if kind == "block" else ref.mx_operands)(g, m, n, k)
    # a guard on both sides of what is written
    guard = torch.full((m + 2, n), 3.0, dtype=out, device="cuda")
    y = (gpu.blockfp8_matmul if kind == "block" else gpu.mxfp8_matmul)(q, s, w, ws, out_dtype=out, out=guard[1:1 + m])
    assert (guard[0] == 3).all() and (guard[-1] == 3).all()
    at = torch.cat([torch.arange(0, 18), torch.arange(62, 66), torch.arange(n - 70, n)])
    at = at[(at >= 0) & (at < n)].unique().cuda()
    if kind == "block":
        x = ref.x_block(q, s)
        v = ref.e4m3_values(w[at]) * ws[at // 128].double().repeat_interleave(128, -1)[:, :k]
    else:
        x, v = ref.mx(q, s), ref.mx(w[at], ws[at])
    ref.check(y[:, at], x, v)


@BOTH
@KINDS
@pytest.mark.parametrize("n", [4096, 4097, 8192, 8193])
@pytest.mark.parametrize("m", [1, 16, 17, 32, 33, 48, 49, 64])
def test_tokens_and_rows(gpu, kind, m, n, out):
    """16, 32 and 64 weight rows to a workgroup begin past 4096 and 8192 of them."""
    run(gpu, kind, m, n, 672, out)


@BOTH
@KINDS
@pytest.mark.parametrize("m,n,k", [(3, 4200, 8320), (20, 4200, 8320), (40, 8300, 8320), (64, 8300, 16640), (1, 4200, 16640),
                                   (5, 300, 16640), (33, 300, 16640), (64, 300, 33408)])
def test_scales_loaded_again(gpu, kind, m, n, k, out):
    """More than 16 steps of 128 to each of four or eight waves."""
    run(gpu, kind, m, n, k, out)


@BOTH
@KINDS
@pytest.mark.parametrize("rows,groups,n", [(24, 16, 300), (24, 3, 300), (10, 40, 300), (10, 3, 300), (30, 3, 3000)])
def test_grouped(gpu, kind, rows, groups, n, out):
    """`rows` a group on average, unevenly; few and many weight rows over all groups."""
    g = ref.generator(rows * groups)
    m, k = rows * groups, 544
    cut = torch.randint(0, m + 1, (groups - 1,), generator=g, device="cuda").sort().values.tolist()
    off = [0, *cut, m]
    q, s, w, ws = (ref.block_operands if kind == "block" else ref.mx_operands)(g, m, n, k, (groups,))
    y = (gpu.blockfp8_matmul_grouped if kind == "block" else gpu.mxfp8_matmul_grouped)(
        q, s, w, ws, torch.tensor(off, dtype=torch.int32, device="cuda"), out_dtype=out)
    for e, (i, j) in enumerate(zip(off, off[1:])):
        if j > i:
            if kind == "block":
                ref.check(y[i:j], ref.x_block(q[i:j], s[i:j]), ref.w_block(w[e], ws[e]))
            else:
                ref.check(y[i:j], ref.mx(q[i:j], s[i:j]), ref.mx(w[e], ws[e]))
