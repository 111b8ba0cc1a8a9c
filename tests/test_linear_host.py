"""The 8-bit linear operators on the host (no GPU): the C entry points refuse bad
arguments before launching anything, and the binding refuses bad tensors."""
import struct

import pytest
import torch

import block_scaled_precision_mxfp8_amd as mxq
from block_scaled_precision_mxfp8_amd import linear

P = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return mxq.load()


MATMUL = dict(x=P, sx=P, ldx=128, ld_sx=4, w=P, sw=P, ldw=128, ld_sw=4, w_group_stride=0, sw_group_stride=0, y=P, ldy=8,
              y_group_stride=0, offsets=0, m=4, n=8, k=128, groups=0, out_fp32=0, reserved=0)
DENSE, GROUPED = ("blockfp8_matmul", "mxq_matmul"), ("blockfp8_matmul_grouped", "mxq_matmul_grouped", "mxq_matmul_wgrad")


def matmul(lib, fn, **kw):
    d = dict(MATMUL)
    if fn in GROUPED:
        d.update(offsets=P, groups=3)
    d.update(kw)
    assert list(d) == list(MATMUL)
    return getattr(lib, fn)(linear._MATMUL.pack(*d.values()), None)


def test_struct_sizes():
    """The packed bytes are the header's structures on this machine."""
    assert linear._MATMUL.size == 19 * 8 and linear._RMSNORM.size == 14 * 8 and linear._RMSNORM_BACKWARD.size == 15 * 8
    assert struct.calcsize("P") == struct.calcsize("N") == 8


def test_matmul_refusals(lib):
    for fn in DENSE + GROUPED:
        for name in ("m", "n", "k", "ldx", "ldw", "ld_sx", "ld_sw", "ldy", "w_group_stride", "sw_group_stride", "y_group_stride"):
            assert matmul(lib, fn, **{name: -16}) == mxq.MXQ_EINVAL, name
        assert getattr(lib, fn)(None, None) == mxq.MXQ_EINVAL
        assert matmul(lib, fn, reserved=1) == mxq.MXQ_EINVAL
        for name in ("x", "sx", "w", "sw", "y"):
            assert matmul(lib, fn, **{name: 0}) == mxq.MXQ_EINVAL, name
        assert matmul(lib, fn, ldx=112) == mxq.MXQ_ESHAPE
        assert matmul(lib, fn, ldw=112) == mxq.MXQ_ESHAPE
        assert matmul(lib, fn, ldy=7) == mxq.MXQ_ESHAPE
        blocks = 1 if fn.startswith("blockfp8") else 4
        assert matmul(lib, fn, ld_sx=blocks - 1) == mxq.MXQ_ESHAPE
        assert matmul(lib, fn, ld_sw=blocks - 1) == mxq.MXQ_ESHAPE
        assert matmul(lib, fn, x=P + 8) == mxq.MXQ_EALIGN
        assert matmul(lib, fn, w=P + 8) == mxq.MXQ_EALIGN
        assert matmul(lib, fn, ldx=136) == mxq.MXQ_EALIGN
        assert matmul(lib, fn, ldw=136) == mxq.MXQ_EALIGN
        assert matmul(lib, fn, w_group_stride=1032) == mxq.MXQ_EALIGN
        assert matmul(lib, fn, y=P + 1) == mxq.MXQ_EALIGN
        assert matmul(lib, fn, y=P + 2, out_fp32=1) == mxq.MXQ_EALIGN
        if fn.startswith("blockfp8"):
            assert matmul(lib, fn, sx=P + 2) == mxq.MXQ_EALIGN and matmul(lib, fn, sw=P + 2) == mxq.MXQ_EALIGN
        assert matmul(lib, fn, ldx=(1 << 22) + 16) == mxq.MXQ_ESIZE
        assert matmul(lib, fn, ldw=1 << 23) == mxq.MXQ_ESIZE
        assert matmul(lib, fn, m=1 << 31) == mxq.MXQ_ESIZE
        assert matmul(lib, fn, n=1 << 31, ldy=1 << 31) == mxq.MXQ_ESIZE
        assert matmul(lib, fn, ld_sx=1 << 62) == mxq.MXQ_ESIZE
        assert matmul(lib, fn, ldy=1 << 62) == mxq.MXQ_ESIZE
        assert matmul(lib, fn, m=0, x=0, sx=0, w=0, sw=0, y=0) == mxq.MXQ_OK
        assert matmul(lib, fn, n=0, x=0, sx=0, w=0, sw=0, y=0) == mxq.MXQ_OK
    assert matmul(lib, "blockfp8_matmul", k=24) == mxq.MXQ_ESHAPE
    assert matmul(lib, "mxq_matmul", k=48) == mxq.MXQ_ESHAPE
    for fn in DENSE:
        assert matmul(lib, fn, offsets=P) == mxq.MXQ_EINVAL
        assert matmul(lib, fn, groups=1) == mxq.MXQ_EINVAL
    for fn in GROUPED:
        assert matmul(lib, fn, offsets=0) == mxq.MXQ_EINVAL
        assert matmul(lib, fn, groups=-1) == mxq.MXQ_EINVAL
        assert matmul(lib, fn, offsets=P + 2) == mxq.MXQ_EALIGN
        assert matmul(lib, fn, groups=65536) == mxq.MXQ_ESIZE
        assert matmul(lib, fn, groups=0, offsets=0) == mxq.MXQ_OK
        assert matmul(lib, fn, w_group_stride=1 << 62) == mxq.MXQ_ESIZE


NORM = dict(x=P, residual=P, weight=P, q=P, scale=P, h=P, y=0, rstd=0, rows=4, cols=64, ldx=64, ld_residual=64, eps=1e-6,
            weight_fp32=0, reserved=0)
BACK = dict(dy=P, h=P, dh=P, weight=P, rstd=P, dx=P, dweight=P, workspace=P, workspace_bytes=1 << 30, rows=4, cols=64,
            ld_dy=64, ldh=64, ld_dh=64, weight_fp32=0, reserved=0)


def norm(lib, fn, **kw):
    d = {**NORM, **kw}
    assert list(d) == list(NORM)
    return getattr(lib, fn)(linear._RMSNORM.pack(*d.values()), None)


def back(lib, **kw):
    d = {**BACK, **kw}
    assert list(d) == list(BACK)
    return lib.mxq_rmsnorm_backward(linear._RMSNORM_BACKWARD.pack(*d.values()), None)


def test_rmsnorm_refusals(lib):
    for fn in ("blockfp8_rmsnorm", "mxq_rmsnorm"):
        assert getattr(lib, fn)(None, None) == mxq.MXQ_EINVAL
        for name in ("rows", "cols", "ldx", "ld_residual"):
            assert norm(lib, fn, **{name: -8}) == mxq.MXQ_EINVAL
        for name in ("x", "weight", "q", "scale", "h"):
            assert norm(lib, fn, **{name: 0}) == mxq.MXQ_EINVAL, name
        assert norm(lib, fn, reserved=1) == mxq.MXQ_EINVAL
        assert norm(lib, fn, cols=4) == mxq.MXQ_ESHAPE
        assert norm(lib, fn, ldx=56) == mxq.MXQ_ESHAPE
        assert norm(lib, fn, ld_residual=56) == mxq.MXQ_ESHAPE
        for name in ("x", "residual", "weight", "h", "y"):
            assert norm(lib, fn, **{name: P + 8}) == mxq.MXQ_EALIGN, name
        assert norm(lib, fn, q=P + 4) == mxq.MXQ_EALIGN
        assert norm(lib, fn, rstd=P + 2) == mxq.MXQ_EALIGN
        assert norm(lib, fn, ldx=68) == mxq.MXQ_EALIGN
        assert norm(lib, fn, ld_residual=68) == mxq.MXQ_EALIGN
        assert norm(lib, fn, cols=16416, ldx=16416, ld_residual=16416) == mxq.MXQ_ESIZE
        assert norm(lib, fn, rows=1 << 60) == mxq.MXQ_ESIZE
        assert norm(lib, fn, rows=0, x=0, weight=0, q=0, scale=0) == mxq.MXQ_OK
    assert norm(lib, "mxq_rmsnorm", cols=48) == mxq.MXQ_ESHAPE
    assert norm(lib, "blockfp8_rmsnorm", scale=P + 2) == mxq.MXQ_EALIGN


def test_rmsnorm_backward_refusals(lib):
    size = lib.mxq_rmsnorm_backward_workspace_size
    assert size(4, 64) > 0 and size(4, 64) % (64 * 4) == 0
    assert size(0, 64) == size(4, 0) == size(-1, 64) == size(4, 16416) == 0
    assert size(1 << 40, 16384) < 1 << 27  # does not grow with the rows
    assert lib.mxq_rmsnorm_backward(None, None) == mxq.MXQ_EINVAL
    for name in ("rows", "cols", "ld_dy", "ldh", "ld_dh"):
        assert back(lib, **{name: -8}) == mxq.MXQ_EINVAL
    for name in ("dy", "h", "weight", "rstd", "dx", "dweight", "workspace"):
        assert back(lib, **{name: 0}) == mxq.MXQ_EINVAL, name
    assert back(lib, reserved=1) == mxq.MXQ_EINVAL
    assert back(lib, cols=60) == mxq.MXQ_ESHAPE
    for name in ("ld_dy", "ldh", "ld_dh"):
        assert back(lib, **{name: 56}) == mxq.MXQ_ESHAPE
        assert back(lib, **{name: 68}) == mxq.MXQ_EALIGN
    for name in ("dy", "h", "dh", "weight", "dx", "workspace"):
        assert back(lib, **{name: P + 8}) == mxq.MXQ_EALIGN, name
    assert back(lib, rstd=P + 2) == mxq.MXQ_EALIGN and back(lib, dweight=P + 2) == mxq.MXQ_EALIGN
    assert back(lib, workspace_bytes=size(4, 64) - 1) == mxq.MXQ_ESIZE
    assert back(lib, cols=16416, ld_dy=16416, ldh=16416, ld_dh=16416) == mxq.MXQ_ESIZE
    assert back(lib, rows=1 << 60) == mxq.MXQ_ESIZE
    assert back(lib, cols=0) == mxq.MXQ_OK


def test_binding_refuses_cpu_tensors_and_types():
    q = torch.zeros(2, 128, dtype=torch.uint8)
    for fn in (mxq.blockfp8_matmul, mxq.mxfp8_matmul):
        with pytest.raises(ValueError):
            fn(q, q, q, q)
        with pytest.raises(TypeError):
            fn(q.float(), q, q, q)
        with pytest.raises(TypeError):
            fn(None, q, q, q)
    for fn in (mxq.blockfp8_matmul_grouped, mxq.mxfp8_matmul_grouped, mxq.mxfp8_matmul_wgrad):
        with pytest.raises(ValueError):
            fn(q, q, q, q, torch.zeros(2, dtype=torch.int32))
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    for fn in (mxq.rmsnorm_blockfp8, mxq.rmsnorm_mxfp8):
        with pytest.raises(ValueError):
            fn(x, x[0])
        with pytest.raises(TypeError):
            fn(x.float(), x[0])
    with pytest.raises(ValueError):
        mxq.rmsnorm_backward(x, x, x[0], torch.ones(2))
