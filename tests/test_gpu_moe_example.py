"""examples/moe_8bit.py: the 8-bit linear operators together, as programs use them."""
import os
import subprocess
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(gpu):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_8bit
    return moe_8bit


def exact(layer, x, res, dout, routing):
    """The layer and its gradients in 64 bits, without quantizing, for a given routing."""
    p, slot, offsets = routing
    h = (x.double() + res.double()).requires_grad_()
    norm, up, down = (t.double().requires_grad_() for t in (layer.norm, layer.up, layer.down))
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * norm
    out = h
    expert = torch.searchsorted(offsets.long(), slot, right=True) - 1
    for c in range(slot.shape[1]):
        u = (up[expert[:, c]] @ y[..., None])[..., 0]
        d = (down[expert[:, c]] @ torch.nn.functional.silu(u)[..., None])[..., 0]
        out = out + p[:, c, None].double() * d
    return out.detach(), torch.autograd.grad(out, (h, norm, up, down), dout.double())


@pytest.mark.parametrize("tokens", [1, 45, 300])
def test_gradients(example, tokens):
    """Every product has two operands in E4M3, each off by at most 2^-4 of an element
    and by 0.03 of the whole (a uniform error in half a step, over all places in a
    binade); at most five products lie on a way, so 0.03 * sqrt(2 * 5) < 0.1 of a
    result's norm, and half as much again for bf16 between them and few tokens."""
    cfg = example.Config()
    layer = example.Layer(cfg)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x, res, dout = (torch.randn(tokens, cfg.hidden, generator=g, device="cuda").bfloat16() for _ in range(3))
    out, kept = layer.forward(x, res)
    grads = layer.backward(dout, kept)
    p, slot, offsets = kept[-3:]
    assert offsets[-1] <= layer.rows(tokens) and slot.flatten().unique().numel() == slot.numel()
    want, wants = exact(layer, x, res, dout, (p, slot, offsets))
    for got, e in zip((out, *grads), (want, *wants)):
        assert got.shape == e.shape
        off = ((got.double() - e).norm() / e.norm()).item()
        assert off < 0.15, off
    idle = (offsets[1:] == offsets[:-1]).nonzero().flatten()
    assert (grads[2][idle] == 0).all() and (grads[3][idle] == 0).all()


def test_served_tokens_do_not_depend_on_their_batch(example, gpu):
    """One token, a few, many: the same codes go in, sums of other orders come out, so
    results agree within two roundings to bf16 (2^-7) and what the 8-bit instruction
    cuts (2^-13 of the largest of 8 products, far below)."""
    cfg = example.Config()
    layer = example.Layer(cfg)
    weight = gpu.blockfp8_quantize(layer.up.flatten(0, 1))
    g = torch.Generator(device="cuda").manual_seed(5)
    x, res = (torch.randn(400, cfg.hidden, generator=g, device="cuda").bfloat16() for _ in range(2))
    y, h = example.serve(x, res, layer.norm, weight)
    for n in (1, 20, 64, 200):
        part, hp = example.serve(x[:n], res[:n], layer.norm, weight)
        assert torch.equal(hp, h[:n])
        assert ((part.double() - y[:n].double()).abs() <= 2.0 ** -7 * y[:n].double().abs() + 0.004).all()


def test_runs_as_a_program(example):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "moe_8bit.py"), "--tokens", "70", "--steps", "1"],
                       capture_output=True, text=True, timeout=110)
    assert r.returncode == 0 and "one token served" in r.stdout, r.stderr
