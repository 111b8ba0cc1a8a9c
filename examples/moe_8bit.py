"""A mixture-of-experts layer on 8-bit products.

Training in MXFP8: the norm, with the residual added, leaves 8-bit tokens; every
expert's tokens, sorted and padded to multiples of 32, go through grouped products
up and down; the backward pass makes the experts' weight gradients, ragged along the
tokens, the tokens' gradients and the norm's.  Serving in block-FP8: the norm and a
product for one token or a batch.  Random weights.

    python examples/moe_8bit.py [--tokens 300] [--steps 3]
"""
from __future__ import annotations

import argparse
import os
import sys
import time
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_mxfp8_amd as mxq  # noqa: E402


@dataclass
class Config:
    hidden: int = 512
    inter: int = 256
    experts: int = 8
    chosen: int = 2


def quantize_experts(w: torch.Tensor):
    """Row-wise MXFP8 of bf16 [experts, n, k]."""
    q, s = mxq.mxfp8_quantize(w)
    return q.view(w.shape), s.view(*w.shape[:2], -1)


class Layer:
    """out = h + sum over a token's experts of p * down(silu(up(norm(h)))), h = x + residual."""

    def __init__(self, cfg: Config, seed: int = 0, device="cuda"):
        self.cfg = cfg
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5).bfloat16()

        self.norm = (1 + 0.1 * torch.randn(cfg.hidden, generator=g, device=device)).bfloat16()
        self.router = weight(cfg.experts, cfg.hidden)
        self.up, self.down = weight(cfg.experts, cfg.inter, cfg.hidden), weight(cfg.experts, cfg.hidden, cfg.inter)

    def route(self, y: torch.Tensor):
        """Each token's experts: their weights p, its rows among the experts' sorted and
        padded rows, and where each expert's rows begin."""
        cfg = self.cfg
        p, expert = torch.softmax(y.float() @ self.router.float().t(), -1).topk(cfg.chosen)
        flat = expert.flatten()
        count = torch.bincount(flat, minlength=cfg.experts)
        padded = (count + 31) // 32 * 32
        offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
        order = flat.sort(stable=True).indices
        rank = torch.empty_like(order)
        rank[order] = torch.arange(order.numel(), device=y.device)
        slot = offsets[flat] + rank - (count.cumsum(0) - count)[flat]
        return p / p.sum(-1, keepdim=True), slot.view(expert.shape), offsets.int()

    def rows(self, tokens: int) -> int:
        """Rows that hold any routing of so many tokens."""
        return (tokens * self.cfg.chosen + 31 * self.cfg.experts + 31) // 32 * 32

    def forward(self, x: torch.Tensor, residual: torch.Tensor):
        """(out, what the backward pass needs); x, residual bf16 [tokens, hidden]."""
        q, s, h, rstd, y = mxq.rmsnorm_mxfp8(x, self.norm, residual, return_rstd=True, return_normed=True)
        p, slot, offsets = self.route(y)
        rows = self.rows(x.shape[0])
        at = slot.flatten()
        token = torch.arange(x.shape[0], device=x.device).repeat_interleave(self.cfg.chosen)
        xq, xs, ys = q.new_zeros(rows, q.shape[1]), s.new_zeros(rows, s.shape[1]), y.new_zeros(rows, y.shape[1])
        xq[at], xs[at], ys[at] = q[token], s[token], y[token]
        u = mxq.mxfp8_matmul_grouped(xq, xs, *quantize_experts(self.up), offsets, out=y.new_zeros(rows, self.cfg.inter))
        a = torch.nn.functional.silu(u.float()).bfloat16()
        act = mxq.quantize_colwise_t(a, rowwise=True, fake_quant=False)
        d = mxq.mxfp8_matmul_grouped(act["q_row"], act["s_row"], *quantize_experts(self.down), offsets,
                                     out=y.new_zeros(rows, self.cfg.hidden))
        out = (h.float() + (p[..., None] * d[slot].float()).sum(1)).bfloat16()
        return out, (h, rstd, ys, u, act, p, slot, offsets)

    def backward(self, dout: torch.Tensor, kept):
        """Gradients of x (and of the residual alike), the norm's weight, up and down;
        the routing counts as given."""
        h, rstd, ys, u, act, p, slot, offsets = kept
        dd = dout.new_zeros(ys.shape)
        dd[slot.flatten()] = (p[..., None] * dout.float()[:, None]).bfloat16().flatten(0, 1)
        dd = mxq.quantize_colwise_t(dd, rowwise=True, fake_quant=False)
        ddown = mxq.mxfp8_matmul_wgrad(dd["q_colT"], dd["s_colT"], act["q_colT"], act["s_colT"], offsets, torch.float32)
        da = mxq.mxfp8_matmul_grouped(dd["q_row"], dd["s_row"], *quantize_experts(self.down.mT.contiguous()), offsets,
                                      out=u.new_zeros(u.shape))
        gate = torch.sigmoid(u.float())
        du = (da.float() * gate * (1 + u.float() * (1 - gate))).bfloat16()
        du = mxq.quantize_colwise_t(du, rowwise=True, fake_quant=False)
        yt = mxq.quantize_colwise_t(ys, rowwise=False, fake_quant=False)
        dup = mxq.mxfp8_matmul_wgrad(du["q_colT"], du["s_colT"], yt["q_colT"], yt["s_colT"], offsets, torch.float32)
        dy = mxq.mxfp8_matmul_grouped(du["q_row"], du["s_row"], *quantize_experts(self.up.mT.contiguous()), offsets,
                                      out=ys.new_zeros(ys.shape))
        dx, dnorm = mxq.rmsnorm_backward(dy[slot].float().sum(1).bfloat16(), h, self.norm, rstd, dh=dout)
        return dx, dnorm, dup, ddown


def serve(x: torch.Tensor, residual: torch.Tensor, norm: torch.Tensor, weight):
    """A serving step in block-FP8: (norm(x + residual) W^T, x + residual); weight as
    blockfp8_quantize returns it."""
    q, S, h = mxq.rmsnorm_blockfp8(x, norm, residual)
    return mxq.blockfp8_matmul(q, S, *weight), h


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=300)
    ap.add_argument("--steps", type=int, default=3)
    args = ap.parse_args()
    cfg = Config()
    layer = Layer(cfg)
    g = torch.Generator(device="cuda").manual_seed(1)
    for step in range(args.steps):
        x, res, dout = (torch.randn(args.tokens, cfg.hidden, generator=g, device="cuda").bfloat16() for _ in range(3))
        torch.cuda.synchronize()
        began = time.perf_counter()
        out, kept = layer.forward(x, res)
        dx, dnorm, dup, ddown = layer.backward(dout, kept)
        torch.cuda.synchronize()
        print(f"step {step}: {1e3 * (time.perf_counter() - began):.2f} ms, |out| {out.float().norm():.2f}, |dx| {dx.float().norm():.2f}, "
              f"|dup| {dup.norm():.2f}, |ddown| {ddown.norm():.2f}")
    y, _ = serve(x[:1], res[:1], layer.norm, mxq.blockfp8_quantize(layer.up.flatten(0, 1)))
    print(f"one token served: {tuple(y.shape)}")


if __name__ == "__main__":
    main()
