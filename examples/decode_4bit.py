"""Decoding with 4-bit weights and a 4-bit key/value cache.

A small decoder (random weights) as a serving program would run it on this
library: projections in MXFP4, the output head in NVFP4, keys and values in a
paged MXFP4 cache.  It fills the cache with a prompt in chunks, forks the
sequence (whole pages shared, the last one copied when it is written), decodes
both forks greedily in one batch, frees one, and compacts the cache.

    python examples/decode_4bit.py [--prompt 200] [--tokens 32]
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
    layers: int = 2
    hidden: int = 1024
    inter: int = 2048
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 128
    vocab: int = 2048
    page_size: int = 32
    pages: int = 64


def norm(x: torch.Tensor) -> torch.Tensor:
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Decoder:
    def __init__(self, cfg: Config, seed: int = 0, device="cuda"):
        self.cfg, self.device = cfg, device
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device=device) * k ** -0.5).bfloat16()

        qkv = (cfg.q_heads + 2 * cfg.kv_heads) * cfg.head_dim
        self.embed = torch.randn(cfg.vocab, cfg.hidden, generator=g, device=device).bfloat16()
        self.weights = [{name: mxq.mxfp4_quantize(weight(n, k)) for name, n, k in (
            ("qkv", qkv, cfg.hidden), ("o", cfg.hidden, cfg.q_heads * cfg.head_dim),
            ("gate_up", 2 * cfg.inter, cfg.hidden), ("down", cfg.hidden, cfg.inter))} for _ in range(cfg.layers)]
        self.head = mxq.nvfp4_quantize(weight(cfg.vocab, cfg.hidden))
        self.cache = mxq.mxfp4_kv_cache(cfg.layers, cfg.pages, cfg.kv_heads, cfg.head_dim, cfg.page_size, device)
        self.pool = mxq.KVPagePool(cfg.pages, cfg.page_size)

    def room(self, seqs, tokens: int):
        """Places for `tokens` more tokens of each sequence, shared pages copied first."""
        slots, src, dst = [], [], []
        for s in seqs:
            a, b, c = self.pool.extend(s, tokens)
            slots, src, dst = slots + a, src + b, dst + c
        if src:
            pairs = torch.tensor([src, dst], dtype=torch.int32, device=self.device)
            mxq.mxfp4_kv_copy_pages(self.cache, pairs[0], pairs[1])
        return torch.tensor(slots, dtype=torch.int64, device=self.device)

    def compact(self):
        src, dst = self.pool.compact()
        if src:
            pairs = torch.tensor([src, dst], dtype=torch.int32, device=self.device)
            mxq.mxfp4_kv_copy_pages(self.cache, pairs[0], pairs[1])
        return len(src)

    def forward(self, seqs, ids: torch.Tensor) -> torch.Tensor:
        """fp32 logits [seqs, tokens, vocab] of the next tokens `ids` [seqs, tokens]."""
        cfg = self.cfg
        n, t = ids.shape
        slots = self.room(seqs, t)
        table, lengths = self.pool.table(seqs, device=self.device)
        x = self.embed[ids]
        for layer, w in enumerate(self.weights):
            qkv = mxq.mxfp4_matvec(norm(x), *w["qkv"]).view(n * t, -1, cfg.head_dim)
            q, k, v = qkv.split((cfg.q_heads, cfg.kv_heads, cfg.kv_heads), 1)
            mxq.mxfp4_kv_append(self.cache[layer], k, v, slots, cfg.page_size)
            o = mxq.mxfp4_kv_attention(q.unflatten(0, (n, t)), self.cache[layer], table, lengths, cfg.kv_heads, cfg.page_size)
            x = x + mxq.mxfp4_matvec(o.flatten(2), *w["o"])
            gate, up = mxq.mxfp4_matvec(norm(x), *w["gate_up"]).chunk(2, -1)
            x = x + mxq.mxfp4_matvec(torch.nn.functional.silu(gate) * up, *w["down"])
        return mxq.nvfp4_matvec(norm(x), *self.head, out_dtype=torch.float32)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompt", type=int, default=200)
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--chunk", type=int, default=64)
    a = ap.parse_args(argv)
    model = Decoder(Config())
    prompt = torch.randint(0, model.cfg.vocab, (1, a.prompt), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    for at in range(0, a.prompt, a.chunk):
        logits = model.forward(["a"], prompt[:, at:at + a.chunk])
    model.pool.fork("a", "b")
    best = logits[0, -1].topk(2).indices  # the forks begin with different tokens
    ids, out = best[:, None], [best[:, None]]
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(a.tokens):
        ids = model.forward(["a", "b"], ids)[:, -1].argmax(-1, keepdim=True)
        out.append(ids)
    torch.cuda.synchronize()
    ms = 1e3 * (time.perf_counter() - began) / a.tokens
    used = sum(r > 0 for r in model.pool.refs)
    model.pool.free("a")
    moved = model.compact()
    print(f"{a.prompt} prompt tokens, {a.tokens} steps of 2 forks: {ms:.2f} ms a step; {used} pages in use, "
          f"{sum(r > 0 for r in model.pool.refs)} after freeing one fork ({moved} moved)")
    return torch.cat(out, 1)


if __name__ == "__main__":
    main()
