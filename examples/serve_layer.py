"""One Transformer layer served from a paged key-value cache, with every step in the library's
kernels: LayerNorm and the column-parallel Q/K/V projection, the rotation and the cache's append,
attention of a prompt or of single tokens, the row-parallel output projection, and the MLP block
with its LayerNorm and residual (AI大模型分布式训练 §2.3 and §3.4).

    python examples/serve_layer.py [--kv e4m3]

A ragged batch of prompts goes through the layer, then a few tokens are generated with the decode
step captured in a CUDA graph; the last lines compare the generated rows with one pass over the
whole sequences (exit code 1 if they differ by more than rounding).
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import tensor_transformer_mlp_tmem_gb300 as tp


class Layer:
    """x + attention(LayerNorm(x)), then x + MLP(LayerNorm(x)), for B sequences of at most
    max_len tokens. H = Hq * D hidden columns, k shards."""

    def __init__(self, Hq, Hkv, D, k, B, max_len, kv="bf16", page=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        H, self.F = Hq * D, 4 * Hq * D
        self.Hq, self.Hkv, self.D, self.B = Hq, Hkv, D, B

        def normal(*shape, std=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()

        self.qkv = tp.Linear("column", H, (Hq + 2 * Hkv) * D, k)
        self.qkv.pack(normal(H, (Hq + 2 * Hkv) * D, std=H ** -0.5),
                      normal((Hq + 2 * Hkv) * D, std=0.02))
        tp.tpmlp_set_layernorm(self.qkv.ctx, torch.ones(H, device="cuda").bfloat16(),
                               torch.zeros(H, device="cuda").bfloat16(), 1e-5)
        self.proj = tp.Linear("row", H, H, k)
        self.proj.pack(normal(H, H, std=H ** -0.5), normal(H, std=0.02))
        self.mlp = tp.TPMLP(H, self.F, k)
        self.mlp.pack(normal(H, self.F, std=H ** -0.5), normal(self.F, std=0.02),
                      normal(self.F, H, std=self.F ** -0.5), normal(H, std=0.02))
        self.mlp.set_layernorm(torch.ones(H, device="cuda").bfloat16(),
                               torch.zeros(H, device="cuda").bfloat16())
        self.attn = tp.Attention(Hq, Hkv, D, page, kv_dtype=kv)
        self.attn.set_rope(D)
        if kv == "e4m3":  # keys and values of about unit size, in the upper half of e4m3's range
            scale = torch.full((Hkv,), 1.0 / 32, device="cuda")
            self.attn.set_scales(scale, scale)
        width = -(-max_len // page)
        table = torch.randperm(B * width, generator=g, device="cuda").int().view(B, width)
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.cache = self.attn.new_cache(B * width, table, self.lens)

    def _run(self, x, attend, pos, seq):
        n = torch.empty_like(x)
        tp.tpmlp_layernorm(self.qkv.ctx, x, x.shape[0], n)
        q, k, v = self.qkv(n).split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], 1)
        q = self.attn.append(q, k, v, self.cache, pos, seq)
        x = x + self.proj(attend(q))
        return self.mlp.block(x.unsqueeze(0)).squeeze(0)

    def prompt(self, x, cu, pos, seq):
        """x [T, H]: new tokens, sequence b's in rows cu[b] .. cu[b + 1] - 1. The lengths are
        counted up by the new tokens first."""
        self.lens += cu[1:] - cu[:-1]
        return self._run(x, lambda q: self.attn.prompt(q, cu, self.cache), pos, seq)

    def decode(self, x):
        """x [B, H]: one new token of each sequence."""
        pos = self.lens.clone()
        self.lens += 1
        return self._run(x, lambda q: self.attn.decode(q, self.cache), pos, None)


def rows(lens, starts):
    """cu, pos, seq of `lens[b]` new tokens of each sequence b from position starts[b]."""
    cu = [sum(lens[:b]) for b in range(len(lens) + 1)]
    pos = [s + i for n, s in zip(lens, starts) for i in range(n)]
    seq = [b for b, n in enumerate(lens) for _ in range(n)]
    return [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (cu, pos, seq)]


def generate(kv="bf16", Hq=8, Hkv=2, D=128, k=4, prompts=(37, 200, 1, 129), steps=6, seed=0):
    """The generated rows [steps, B, H], and the same rows of one pass over whole sequences."""
    B, most = len(prompts), max(prompts) + steps
    layer = Layer(Hq, Hkv, D, k, B, most, kv)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn((sum(prompts), Hq * D), generator=g, device="cuda").bfloat16()
    tokens = torch.randn((steps, B, Hq * D), generator=g, device="cuda").bfloat16()

    layer.prompt(x, *rows(prompts, [0] * B))
    got = [layer.decode(tokens[0])]  # eager once: the MLP's buffers take their size
    step, graph = tokens[0].clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.decode(step)
    for i in range(1, steps):
        step.copy_(tokens[i])
        graph.replay()
        got.append(out.clone())

    whole = [n + steps for n in prompts]
    cut = torch.split(x, list(prompts))
    full = torch.cat([torch.cat([cut[b], tokens[:, b]]) for b in range(B)])
    layer.lens.zero_()
    cu, pos, seq = rows(whole, [0] * B)
    want = layer.prompt(full, cu, pos, seq)
    at = torch.stack([cu[1:].long() - steps + i for i in range(steps)])
    for ctx in (layer.qkv, layer.proj, layer.mlp, layer.attn):
        rc, detail = ctx.status()
        assert rc == tp.TPMLP_OK, f"device status {rc} ({detail:#x})"
    return torch.stack(got), want[at]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--kv", choices=["bf16", "e4m3"], default="bf16")
    got, want = generate(ap.parse_args().kv)
    off = float((got.float() - want.float()).norm() / want.float().norm())
    print(f"generated {tuple(got.shape)}: relative difference from one pass {off:.2e}")
    return int(not off < 1e-2)


if __name__ == "__main__":
    sys.exit(main())
