"""Decoder blocks of a rotated MXFP4 model: prompt, then single tokens.

Between the products of a block stand the library's norms: the end of one half
(output norm, residual) and the norm before the next are one call that leaves the
next product's operand in MXFP4 (hr_norm_residual_quant_mxfp4), rotated as its
weights are (hr_rotate_quant_mxfp4); the products are hr_mxfp4_gemm, keys and values
go to the 4-bit cache and the attention runs over it (hr_kv4_append,
hr_kv4_attention).  Random weights and inputs; the same blocks in fp32, with nothing
quantized, are run beside them to say what the 4 bits cost.

Usage: python examples/mxfp4_block.py [--layers L] [--batch B] [--prompt N] [--steps S]
"""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import hadamard_rotation_int4_amd as hr  # noqa: E402

WIDTH, Q_HEADS, HEADS, DIM, PAGE, HIDDEN, ORDER = 2048, 32, 8, 64, 64, 4096, 128
QKV = (Q_HEADS + 2 * HEADS) * DIM
EPS = 1e-5
DEPTH = 0.5      # scale of what a half adds to the residual stream


class Linear:
    """Weights in MXFP4, rotated along their inputs."""

    def __init__(self, gen, n: int, k: int):
        self.w = (torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k)).to(torch.bfloat16)
        self.signs = (torch.randint(0, 2, (k,), generator=gen, device="cuda") * 2 - 1).to(torch.int8)
        self.q = hr.rotate_quant_mxfp4(self.w, ORDER, self.signs, rule="ceil")

    def __call__(self, codes, scales):
        return hr.mxfp4_gemm(codes, scales, *self.q, dtype=torch.bfloat16)

    def of(self, x):
        """The same of rows that are not quantized yet."""
        return self(*hr.rotate_quant_mxfp4(x, ORDER, self.signs))


class Block:
    def __init__(self, gen, batch: int, length: int):
        def gain():
            return 1.0 + 0.1 * torch.randn((WIDTH,), generator=gen, device="cuda")

        self.norm_in, self.norm_attn, self.norm_mid, self.norm_mlp = (gain() for _ in range(4))
        self.qkv, self.out = Linear(gen, QKV, WIDTH), Linear(gen, WIDTH, Q_HEADS * DIM)
        self.up, self.down = Linear(gen, 2 * HIDDEN, WIDTH), Linear(gen, WIDTH, HIDDEN)
        per = -(-length // PAGE)
        signs = (torch.randint(0, 2, (DIM,), generator=gen, device="cuda") * 2 - 1).to(torch.int8)
        self.cache = hr.kv4_cache(batch * per, HEADS, DIM, PAGE, signs=signs)


class Model:
    def __init__(self, layers: int, batch: int, length: int, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.blocks = [Block(gen, batch, length) for _ in range(layers)]
        self.norm_out = 1.0 + 0.1 * torch.randn((WIDTH,), generator=gen, device="cuda")
        per = -(-length // PAGE)
        self.table = torch.randperm(batch * per, generator=gen, device="cuda").to(torch.int32).view(batch, per)
        self.lens = torch.zeros((batch,), dtype=torch.int32, device="cuda")
        self.length = length

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """x fp32 [batch][new][WIDTH]: the next `new` tokens of every sequence; the
        normed stream behind the last block, bf16."""
        batch, new, _ = x.shape
        rows = batch * new
        pos = self.lens.long().unsqueeze(1) + torch.arange(new, device="cuda")
        slots = (self.table.long().gather(1, pos // PAGE) * PAGE + pos % PAGE).view(-1)
        self.lens += new
        stream, added, added_norm = x.reshape(rows, WIDTH).contiguous(), None, None
        for b in self.blocks:
            # the end of the block before (none before the first) and this one's norm
            end = {} if added is None else {"post_norm": True, "post_weight": added_norm, "scale": DEPTH}
            stream, codes, scales = hr.norm_residual_quant_mxfp4(stream, added, b.norm_in, eps=EPS, order=ORDER,
                                                                 signs=b.qkv.signs, **end)
            qkv = b.qkv(codes, scales)
            q = qkv[:, :Q_HEADS * DIM].view(rows, Q_HEADS, DIM)
            k = qkv[:, Q_HEADS * DIM:(Q_HEADS + HEADS) * DIM].view(rows, HEADS, DIM)
            v = qkv[:, (Q_HEADS + HEADS) * DIM:].view(rows, HEADS, DIM)
            hr.kv4_append(b.cache, k, v, slots)
            o = hr.kv4_attention(b.cache, q, self.table, self.lens, max_new=new, max_len=self.length)
            stream, codes, scales = hr.norm_residual_quant_mxfp4(stream, b.out.of(o.view(rows, -1)), b.norm_mid, post_norm=True,
                                                                 post_weight=b.norm_attn, scale=DEPTH, eps=EPS,
                                                                 order=ORDER, signs=b.up.signs, residual=stream if added is not None else None)
            gate, up = b.up(codes, scales).chunk(2, 1)
            added, added_norm = b.down.of(torch.nn.functional.silu(gate) * up), b.norm_mlp
        _, h = hr.norm_residual(stream, added, self.norm_out, post_norm=True, post_weight=added_norm, scale=DEPTH, eps=EPS)
        return h.view(batch, new, WIDTH)


def reference(model: Model, x: torch.Tensor) -> torch.Tensor:
    """The whole sequence through the same blocks in fp32, nothing quantized."""
    def rms(v, w):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w

    batch, n, _ = x.shape
    hidden = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
    for b in model.blocks:
        q, k, v = (rms(x, b.norm_in) @ b.qkv.w.float().t()).split((Q_HEADS * DIM, HEADS * DIM, HEADS * DIM), -1)
        q = q.view(batch, n, HEADS, Q_HEADS // HEADS, DIM).permute(0, 2, 3, 1, 4)
        k = k.view(batch, n, HEADS, DIM).permute(0, 2, 1, 3).unsqueeze(2)
        v = v.view(batch, n, HEADS, DIM).permute(0, 2, 1, 3).unsqueeze(2)
        z = q @ k.transpose(-1, -2).contiguous() / math.sqrt(DIM)
        o = (z.masked_fill(hidden, -math.inf).softmax(-1) @ v).permute(0, 3, 1, 2, 4).reshape(batch, n, Q_HEADS * DIM)
        x = x + DEPTH * rms(o @ b.out.w.float().t(), b.norm_attn)
        gate, up = (rms(x, b.norm_mid) @ b.up.w.float().t()).chunk(2, -1)
        x = x + DEPTH * rms((torch.nn.functional.silu(gate) * up) @ b.down.w.float().t(), b.norm_mlp)
    return rms(x, model.norm_out)


def run(layers: int = 2, batch: int = 4, prompt: int = 100, steps: int = 10, seed: int = 0):
    """Returns (relative error against fp32 of the prompt, of the single tokens,
    seconds a step)."""
    model = Model(layers, batch, prompt + steps, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    xs = torch.randn((batch, prompt + steps, WIDTH), generator=gen, device="cuda")
    xs[..., torch.randint(0, WIDTH, (4,), generator=gen, device="cuda")] *= 20.0      # outlier channels
    want = reference(model, xs)
    got = [model.forward(xs[:, :prompt])]
    torch.cuda.synchronize()
    t = time.perf_counter()
    for i in range(prompt, prompt + steps):
        got.append(model.forward(xs[:, i:i + 1]))
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / max(1, steps)
    got = torch.cat(got, 1).float()

    def off(a, b):
        return (torch.linalg.norm(a - b) / torch.linalg.norm(b)).item() if b.numel() else 0.0

    return off(got[:, :prompt], want[:, :prompt]), off(got[:, prompt:], want[:, prompt:]), t


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    e0, e1, t = run(a.layers, a.batch, a.prompt, a.steps)
    print(f"{a.layers} blocks, prompt of {a.prompt} tokens x {a.batch}: {100 * e0:.1f}% from fp32; {a.steps} single tokens: "
          f"{100 * e1:.1f}%, {1e6 * t:.0f} us a step")


if __name__ == "__main__":
    main()
