"""One attention layer of a rotated 4-bit model: prompt, then single tokens.

Every product is the library's: the hidden states are rotated and quantized as
they enter the W4A4 GEMMs (hr_rotate_quant_int4, hr_rotate_quant_w4a4_gemm),
keys and values are rotated per head and quantized as they enter the cache
(hr_kv4_append), and the attention runs over the cache in its 4-bit form
(hr_kv4_attention).  Random weights and inputs; the same layer in fp32, with
nothing quantized, is run beside it to say what the 4 bits cost.

Usage: python examples/kv4_decode.py [--batch B] [--prompt N] [--steps S]
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

WIDTH, Q_HEADS, HEADS, DIM, PAGE, GROUP = 4096, 32, 8, 128, 64, 128
QKV = (Q_HEADS + 2 * HEADS) * DIM


class Layer:
    """Projections in int4 on rotated inputs, and a paged 4-bit cache."""

    def __init__(self, batch: int, length: int, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def signs(n):
            return (torch.randint(0, 2, (n,), generator=gen, device="cuda") * 2 - 1).to(torch.int8)

        def weight(n, k):
            return (torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k)).to(torch.bfloat16)

        self.batch = batch
        self.w_qkv, self.w_out = weight(QKV, WIDTH), weight(WIDTH, Q_HEADS * DIM)
        # both operands of a product are rotated the same way, so the product does not change
        self.s_in, self.s_out = signs(WIDTH), signs(Q_HEADS * DIM)
        self.qkv4 = hr.rotate_quant_int4(self.w_qkv, GROUP, self.s_in)
        self.out4 = hr.rotate_quant_int4(self.w_out, GROUP, self.s_out)
        per = -(-length // PAGE)
        self.cache = hr.kv4_cache(batch * per, HEADS, DIM, PAGE, signs=signs(DIM))
        self.table = torch.randperm(batch * per, generator=gen, device="cuda").to(torch.int32).view(batch, per)
        self.lens = torch.zeros((batch,), dtype=torch.int32, device="cuda")
        self.length = length

    def _project(self, x, w4, s, n):
        """x bf16 [rows][K] times the int4 weights; one kernel for few rows."""
        if x.shape[0] <= 16:
            return hr.rotate_quant_w4a4_gemm(x, *w4, GROUP, s).to(torch.bfloat16)
        return hr.w4a4_gemm(*hr.rotate_quant_int4(x, GROUP, s), *w4, GROUP).to(torch.bfloat16)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """x bf16 [batch][new][WIDTH]: the next `new` tokens of every sequence."""
        batch, new, _ = x.shape
        qkv = self._project(x.reshape(batch * new, WIDTH).contiguous(), self.qkv4, self.s_in, QKV)
        q = qkv[:, :Q_HEADS * DIM].view(batch * new, Q_HEADS, DIM)
        k = qkv[:, Q_HEADS * DIM:(Q_HEADS + HEADS) * DIM].view(batch * new, HEADS, DIM)
        v = qkv[:, (Q_HEADS + HEADS) * DIM:].view(batch * new, HEADS, DIM)
        pos = self.lens.long().unsqueeze(1) + torch.arange(new, device="cuda")
        slots = self.table.long().gather(1, pos // PAGE) * PAGE + pos % PAGE
        hr.kv4_append(self.cache, k, v, slots.view(-1))
        self.lens += new
        o = hr.kv4_attention(self.cache, q, self.table, self.lens, max_new=new, max_len=self.length)
        return self._project(o.view(batch * new, Q_HEADS * DIM), self.out4, self.s_out, WIDTH).view(batch, new, WIDTH)


def reference(layer: Layer, xs: torch.Tensor) -> torch.Tensor:
    """The whole sequence through the same layer in fp32, nothing quantized."""
    batch, n, _ = xs.shape
    qkv = xs.float() @ layer.w_qkv.float().t()
    q, k, v = qkv.split((Q_HEADS * DIM, HEADS * DIM, HEADS * DIM), -1)
    q = q.view(batch, n, HEADS, Q_HEADS // HEADS, DIM).permute(0, 2, 3, 1, 4)
    k = k.view(batch, n, HEADS, DIM).permute(0, 2, 1, 3).unsqueeze(2)
    v = v.view(batch, n, HEADS, DIM).permute(0, 2, 1, 3).unsqueeze(2)
    z = q @ k.transpose(-1, -2).contiguous() / math.sqrt(DIM)
    hidden = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
    o = z.masked_fill(hidden, -math.inf).softmax(-1) @ v
    return o.permute(0, 3, 1, 2, 4).reshape(batch, n, Q_HEADS * DIM) @ layer.w_out.float().t()


def run(batch: int = 4, prompt: int = 300, steps: int = 20, seed: int = 0):
    """Returns (relative error against fp32 of the prompt, of the single tokens,
    seconds a step, bytes of cache a token)."""
    layer = Layer(batch, prompt + steps, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    xs = torch.randn((batch, prompt + steps, WIDTH), generator=gen, device="cuda")
    xs[..., torch.randint(0, WIDTH, (4,), generator=gen, device="cuda")] *= 20.0      # outlier channels
    xs = xs.to(torch.bfloat16)
    got = [layer.forward(xs[:, :prompt])]
    torch.cuda.synchronize()
    t = time.perf_counter()
    for i in range(prompt, prompt + steps):
        got.append(layer.forward(xs[:, i:i + 1]))
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / max(1, steps)
    want = reference(layer, xs)
    got = torch.cat(got, 1).float()

    def off(a, b):
        return (torch.linalg.norm(a - b) / torch.linalg.norm(b)).item() if b.numel() else 0.0

    held = 2 * HEADS * (DIM // 2 + 2 * (DIM // layer.cache.group))
    return off(got[:, :prompt], want[:, :prompt]), off(got[:, prompt:], want[:, prompt:]), t, held


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    e0, e1, t, held = run(a.batch, a.prompt, a.steps)
    print(f"prompt of {a.prompt} tokens x {a.batch}: {100 * e0:.1f}% from fp32; {a.steps} single tokens: {100 * e1:.1f}%, "
          f"{1e6 * t:.0f} us a step; {held} bytes of cache a token ({4 * HEADS * DIM} in bf16)")


if __name__ == "__main__":
    main()
