"""Operators of a layer in microscaled 4-bit floating point (MXFP4): the cases they are measured on.

Three operators:

* ``quantize``: rows become MXFP4 (blocks of 32 e2m1 codes with a power-of-two scale each), after a blockwise
  randomized Hadamard rotation or as they are, and are read back.
* ``product``: C = A W^T of two MXFP4 operands.
* ``norm``: what stands between two blocks of a layer: the block's output is normed, gated, scaled and added to
  the residual stream, and the new stream normed for the next block, whose operand it becomes in 16 or 32 bits
  or in MXFP4 (read back here).

MXFP4 rows are codes [rows][n / 2], two e2m1 codes a byte (the even element in the low nibble; a sign bit over
the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6), and scales [rows][n / 32], a byte b standing for 2^(b - 127).

Where ``own`` is false, everything here is elementary torch operations in 32 bits; where it is true, ``run``
calls the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-5


# ------------------------------------------------------------------ cases

def _quantize_case(name, rows, n, order, dtype, rule="floor"):
    return {"name": name, "op": "quantize", "rows": rows, "n": n, "order": order, "dtype": dtype, "rule": rule}


def _product_case(name, m, n, k, dtype):
    return {"name": name, "op": "product", "m": m, "n": n, "k": k, "dtype": dtype}


def _norm_case(name, rows, n, stream, dtype, block=True, post=True, gates=0, order=0):
    return {"name": name, "op": "norm", "rows": rows, "n": n, "stream": stream, "dtype": dtype, "block": block,
            "post": post, "gates": gates, "order": order}


def listed():
    return [
        # the activations of one new token, on their way into a product: latency alone
        _quantize_case("quantize one row", 1, 4096, 128, "bf16"),
        # an odd number of fp32 rows of a 5120-wide model, no rotation, the scale that never saturates
        _quantize_case("quantize 1237 fp32 plain", 1237, 5120, 0, "f32", "ceil"),
        # the activations of a large batch of a 2048-wide model: bound by memory
        _quantize_case("quantize 65536", 65536, 2048, 128, "bf16"),
        # one new token through a projection: bound by the weights' bytes and the launch
        _product_case("product one token", 1, 4096, 4096, "bf16"),
        # a small serving batch through the long side of an MLP
        _product_case("product 16 tokens", 16, 4096, 14336, "bf16"),
        # a ragged batch, odd in every direction, fp32 results
        _product_case("product 333 ragged fp32", 333, 5003, 2080, "f32"),
        # a prompt through a square projection: bound by the matrix products
        _product_case("product 4096 prompt", 4096, 4096, 4096, "bf16"),
        # a batch of prompts through the wide side of an MLP, the largest product
        _product_case("product 8192 wide", 8192, 14336, 4096, "bf16"),
        # the end of one block and the norm of the next for one new token: latency alone
        _norm_case("norm one token", 1, 4096, "bf16", "bf16"),
        # an odd number of rows of odd length, an fp32 residual stream, one gate for each of three sequences
        _norm_case("norm 1233 odd fp32 stream", 1233, 2047, "f32", "f16", gates=3),
        # a batch of prompts of a 4096-wide model with a gate for every channel: bound by memory
        _norm_case("norm 16384", 16384, 4096, "bf16", "bf16", gates=1),
        # the same into the next product's operand, rotated and in 4 bits
        _norm_case("norm 16384 to 4 bits", 16384, 4096, "bf16", "bf16", order=64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "norm"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "product":
        most = 8192 * 14336 * 4096
        k = 32 * _log_int(rng, 1, 512)
        m = _log_int(rng, 1, 8192)
        n = _log_int(rng, 1, max(1, min(14336, most // (m * k))))
        case = _product_case("", m, n, k, dtype)
    elif op == "quantize":
        # a code that falls on the other side of a border after a rotation, whose sums have no one order, would
        # show in fp32: those rows are quantized as they are
        order = 0 if dtype == "f32" else rng.choice((0, 32, 64, 128, 128, 256))
        unit = max(32, order)
        n = unit * _log_int(rng, 1, 16384 // unit)
        rows = _log_int(rng, 1, min(65536, 65536 * 2048 // (n * (2 if dtype == "f32" else 1))))
        case = _quantize_case("", rows, n, order, dtype, rng.choice(("floor", "floor", "ceil")))
    else:
        quantized = dtype != "f32" and rng.random() < 0.35
        order = rng.choice((32, 64, 128, 256)) if quantized else 0
        unit = max(1, order)
        n = unit * _log_int(rng, max(1, 64 // unit), 16384 // unit)
        if not quantized and rng.random() < 0.5:
            n = max(8, n // 8 * 8)
        stream = rng.choice((dtype, "f32"))
        rows = _log_int(rng, 1, min(65536, 16384 * 4096 // (n * (2 if "f32" in (dtype, stream) else 1))))
        block = rng.random() < 0.8
        gates = rng.choice((0, 1, rows) + tuple(g for g in (2, 3, 5, 8) if rows % g == 0)) if block else 0
        case = _norm_case("", rows, n, stream, dtype, block, block and rng.random() < 0.6, gates, order)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _signs(gen, n):
    return (torch.randint(0, 2, (n,), generator=gen, device=DEV) * 2 - 1).to(torch.int8)


def _activations(gen, rows, n, dtype):
    """Near Gaussian rows of varying size; a few channels are far larger than the rest."""
    x = torch.randn((rows, n), generator=gen, device=DEV)
    x *= torch.exp(0.3 * torch.randn((rows, 1), generator=gen, device=DEV))
    x *= 1.0 + 19.0 * (torch.rand((n,), generator=gen, device=DEV) < 0.01)
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    state = {"case": case}
    if case["op"] == "product":
        # activations after a rotation, and weights: both near Gaussian
        a = torch.randn((case["m"], case["k"]), generator=gen, device=DEV)
        a *= torch.exp(0.3 * torch.randn((case["m"], 1), generator=gen, device=DEV))
        state["a"] = _pack(*_quantized(a, "floor"))
        del a
        w = torch.randn((case["n"], case["k"]), generator=gen, device=DEV) / math.sqrt(case["k"])
        state["w"] = _pack(*_quantized(w, "ceil"))
        return state
    n, rows, dtype = case["n"], case["rows"], DTYPES[case["dtype"]]
    state["signs"] = _signs(gen, n) if case["order"] else None
    if case["op"] == "quantize":
        state["x"] = _activations(gen, rows, n, dtype)
        return state
    state["x"] = _activations(gen, rows, n, DTYPES[case["stream"]])
    state["block"] = _activations(gen, rows, n, dtype) if case["block"] else None
    state["weight"] = 1.0 + 0.2 * torch.randn((n,), generator=gen, device=DEV)
    state["post"] = 1.0 + 0.2 * torch.randn((n,), generator=gen, device=DEV) if case["post"] else None
    gate = torch.randn((case["gates"], n), generator=gen, device=DEV) if case["gates"] else None
    state["gate"] = gate.to(dtype) if gate is not None else None
    state["scale"] = 0.5 + torch.rand((), generator=gen, device=DEV).item()
    return state


# ------------------------------------------------------------------ plain forms

def _power(e):
    """2^e in fp32 for integers -127 <= e <= 127, by its bits."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, 0x00400000).view(torch.float32)


def _quantized(y, rule):
    """Signed e2m1 values (as fp32) [rows][n / 32][32] and exponents int32 [rows][n / 32] of fp32 rows y."""
    g = y.unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    bits = top.contiguous().view(torch.int32)
    e = (bits >> 23) - 127 - 2
    if rule == "ceil":       # 6 = 1.5 * 4: one more where the largest is over 1.5 powers of two
        e = e + ((bits & 0x7FFFFF) > 0x400000).to(torch.int32)
    e = e.clamp_(min=-127)
    v = g * _power(-e).unsqueeze(-1)
    a = v.abs().clamp_(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    q = (a / step).round_().mul_(step)
    return torch.copysign(q, v), e


def _pack(q, e):
    a = q.abs()
    code = torch.where(a < 2.0, a * 2.0, torch.where(a < 4.0, a + 2.0, a * 0.5 + 4.0)).to(torch.uint8)
    code = (code | (torch.signbit(q).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """fp32 rows that codes and scales stand for."""
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=DEV)
    q = level[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    return (q.unflatten(-1, (-1, 32)) * _power(scales.int() - 127).unsqueeze(-1)).flatten(-2)


def _hadamard(order):
    """H_order / sqrt(order), H[i][j] = (-1)^popcount(i & j)."""
    i = torch.arange(order, device=DEV)
    bits = i.unsqueeze(0) & i.unsqueeze(1)
    bits = bits ^ (bits >> 4)
    bits = bits ^ (bits >> 2)
    return (1 - 2 * ((bits ^ (bits >> 1)) & 1)).float() / math.sqrt(order)


def _through(y, order, signs, rule, dtype):
    """fp32 rows y: rotated, quantized, packed, read back and rotated back, as dtype."""
    if order:
        h = _hadamard(order)
        y = ((y * signs.float()).unflatten(-1, (-1, order)) @ h).flatten(-2)
    y = _values(*_pack(*_quantized(y, rule)))
    if order:
        y = (y.unflatten(-1, (-1, order)) @ h).flatten(-2) * signs.float()
    return y.to(dtype)


def _plain_norm(state):
    case, x = state["case"], state["x"]
    dtype = DTYPES[case["dtype"]]
    r = x.float()
    if state["block"] is not None:
        u = state["block"].float()
        if state["post"] is not None:
            u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS) * state["post"]
        if state["gate"] is not None:
            u = (u.unflatten(0, (case["gates"], -1)) * state["gate"].float().unsqueeze(1)).flatten(0, 1)
        r = r + state["scale"] * u
    h = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * state["weight"]
    h = _through(h, case["order"], state["signs"], "floor", dtype) if case["order"] else h.to(dtype)
    return r.to(x.dtype), h


def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "quantize":
            return _through(state["x"].float(), case["order"], state["signs"], case["rule"], state["x"].dtype)
        if case["op"] == "product":
            return (_values(*state["a"]) @ _values(*state["w"]).t()).to(DTYPES[case["dtype"]])
        return _plain_norm(state)
    import hadamard_rotation_int4_amd as hr

    order, dtype = case.get("order"), DTYPES[case["dtype"]]
    if case["op"] == "product":
        return hr.mxfp4_gemm(*state["a"], *state["w"], dtype=dtype)
    if case["op"] == "quantize":
        if order:
            codes, scales = hr.rotate_quant_mxfp4(state["x"], order, state["signs"], rule=case["rule"])
        else:
            codes, scales = hr.quant_mxfp4(state["x"], rule=case["rule"])
        return hr.dequant_mxfp4(codes, scales, order=order, signs=state["signs"], dtype=dtype)
    norm = {"weight": state["weight"], "post_norm": state["post"] is not None, "post_weight": state["post"],
            "gate": state["gate"], "scale": state["scale"], "eps": EPS}
    if order:
        r, codes, scales = hr.norm_residual_quant_mxfp4(state["x"], state["block"], order=order,
                                                        signs=state["signs"], **norm)
        return r, hr.dequant_mxfp4(codes, scales, order=order, signs=state["signs"], dtype=dtype)
    return hr.norm_residual(state["x"], state["block"], dtype=dtype, **norm)


# ------------------------------------------------------------------ work

def work(case):
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k * 17 // 32 + m * n * SIZE[case["dtype"]], "flops": 2 * m * n * k}
    values, size = case["rows"] * case["n"], SIZE[case["dtype"]]
    turn = int(math.log2(case["order"])) if case["order"] else 0
    if case["op"] == "quantize":
        # rows in, codes and scales out, codes and scales in, rows out
        return {"bytes": values * (2 * size + 17 / 16), "flops": values * (2 * turn + 4)}
    stream = SIZE[case["stream"]]
    moved = stream + (size + stream if case["block"] else 0)      # the stream and the block in, the new stream out
    moved += size + (17 / 16 if case["order"] else 0)             # the norm out; codes and scales out and in
    return {"bytes": values * moved + case["n"] * (4 + (4 if case["post"] else 0) + case["gates"] * size),
            "flops": values * (8 + 2 * turn)}


# ------------------------------------------------------------------ in 64 bits

def _sylvester(order):
    h = np.ones((1, 1))
    while h.shape[0] < order:
        h = np.block([[h, h], [h, -h]])
    return torch.from_numpy(h).to(DEV) / math.sqrt(order)


def _decoded(codes, scales):
    """Rows in 64 bits, element by element from the format."""
    b = codes.long()
    c = torch.empty((b.shape[0], 2 * b.shape[1]), dtype=torch.long, device=DEV)
    c[:, 0::2], c[:, 1::2] = b % 16, b // 16
    high, low = c % 8 // 2, (c % 2).double()
    # exponent 0: the mantissa counts halves; else (1 + mantissa / 2) 2^(exponent - 1)
    size = torch.where(high == 0, 0.5 * low, (1.0 + 0.5 * low) * torch.pow(2.0, high.double() - 1.0))
    size *= torch.pow(2.0, scales.double() - 127.0).repeat_interleave(32, 1)
    return torch.where(c >= 8, -size, size)


def _nearest(y, rule):
    """The MXFP4 values nearest to rows y in 64 bits; a value half way goes to the even code."""
    g = y.reshape(-1, 32)
    top = g.abs().max(1, keepdim=True).values
    mantissa, e = torch.frexp(top)                       # top = mantissa 2^e, mantissa in [1/2, 1)
    e = e - 3
    if rule == "ceil":
        e = torch.where(mantissa > 0.75, e + 1, e)
    unit = torch.pow(2.0, e.double().clamp(min=-127.0))
    a = (g.abs() / unit).clamp(max=6.0)
    level = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)
    border = (level[1:] + level[:-1]) / 2
    # the borders after even codes go down, those after odd ones up
    down, up = border[0::2].contiguous(), border[1::2].contiguous()
    i = torch.bucketize(a, down) + torch.bucketize(a, up, right=True)
    return (torch.where(g < 0, -level[i], level[i]) * unit).reshape(y.shape)


def _exact_through(y, order, signs, rule):
    if not order:
        return _nearest(y, rule)
    turn = _sylvester(order)
    z = (y * signs.double()).reshape(-1, order) @ turn
    return (_nearest(z, rule) @ turn).reshape(y.shape) * signs.double()


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "product":
        return _decoded(*state["a"]) @ _decoded(*state["w"]).t()
    x = state["x"].double()
    if case["op"] == "quantize":
        return _exact_through(x, case["order"], state["signs"], case["rule"])
    if state["block"] is not None:
        o = state["block"].double()
        if state["post"] is not None:
            o = o / torch.sqrt((o * o).sum(1, keepdim=True) / o.shape[1] + EPS) * state["post"].double()
        if state["gate"] is not None:
            o = o * state["gate"].double().repeat_interleave(case["rows"] // case["gates"], 0)
        x = x + state["scale"] * o
    h = x / torch.sqrt((x * x).sum(1, keepdim=True) / x.shape[1] + EPS) * state["weight"].double()
    return x, _exact_through(h, case["order"], state["signs"], "floor") if case["order"] else h
