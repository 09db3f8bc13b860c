"""The norms between two blocks on the GPU against the fp64 oracle.

r is a few fp32 operations on terms of size T = |x| + |scale gate u|; the norms'
factors come from sums of n squares, each lane's at most 32 of them in a row and
then a tree of 10 steps: their relative error stays under 48 2^-24, half of it
after the root.  Together r is within 32 2^-24 T, and h within 32 2^-24 |h| and
what r's error makes of it, 32 2^-24 |weight| T / rms(r).  Allowed: 2^-19 of
T and of |weight| T / rms(r) (which is at least |h|), and half a step of the
output's type.
"""
import numpy as np
import pytest
import torch

import hadamard_rotation_int4_amd as hr
from oracle import mxfp4, norm
from test_gpu_mxfp4 import DEV, TYPES, _half_step, _num, _rng, _rows, _signs, _t, check_near, rotation_error

pytestmark = pytest.mark.gpu

EPS = 1e-5
PAIRS = [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16"), ("f32", "f16")]


def _case(rng, rows, n, stream, dtype, block=True, post=True, weights=True, gates=0, pad=0):
    """Inputs of a call; rows are slices of wider ones where pad is set."""
    x = _rows(rng, rows, n + pad, TYPES[stream])[:, pad:]
    a = {"x": x, "block_out": None, "weight": None, "post_norm": False, "post_weight": None, "gate": None,
         "scale": 0.7, "eps": EPS}
    if weights:
        a["weight"] = _t((1 + 0.2 * rng.standard_normal(n)).astype(np.float32))
    if block:
        a["block_out"] = _rows(rng, rows, n + pad, TYPES[dtype])[:, pad:]
        if post:
            a["post_norm"] = True
            if weights:
                a["post_weight"] = _t((1 + 0.2 * rng.standard_normal(n)).astype(np.float32))
        if gates:
            a["gate"] = _t(rng.standard_normal((gates, n)).astype(np.float32)).to(TYPES[dtype])
    return a


def _oracle(a):
    b = {k: _num(v) if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    return norm.norm_residual(b["x"], b["block_out"], b["weight"], b["post_norm"], b["post_weight"], b["gate"],
                              b["scale"], b["eps"])


def _bounds(a, r, size):
    """What r and h may be off before they are rounded."""
    wt = 1.0 if a["weight"] is None else np.abs(_num(a["weight"]))
    rms = np.sqrt((r * r).mean(-1, keepdims=True) + a["eps"])
    return 2.0 ** -19 * size, 2.0 ** -19 * wt * size.max(-1, keepdims=True) / rms


def check(a, got, dtype):
    r, h, size = _oracle(a)
    dr, dh = _bounds(a, r, size)
    res, out = got
    assert res.dtype == a["x"].dtype and out.dtype == dtype
    assert (np.abs(_num(res) - r) <= dr + np.abs(r) * _half_step(res.dtype)).all()
    tiny = torch.finfo(dtype).tiny * _half_step(dtype)
    assert (np.abs(_num(out) - h) <= dh + np.abs(h) * _half_step(dtype) + tiny).all()


SIZES = [(1, 1), (9, 33), (33, 64), (70, 65), (17, 128), (18, 129), (9, 256), (5, 257), (3, 7), (2, 8), (5, 63), (4, 64), (7, 500), (3, 512), (3, 520), (2, 1000), (3, 2047), (2, 2048),
         (3, 2049), (2, 4096), (3, 5000), (2, 8192), (2, 8200), (3, 14336), (2, 16384), (2, 16385), (1, 32768)]


@pytest.mark.parametrize("rows,n", SIZES)
@pytest.mark.parametrize("stream,dtype", PAIRS)
def test_norm_residual(rows, n, stream, dtype):
    a = _case(_rng(rows * n), rows, n, stream, dtype, gates=1)
    check(a, hr.norm_residual(**a), TYPES[dtype])


@pytest.mark.parametrize("stream,dtype", PAIRS)
@pytest.mark.parametrize("block,post,weights,gates", [(False, False, True, 0), (False, False, False, 0),
                                                      (True, False, True, 0), (True, True, False, 0),
                                                      (True, False, False, 3), (True, True, True, 12)])
@pytest.mark.parametrize("n", [65, 1024, 4100])
def test_parts(n, block, post, weights, gates, stream, dtype):
    a = _case(_rng(n), 12, n, stream, dtype, block, post, weights, gates)
    r, h = hr.norm_residual(**a, dtype=TYPES[dtype])
    check(a, (r, h), TYPES[dtype])
    if not block:
        assert r is a["x"]


@pytest.mark.parametrize("rows,n", [(rows, n) for rows in (1, 2, 255, 300, 5000, 33333)
                                    for n in (24, 64, 100, 200, 384, 2048, 4096) if rows * n < 1.3e7])
def test_many_rows(rows, n):
    gates = rows // 5 if rows % 5 == 0 else rows
    a = _case(_rng(rows), rows, n, "bf16", "bf16", gates=gates)
    check(a, hr.norm_residual(**a), torch.bfloat16)


@pytest.mark.parametrize("stream,dtype", PAIRS)
@pytest.mark.parametrize("n,pad", [(64, 8), (96, 1), (1000, 3), (2048, 16), (4096, 5), (333, 0)])
def test_strided_and_unaligned_rows(n, pad, stream, dtype):
    a = _case(_rng(n + pad), 9, n, stream, dtype, gates=3, pad=pad)
    wide = torch.full((9, n + 2 * pad + 2), 5.0, dtype=TYPES[stream], device=DEV)
    res = wide[:, pad + 1:pad + 1 + n]
    r, h = hr.norm_residual(**a, residual=res)
    assert r is res
    check(a, (r, h), TYPES[dtype])
    assert (wide[:, :pad + 1] == 5.0).all() and (wide[:, pad + 1 + n:] == 5.0).all()


@pytest.mark.parametrize("stream,dtype", PAIRS)
@pytest.mark.parametrize("n", [100, 2048, 5000])
def test_in_place_and_without_h(n, stream, dtype):
    a = _case(_rng(n), 6, n, stream, dtype, gates=2)
    r, h = hr.norm_residual(**a)
    b = dict(a, x=a["x"].clone())
    r2, none = hr.norm_residual(**b, want_h=False)
    assert none is None and torch.equal(r, r2)
    r3, h3 = hr.norm_residual(**b, residual=b["x"])
    assert r3 is b["x"] and torch.equal(r3, r) and torch.equal(h3, h)


@pytest.mark.parametrize("stream,dtype", PAIRS)
def test_zero_rows_and_values_that_are_not_finite(stream, dtype):
    a = _case(_rng(2), 6, 600, stream, dtype)
    a["x"][0] = 0
    a["block_out"][0] = 0
    clean = [v.clone() for v in hr.norm_residual(**a)]
    assert not clean[0][0].any() and not clean[1][0].any()
    a["x"][1, 599] = float("nan")
    a["x"][2, 0] = float("inf")
    a["block_out"][3, 5] = float("inf")
    r, h = hr.norm_residual(**a)
    keep = [0, 4, 5]
    assert torch.equal(r[keep], clean[0][keep]) and torch.equal(h[keep], clean[1][keep])
    assert torch.isnan(h[1]).all() and torch.isnan(h[2, 0]) and torch.isnan(r[3, 5])
    assert torch.isnan(r[1, 599]) and torch.equal(r[1, :599], clean[0][1, :599])
    assert torch.equal(r[2, 1:], clean[0][2, 1:]) and torch.isinf(r[2, 0])


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    r, h = hr.norm_residual(x, x, gate=torch.ones((1, 64), dtype=torch.bfloat16, device=DEV))
    assert r.shape == h.shape == (0, 64)
    r, codes, scales = hr.norm_residual_quant_mxfp4(x)
    assert codes.shape == (0, 32) and scales.shape == (0, 2)


@pytest.mark.parametrize("stream,dtype", PAIRS)
@pytest.mark.parametrize("order", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("rows,blocks", [(1, 1), (37, 1), (19, 2), (3, 3), (2, 8), (3, 17), (2, 24)])
@pytest.mark.parametrize("rule", ["floor", "ceil"])
def test_quantized(rows, blocks, order, stream, dtype, rule):
    rng = _rng(order + rows + blocks)
    n = (order or 96) * blocks
    a = _case(rng, rows, n, stream, dtype, gates=1)
    signs = _signs(rng, n) if order else None
    res, codes, scales = hr.norm_residual_quant_mxfp4(**a, order=order or None, signs=None if signs is None else _t(signs),
                                                      rule=rule)
    r, h, size = _oracle(a)
    dr, dh = _bounds(a, r, size)
    assert torch.equal(res, hr.norm_residual(**a)[0])
    off = np.broadcast_to(dh, h.shape)
    if order:
        # the rotation of an error of at most e a value is at most sqrt(order) e
        off = off.reshape(rows, -1, order).max(-1, keepdims=True) * np.sqrt(order)
        off = np.repeat(off[..., 0], order, -1) + rotation_error(h, order)
        h = mxfp4.rotate(h, order, signs)
    check_near(h, off, codes, scales, rule)


@pytest.mark.parametrize("n", [512, 2048, 4096, 8192, 16384, 32768])
def test_quantized_like_the_two_calls(n):
    """In fp32 the fused call and norm, then quantization, see the same h."""
    a = _case(_rng(n), 5, n, "f32", "f32", gates=5)
    signs = _t(_signs(_rng(1), n))
    _, h = hr.norm_residual(**a)
    want = hr.rotate_quant_mxfp4(h, 64, signs)
    _, codes, scales = hr.norm_residual_quant_mxfp4(**a, order=64, signs=signs)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    want = hr.quant_mxfp4(h, "ceil")
    _, codes, scales = hr.norm_residual_quant_mxfp4(**a, rule="ceil")
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


def test_captured_and_replayed():
    a = _case(_rng(3), 50, 1024, "bf16", "bf16", gates=1)
    w = hr.quant_mxfp4(_rows(_rng(4), 64, 1024, torch.bfloat16))

    def step():
        r, codes, scales = hr.norm_residual_quant_mxfp4(**a, order=128)
        return r, hr.mxfp4_gemm(codes, scales, *w, dtype=torch.bfloat16)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):
        a["x"].copy_(_rows(_rng(seed), 50, 1024, torch.bfloat16))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_another_stream():
    a = _case(_rng(5), 700, 2048, "bf16", "bf16")
    want = hr.norm_residual(**a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = hr.norm_residual(**a)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals_on_the_gpu():
    x = torch.zeros((6, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        hr.norm_residual(x, x[:5])
    with pytest.raises(TypeError):
        hr.norm_residual(x, x.float())
    with pytest.raises(ValueError):
        hr.norm_residual(x, x, gate=x[:4])
    with pytest.raises(ValueError):
        hr.norm_residual(x, x, post_weight=torch.ones(64, device=DEV))
    with pytest.raises(ValueError):
        hr.norm_residual(x, x.cpu())
    with pytest.raises(ValueError):
        hr.norm_residual(x, weight=torch.ones(64))
    with pytest.raises(TypeError):
        hr.norm_residual(x, weight=torch.ones(64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        hr.norm_residual(x, gate=x)
    with pytest.raises(ValueError):
        hr.norm_residual(x, residual=x)
    with pytest.raises(ValueError):
        hr.norm_residual_quant_mxfp4(x, order=128)
    with pytest.raises(ValueError):
        hr.norm_residual_quant_mxfp4(x[:, :40])
    with pytest.raises(hr.HRError):
        hr.norm_residual(x, eps=-1.0)


def test_example_blocks():
    """The example: norms, MXFP4 products, cache and attention together, prompt and single tokens.  Each half of a
    block adds a normed output of half the stream's first size, whose products and 4-bit keys and values are some
    0.3 off fp32 (0.11 rms an operand, three products in a row); four of them stay under 0.6 of the whole, where
    unrelated outputs are 1.4 off."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_block.py")
    spec = importlib.util.spec_from_file_location("mxfp4_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    prompt, single, _ = mod.run(layers=2, batch=3, prompt=70, steps=4)
    assert prompt <= 0.6 and single <= 0.6


def test_a_step_captured_and_replayed_in_place():
    """The end of one half, the next product, its end in place: as a decode step captures them."""
    rng = _rng(21)
    n, rows = 2048, 4
    stream = _rows(rng, rows, n, torch.float32)
    start = stream.clone()
    block = _rows(rng, rows, n, torch.bfloat16)
    wt = _t((1 + 0.2 * rng.standard_normal(n)).astype(np.float32))
    signs = _t(_signs(rng, n))
    w = hr.rotate_quant_mxfp4(_rows(rng, n, n, torch.bfloat16, 0.0) / n ** 0.5, 128, signs)

    def step():
        _, codes, scales = hr.norm_residual_quant_mxfp4(stream, block, wt, post_norm=True, post_weight=wt, order=128,
                                                        signs=signs, residual=stream)
        o = hr.mxfp4_gemm(codes, scales, *w, dtype=torch.bfloat16)
        return hr.norm_residual(stream, o, wt, residual=stream)

    step()
    torch.cuda.synchronize()
    stream.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    want = []
    stream.copy_(start)
    for _ in range(4):
        want.append([v.clone() for v in step()])
    stream.copy_(start)
    for r, h in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], r) and torch.equal(out[1], h)


def test_as_many_rows_as_there_may_be():
    rows, n = 1 << 24, 3
    rng = _rng(51)
    some = _rows(rng, 1 << 12, n, torch.bfloat16), _rows(rng, 1 << 12, n, torch.bfloat16)
    x, block = (v.repeat(rows >> 12, 1) for v in some)
    want = hr.norm_residual(*some, post_norm=True)
    got = hr.norm_residual(x, block, post_norm=True)
    for g, w in zip(got, want):
        assert bool((g.view(-1, (1 << 12) * n) == w.view(-1)).all())
    with pytest.raises(hr.HRError):
        hr.norm_residual(torch.zeros(((1 << 24) + 1, 1), dtype=torch.bfloat16, device=DEV))


@pytest.mark.parametrize("n", [40, 2048, 20000])
def test_no_epsilon(n):
    """eps = 0: rows of zeros are 0 / 0, all others as ever."""
    x = _rows(_rng(n), 5, n, torch.float32)
    x[2] = 0.0
    r, h = hr.norm_residual(x, eps=0.0)
    assert torch.equal(r, x) and torch.isnan(h[2]).all()
    keep = [0, 1, 3, 4]
    v = x[keep].double()
    want = v / v.square().mean(-1, keepdim=True).sqrt()
    # the sum's additions, at most 40 one after another in a lane and over lanes, halved by the root; root, quotient, product
    assert ((h[keep].double() - want).abs() <= 24 * 2.0 ** -24 * want.abs()).all()
