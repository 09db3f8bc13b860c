"""The norms between two blocks in large calls, on the GPU.

A row's lanes and the order of its sums follow from its length alone, so a row's bits
do not depend on how many there are.  Calls large enough that workgroups take several
rows each, that rows are read and written around the L2s, or both, are compared bit
for bit with small calls of the same rows; those small calls go against the fp64 oracle.

Bounds of the small calls, element by element.  r is a few fp32 operations on terms of
size T = |x| + |scale gate u|, within 32 2^-24 T = 2^-19 T.  The factor of h comes from
sum(r^2) + n eps: its own roundings stay under 48 2^-24, halved by the root; r's errors
move the sum by at most 2 2^-19 sum(|r| T), halved likewise.  So h is within
2^-19 |w| T / rms + 2^-19 |h| (1 + sum(|r| T) / (sum(r^2) + n eps)), and half a step of its type.
"""
import numpy as np
import pytest
import torch

import hadamard_rotation_int4_amd as hr
from test_gpu_mxfp4 import DEV, TYPES, _half_step, _num, _rng, _rows, _signs, _t
from test_gpu_norm import EPS, PAIRS, _case, _oracle

pytestmark = pytest.mark.gpu

LENGTHS = [64, 128, 256, 512, 1024, 2048, 4096, 8192, 16384, 32768]
STREAM_BYTES = 64 << 20      # of the stream, from which on aligned rows go around the L2s


def _looped(n):
    """Rows beyond which a workgroup takes at least four turns at rows of n elements."""
    lanes = 8 if n <= 64 else 16 if n <= 128 else 32 if n <= 256 else 64 if n <= 1024 else 256 if n <= 4096 else \
        512 if n <= 8192 else 1024
    threads = max(256, lanes)
    return 4 * (256 * 1024 // threads) * (threads // lanes)


def _many(a, rows, rng):
    """A call of `rows` rows, each one of a's, and which; one gate a row where a has several."""
    at = torch.from_numpy(rng.integers(0, a["x"].shape[0], rows)).to(DEV)
    b = dict(a, x=a["x"][at])
    if a["block_out"] is not None:
        b["block_out"] = a["block_out"][at]
    if a["gate"] is not None and a["gate"].shape[0] > 1:
        b["gate"] = a["gate"][at]
    return b, at


def check_each(a, got, dtype):
    """A small call, each element against its own bound."""
    r, h, size = _oracle(a)
    res, out = got
    # below a type's smallest normal number, tiny, steps no longer shrink: one of 2 half tiny (fp16
    # 2^-24) holds down to 0, and rounding is off by at most half of it, tiny half (2^-14 2^-11)
    half, tiny = _half_step(res.dtype), torch.finfo(res.dtype).tiny
    assert (np.abs(_num(res) - r) <= 2.0 ** -19 * size * (1 + half) + np.abs(r) * half + tiny * half).all()
    wt = 1.0 if a["weight"] is None else np.abs(_num(a["weight"]))
    n = r.shape[1]
    square = (r * r).sum(-1, keepdims=True) + n * a["eps"]
    off = 2.0 ** -19 * (wt * size / np.sqrt(square / n) + np.abs(h) * (1 + (np.abs(r) * size).sum(-1, keepdims=True) / square))
    half = _half_step(dtype)
    assert (np.abs(_num(out) - h) <= off * (1 + half) + np.abs(h) * half + torch.finfo(dtype).tiny * half).all()


@pytest.mark.parametrize("n", [1, 33, 64, 200, 500, 520, 1000, 2047, 2048, 4096, 5000, 8192, 14336, 16385, 32768])
def test_each_element_against_its_own_bound(n):
    """Outlier channels are 20 times the rest: an ordinary element's bound is its own."""
    for stream, dtype in PAIRS:
        for gates in (0, 1, 6):
            a = _case(_rng(n + gates), 6, n, stream, dtype, gates=gates)
            check_each(a, hr.norm_residual(**a), TYPES[dtype])


@pytest.mark.parametrize("short", [0, 3])
@pytest.mark.parametrize("n", LENGTHS)
def test_workgroups_of_several_rows(n, short):
    """Every number of lanes, aligned rows and odd ones: several turns, in place and not."""
    rows, n = _looped(n) + 37, n - short
    for i, (stream, dtype) in enumerate(PAIRS):
        rng = _rng(n + i)
        a = _case(rng, 23, n, stream, dtype, post=i % 2 == 0, gates=(0, 1, 23)[i % 3])
        want = hr.norm_residual(**a)
        check_each(a, want, TYPES[dtype])
        b, at = _many(a, rows, rng)
        r, h = hr.norm_residual(**b)
        assert torch.equal(r, want[0][at]) and torch.equal(h, want[1][at])
        r, h = hr.norm_residual(**b, residual=b["x"])
        assert r is b["x"] and torch.equal(r, want[0][at]) and torch.equal(h, want[1][at])


@pytest.mark.parametrize("n", LENGTHS)
def test_workgroups_of_several_rows_to_mxfp4(n):
    rows = _looped(n) + 37
    for i, (stream, dtype) in enumerate(PAIRS):
        rng = _rng(n + i)
        order = (0, 32, 64, 128, 256)[i]
        order = order if n % (order or 1) == 0 else 0
        signs = _t(_signs(rng, n)) if order else None
        a = _case(rng, 23, n, stream, dtype, post=i % 2 == 1, gates=(23, 0, 1)[i % 3])
        q = dict(order=order or None, signs=signs, rule=("floor", "ceil")[i % 2])
        want = hr.norm_residual_quant_mxfp4(**a, **q)
        b, at = _many(a, rows, rng)
        for got in (hr.norm_residual_quant_mxfp4(**b, **q), hr.norm_residual_quant_mxfp4(**b, **q, residual=b["x"])):
            assert all(torch.equal(g, w[at]) for g, w in zip(got, want))


@pytest.mark.parametrize("n", LENGTHS)
def test_rows_around_the_l2s(n):
    """From 64 MiB of stream on, plain and to MXFP4, in place and not; a few rows more than
    whole turns."""
    for i, (stream, dtype) in enumerate(PAIRS):
        rng = _rng(n + i)
        size = 4 if stream == "f32" else 2
        rows = STREAM_BYTES // (n * size) + 5
        a = _case(rng, 23, n, stream, dtype, post=i % 2 == 0, gates=(1, 23, 0)[i % 3])
        signs = _t(_signs(rng, n))
        q = dict(order=64, signs=signs)
        want, codes = hr.norm_residual(**a), hr.norm_residual_quant_mxfp4(**a, **q)
        b, at = _many(a, rows, rng)
        r, h = hr.norm_residual(**b)
        assert torch.equal(r, want[0][at]) and torch.equal(h, want[1][at])
        got = hr.norm_residual_quant_mxfp4(**b, **q, residual=b["x"])
        assert all(torch.equal(g, w[at]) for g, w in zip(got, codes))


@pytest.mark.parametrize("rows,n,stream,dtype", [(16384, 4096, "bf16", "bf16"), (4096, 16384, "f32", "bf16")])
def test_strided_rows_around_the_l2s(rows, n, stream, dtype):
    rng = _rng(n)
    a = _case(rng, 23, n, stream, dtype, gates=1)
    want = hr.norm_residual(**a)
    b, at = _many(a, rows, rng)
    wide = torch.full((rows, n + 24), 5.0, dtype=TYPES[stream], device=DEV)
    wide[:, 8:8 + n] = b["x"]
    x = wide[:, 8:8 + n]
    r, h = hr.norm_residual(**dict(b, x=x), residual=x)
    assert torch.equal(r, want[0][at]) and torch.equal(h, want[1][at])
    assert (wide[:, :8] == 5.0).all() and (wide[:, 8 + n:] == 5.0).all()


@pytest.mark.parametrize("order", [0, 32, 64, 256])
@pytest.mark.parametrize("stream,dtype", PAIRS)
def test_rows_that_are_not_finite_to_mxfp4(stream, dtype, order):
    """A NaN reaches its whole row, an infinity its own (Hadamard) block, of which the rest of
    the row becomes zeros; no other row changes."""
    rng = _rng(order + 3)
    n, unit = 768, order or 32
    a = _case(rng, 7, n, stream, dtype)
    q = dict(order=order or None, signs=_t(_signs(rng, n)) if order else None)
    _, codes, scales = hr.norm_residual_quant_mxfp4(**a, **q)
    a["x"][1, 700] = float("nan")
    a["x"][2, 0] = float("inf")
    a["block_out"][3, 5] = float("nan")
    a["x"][4, 767] = -float("inf")
    res, got, b = hr.norm_residual_quant_mxfp4(**a, **q)
    keep = [0, 5, 6]
    assert torch.equal(got[keep], codes[keep]) and torch.equal(b[keep], scales[keep])
    for row in (1, 3):
        assert (b[row] == 255).all() and not got[row].any()
    for row, bad in ((2, slice(0, unit // 32)), (4, slice((n - unit) // 32, n // 32))):
        clean = torch.ones(n // 32, dtype=torch.bool, device=DEV)
        clean[bad] = False
        assert (b[row, bad] == 255).all() and not got[row].view(-1, 16)[bad].any()
        assert not b[row, clean].any()
        assert not (got[row].view(-1, 16)[clean] & 0x77).any()      # zeros, of either sign
    assert torch.isnan(res[1, 700]) and torch.isinf(res[2, 0]) and torch.isnan(res[3]).sum() == (n if a["post_norm"] else 1)


def test_the_same_every_time():
    """No sum's order depends on timing: calls repeated over other work give the same bits."""
    rng = _rng(61)
    a = _case(rng, 9000, 4096, "bf16", "bf16", gates=1)
    signs = _t(_signs(rng, 4096))
    want = hr.norm_residual_quant_mxfp4(**a, order=64, signs=signs)
    back = hr.dequant_mxfp4(*want[1:], order=64, signs=signs, dtype=torch.bfloat16)
    x = a["x"]
    there = hr.rotate_quant_mxfp4(x, 128, signs)
    for _ in range(5):
        got = hr.norm_residual_quant_mxfp4(**a, order=64, signs=signs)
        assert all(torch.equal(g, w) for g, w in zip(got, want))
        assert torch.equal(hr.dequant_mxfp4(*got[1:], order=64, signs=signs, dtype=torch.bfloat16), back)
        assert all(torch.equal(g, w) for g, w in zip(hr.rotate_quant_mxfp4(x, 128, signs), there))


@pytest.mark.parametrize("n", [96, 2048, 20000])
def test_magnitudes_up_to_what_sums_of_squares_hold(n):
    """Below 2^64 / sqrt(n) as ever; a row whose sum passes fp32's range has infinite size."""
    for stream, dtype in (("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")):
        rng = _rng(n)
        x = rng.uniform(-1, 1, (4, n)) * 2.0 ** 64 / np.sqrt(n) * 0.99
        a = {"x": _t(x.astype(np.float32)).to(TYPES[stream]), "block_out": None, "weight": None, "post_norm": False,
             "post_weight": None, "gate": None, "scale": 1.0, "eps": EPS}
        got = hr.norm_residual(**a, dtype=TYPES[dtype])
        check_each(a, got, TYPES[dtype])
        a["x"] = a["x"] * 2.0 ** 30
        r, h = hr.norm_residual(**a, dtype=TYPES[dtype])
        assert r is a["x"] and not h.any()
