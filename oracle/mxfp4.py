"""Oracle: MXFP4 (microscaled 4-bit floating point) in fp64.

Test infrastructure only.

Source: the OCP Microscaling Formats specification (blocks of 32 e2m1 elements
under one power-of-two scale, the scale from the exponent of the largest
magnitude); the per-group quantizer it stands in for is that of "Experiment --
Hadamard rotation for int4 (W4A4) accuracy" (Method).
"""
from __future__ import annotations

import numpy as np

from .hadamard import rht

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def rotate(x, order, signs=None):
    """(I kron H_order)(d * x) / sqrt(order) over the last axis (fp64)."""
    x = np.asarray(x, dtype=np.float64)
    if signs is not None:
        x = x * np.asarray(signs, dtype=np.float64)
    return rht(x.reshape(-1, order), np.ones(order, dtype=np.int8)).reshape(x.shape)


def unrotate(y, order, signs=None):
    """The inverse of rotate."""
    x = rotate(y, order)
    return x if signs is None else x * np.asarray(signs, dtype=np.float64)


def scale_bytes(a, rule):
    """Scale byte of blocks whose largest magnitudes are a (fp64)."""
    a = np.asarray(a, dtype=np.float64)
    fine = np.isfinite(a) & (a > 0)
    m, e = np.frexp(np.where(fine, a, 1.0))      # a = m 2^e, 1/2 <= m < 1
    e = e - 1 - 2
    if rule == "ceil":
        e = e + (m > 0.75)
    b = np.where(fine, np.maximum(e, -127) + 127, 0)
    return np.where(np.isfinite(a), b, 255).astype(np.uint8)


def encode(t):
    """Codes of fp64 values t, already divided by their scale: the nearest level
    by distance, the even code of two equally near, sign kept."""
    t = np.asarray(t, dtype=np.float64)
    a = np.minimum(np.abs(t), 6.0)
    dist = np.abs(a[..., None] - LEVELS)
    near = dist == dist.min(-1, keepdims=True)
    even = np.argmax(near & (np.arange(8) % 2 == 0), -1)
    first = np.argmax(near, -1)
    code = np.where((near & (np.arange(8) % 2 == 0)).any(-1), even, first)
    return (code | (np.signbit(t).astype(np.int64) << 3)).astype(np.uint8)


def quantize(y, rule="floor"):
    """(codes uint8 [..., n], scale bytes uint8 [..., n/32]) of fp64 rows y."""
    y = np.asarray(y, dtype=np.float64)
    g = y.reshape(*y.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        b = scale_bytes(np.abs(g).max(-1), rule)      # NaN and infinity come through the maximum
        t = g / np.ldexp(1.0, b.astype(np.int64) - 127)[..., None]
    codes = np.where(b[..., None] == 255, 0, encode(np.where(np.isfinite(t), t, 0.0)))
    return codes.reshape(y.shape).astype(np.uint8), b


def pack(codes):
    """Codes [..., n] -> bytes [..., n/2], the even element in the low nibble."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty((*packed.shape[:-1], 2 * packed.shape[-1]), dtype=np.uint8)
    out[..., 0::2] = packed & 15
    out[..., 1::2] = packed >> 4
    return out


def values(packed, scales):
    """fp64 rows that packed codes and scale bytes stand for; NaN under byte 255."""
    c = unpack(packed)
    v = np.where(c & 8, -LEVELS[c & 7], LEVELS[c & 7])
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def gemm(a, sa, w, sw):
    """C = A W^T in fp64, and the sums of magnitudes that bound its rounding."""
    x, y = values(a, sa), values(w, sw)
    return x @ y.T, np.abs(x) @ np.abs(y).T
