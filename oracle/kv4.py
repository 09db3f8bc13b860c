"""Oracle: the 4-bit key/value cache and attention over it, in fp64.

Test infrastructure only.

Source: the quantizer and the rotation of "Experiment -- Hadamard rotation for
int4 (W4A4) accuracy" (Hypothesis and Method) applied per attention head; the
sign diagonal of HARP's incoherence processing.  Softmax attention itself is
the textbook definition.

Cache layout: codes uint8 [pages][heads][page][dim/2] (packed int4, see
``quant``), scales fp16 [pages][heads][dim/group][page].
"""
from __future__ import annotations

import numpy as np

from .hadamard import rht
from .quant import unpack_int4


def rotate(x, signs):
    """y = H (d * x) / sqrt(dim) over the last axis (fp64)."""
    x = np.asarray(x, dtype=np.float64)
    s = np.ones(x.shape[-1], dtype=np.int8) if signs is None else np.asarray(signs)
    return rht(x.reshape(-1, x.shape[-1]), s).reshape(x.shape)


def unrotate(y, signs):
    """The inverse: d * H y / sqrt(dim) (H is symmetric)."""
    y = np.asarray(y, dtype=np.float64)
    ones = np.ones(y.shape[-1], dtype=np.int8)
    x = rht(y.reshape(-1, y.shape[-1]), ones).reshape(y.shape)
    return x if signs is None else x * np.asarray(signs, dtype=np.float64)


def quantize_plain(x, group):
    """The stored codes (int8) and fp16 scales of fp32 vectors [..., dim] without
    a rotation, every step in fp32: s = fp16(a / 7), k = 1 / s, q = rint(y k).
    A vector that is not finite, or needs a scale above 9352, gets zero codes and
    NaN scales."""
    y = np.asarray(x, dtype=np.float32)
    g = y.reshape(*y.shape[:-1], -1, group)
    with np.errstate(all="ignore"):
        s = (np.abs(g).max(-1) / np.float32(7)).astype(np.float16)
        f = s.astype(np.float32)[..., None]
        k = np.where(f > 0, np.float32(1) / np.where(f > 0, f, np.float32(1)), np.float32(0)).astype(np.float32)
        q = np.clip(np.rint((g * k).astype(np.float32)), -7, 7)
    bad = ~(np.isfinite(y).all(-1) & (s <= np.float16(9352)).all(-1))
    q = np.where(bad[..., None, None], 0, q)
    s = np.where(bad[..., None], np.float16(np.nan), s)
    return q.reshape(y.shape).astype(np.int8), s


def values(codes, scales):
    """fp64 values [pages][heads][page][dim] that a cache's codes and scales hold
    (in the rotated basis)."""
    pages, heads, page, half = codes.shape
    q = unpack_int4(codes.reshape(-1, half)).astype(np.float64).reshape(pages, heads, page, 2 * half)
    s = np.swapaxes(scales.astype(np.float64), -1, -2)          # [pages][heads][page][groups]
    return q * np.repeat(s, 2 * half // s.shape[-1], axis=-1)


def gather(vals, table_row, length):
    """[heads][length][dim] of one sequence."""
    page = vals.shape[2]
    j = np.arange(length)
    return np.moveaxis(vals[np.asarray(table_row)[j // page], :, j % page], 0, 1)


def attention(q, kvals, vvals, table, lens, starts, scale, signs=None, rotated=True, causal=True, window=0):
    """out [total][q_heads][dim] in fp64 of queries over cache values kvals,
    vvals (``values`` of the cache); 0 in a row that sees no token.  A NaN in a
    key or a value reaches the rows that see it and no other."""
    q = np.asarray(q, dtype=np.float64)
    total, q_heads, dim = q.shape
    rep = q_heads // kvals.shape[1]
    out = np.zeros_like(q)
    qr = rotate(q, signs) if rotated else q
    for b, n in enumerate(lens):
        s0, s1 = int(starts[b]), int(starts[b + 1])
        n = int(n)
        if n == 0:
            continue
        k, v = gather(kvals, table[b], n), gather(vvals, table[b], n)
        j = np.arange(n)
        for t in range(s0, s1):
            pos = n - (s1 - s0) + (t - s0)
            see = np.ones(n, dtype=bool)
            if causal:
                see &= j <= pos
            if window:
                see &= j > pos - window
            if not see.any():
                continue
            for h in range(q_heads):
                z = scale * (k[h // rep][see] @ qr[t, h])
                with np.errstate(invalid="ignore"):
                    p = np.exp(z - z.max())
                    out[t, h] = (p / p.sum()) @ v[h // rep][see]
    return unrotate(out, signs) if rotated else out
