"""Oracle: the norms between two blocks of a layer, in fp64.

Test infrastructure only.  Root-mean-square norms, a gate and a residual scale:
textbook definitions.
"""
from __future__ import annotations

import numpy as np


def norm_residual(x, block=None, weight=None, post_norm=False, post_weight=None, gate=None, scale=1.0, eps=1e-6):
    """(r, h, size): size bounds the terms of r, |x| + |scale gate u|."""
    x = np.asarray(x, dtype=np.float64)
    size = np.abs(x)
    r = x
    if block is not None:
        u = np.asarray(block, dtype=np.float64)
        if post_norm:
            u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
            if post_weight is not None:
                u = u * np.asarray(post_weight, dtype=np.float64)
        if gate is not None:
            g = np.asarray(gate, dtype=np.float64)
            u = u * np.repeat(g, x.shape[0] // g.shape[0], axis=0)
        r = x + scale * u
        size = size + np.abs(scale * u)
    h = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    if weight is not None:
        h = h * np.asarray(weight, dtype=np.float64)
    return r, h, size
