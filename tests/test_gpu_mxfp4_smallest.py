"""Rotated MXFP4 of the smallest values there are, on the GPU: subnormal inputs, scale bytes at 0.

Sums of subnormal numbers are exact and a product with 1/sqrt(p) is off by at most half
of 2^-149 beside the bound of normal ones, of which the exchanges add up order / 32.
Reading back, the factor 2^(b - 127) / sqrt(p) of byte 0 is itself off by half of 2^-149, and
multiplies sums of at most 32 * 6 of each of order / 32 blocks.
"""
import numpy as np
import pytest
import torch

import hadamard_rotation_int4_amd as hr
from oracle import mxfp4
from test_gpu_mxfp4 import TYPES, _half_step, _num, _rng, _signs, _t, check_near, rotation_error

pytestmark = pytest.mark.gpu

TYPE_NAMES = ["bf16", "f16", "f32"]


@pytest.mark.parametrize("rule", ["floor", "ceil"])
@pytest.mark.parametrize("dtype", TYPE_NAMES)
@pytest.mark.parametrize("order", [32, 64, 128, 256])
def test_subnormal_rows(order, dtype, rule):
    rng = _rng(order)
    x = rng.standard_normal((6, 768)) * torch.finfo(TYPES[dtype]).tiny * np.ldexp(1.0, np.arange(-4, 2))[:, None]
    x, signs = _t(x).to(TYPES[dtype]), _signs(rng, 768)
    xs = _num(x)
    assert (np.abs(xs)[xs != 0] < torch.finfo(TYPES[dtype]).tiny).mean() > 0.5
    codes, scales = hr.rotate_quant_mxfp4(x, order, _t(signs), rule)
    off = rotation_error(xs, order) + order / 32 * 2.0 ** -149
    check_near(mxfp4.rotate(xs, order, signs), off, codes, scales, rule)


@pytest.mark.parametrize("dtype", TYPE_NAMES)
@pytest.mark.parametrize("order", [32, 64, 128, 256])
def test_smallest_scales_read_back(order, dtype):
    rng = _rng(order + 1)
    packed, scales = rng.integers(0, 256, (9, 384), dtype=np.uint8), rng.integers(0, 5, (9, 24), dtype=np.uint8)
    signs = _signs(rng, 768)
    got = _num(hr.dequant_mxfp4(_t(packed), _t(scales), order, _t(signs), TYPES[dtype]))
    v = mxfp4.values(packed, scales)
    want, half = mxfp4.unrotate(v, order, signs), _half_step(TYPES[dtype])
    off = rotation_error(v, order) + order / 32 * 192 * 2.0 ** -150
    assert (np.abs(got - want) <= off * (1 + half) + np.abs(want) * half + torch.finfo(TYPES[dtype]).tiny * half).all()
