"""CPU-only checks of the MXFP4 and norm calls: refusals of the C entry points and
of the binding (nothing here launches a kernel), and pins of the oracle they are
tested against."""
import ctypes

import numpy as np
import pytest
import torch

import hadamard_rotation_int4_amd as hr
from oracle import mxfp4, norm

P = 0x10000      # a fake 16-byte aligned address, never dereferenced


# ------------------------------------------------------------------ the C entry points

def _quant(fn="hr_rotate_quant_mxfp4", **kw):
    a = dict(x=P, dt=hr.HR_BF16, stride=256, rows=4, n=256, order=128, signs=P, rule=0, codes=P, scales=P)
    a.update(kw)
    if fn == "hr_quant_mxfp4":
        return hr.lib.hr_quant_mxfp4(a["x"], a["dt"], a["stride"], a["rows"], a["n"], a["rule"], a["codes"],
                                     a["scales"], None)
    return hr.lib.hr_rotate_quant_mxfp4(a["x"], a["dt"], a["stride"], a["rows"], a["n"], a["order"], a["signs"],
                                        a["rule"], a["codes"], a["scales"], None)


@pytest.mark.parametrize("fn", ["hr_quant_mxfp4", "hr_rotate_quant_mxfp4"])
@pytest.mark.parametrize("kw,status", [
    (dict(x=None), hr.HR_EINVAL),
    (dict(codes=None), hr.HR_EINVAL),
    (dict(scales=None), hr.HR_EINVAL),
    (dict(x=P + 8), hr.HR_EINVAL),
    (dict(codes=P + 4), hr.HR_EINVAL),
    (dict(dt=3), hr.HR_EINVAL),
    (dict(rule=2), hr.HR_EINVAL),
    (dict(rule=-1), hr.HR_EINVAL),
    (dict(rows=-1), hr.HR_EINVAL),
    (dict(stride=255), hr.HR_EINVAL),            # rows would overlap
    (dict(stride=260), hr.HR_EINVAL),            # not a multiple of 16 bytes
    (dict(n=0), hr.HR_EUNSUPPORTED),
    (dict(n=-32), hr.HR_EUNSUPPORTED),
    (dict(n=48), hr.HR_EUNSUPPORTED),
    (dict(n=(1 << 18) + 256, stride=1 << 20), hr.HR_EUNSUPPORTED),
    (dict(rows=(1 << 26) + 1), hr.HR_EUNSUPPORTED),
    (dict(rows=0), hr.HR_OK),
    (dict(rows=0, x=None, codes=None, scales=None), hr.HR_OK),
])
def test_quant_refusals(fn, kw, status):
    assert _quant(fn, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(order=0), hr.HR_EUNSUPPORTED),
    (dict(order=16), hr.HR_EUNSUPPORTED),
    (dict(order=512, n=512, stride=512), hr.HR_EUNSUPPORTED),
    (dict(order=256, n=384, stride=384), hr.HR_EUNSUPPORTED),
    (dict(signs=P + 4), hr.HR_EINVAL),
])
def test_rotation_refusals(kw, status):
    assert _quant(**kw) == status


def _dequant(**kw):
    a = dict(codes=P, scales=P, rows=4, n=256, order=128, signs=P, dt=hr.HR_F32, out=P)
    a.update(kw)
    return hr.lib.hr_dequant_mxfp4(a["codes"], a["scales"], a["rows"], a["n"], a["order"], a["signs"], a["dt"],
                                   a["out"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(codes=None), hr.HR_EINVAL),
    (dict(scales=None), hr.HR_EINVAL),
    (dict(out=None), hr.HR_EINVAL),
    (dict(out=P + 8), hr.HR_EINVAL),
    (dict(order=0), hr.HR_EINVAL),               # signs without an order
    (dict(order=48, n=96), hr.HR_EUNSUPPORTED),
    (dict(n=40, order=0, signs=None), hr.HR_EUNSUPPORTED),
    (dict(dt=5), hr.HR_EINVAL),
    (dict(rows=-3), hr.HR_EINVAL),
    (dict(rows=0, codes=None, scales=None, out=None), hr.HR_OK),
])
def test_dequant_refusals(kw, status):
    assert _dequant(**kw) == status


def _gemm(**kw):
    a = dict(a=P, sa=P, w=P, sw=P, M=4, N=8, K=64, dt=hr.HR_BF16, c=P)
    a.update(kw)
    return hr.lib.hr_mxfp4_gemm(a["a"], a["sa"], a["w"], a["sw"], a["M"], a["N"], a["K"], a["dt"], a["c"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(a=None), hr.HR_EINVAL),
    (dict(sa=None), hr.HR_EINVAL),
    (dict(w=None), hr.HR_EINVAL),
    (dict(sw=None), hr.HR_EINVAL),
    (dict(c=None), hr.HR_EINVAL),
    (dict(a=P + 8), hr.HR_EINVAL),
    (dict(w=P + 2), hr.HR_EINVAL),
    (dict(c=P + 4), hr.HR_EINVAL),
    (dict(M=-1), hr.HR_EINVAL),
    (dict(dt=3), hr.HR_EINVAL),
    (dict(K=0), hr.HR_EUNSUPPORTED),
    (dict(K=48), hr.HR_EUNSUPPORTED),
    (dict(K=(1 << 18) + 32), hr.HR_EUNSUPPORTED),
    (dict(M=(1 << 21) + 1), hr.HR_EUNSUPPORTED),
    (dict(N=1 << 40), hr.HR_EUNSUPPORTED),
    (dict(M=1 << 21, N=1 << 16, K=128), hr.HR_EUNSUPPORTED),
    (dict(M=1 << 21, N=1 << 16), hr.HR_EUNSUPPORTED),
    (dict(M=0, a=None, sa=None, c=None), hr.HR_OK),
    (dict(N=0, w=None, sw=None, c=None), hr.HR_OK),
])
def test_gemm_refusals(kw, status):
    assert _gemm(**kw) == status


def _norm(mx=False, **kw):
    a = dict(x=P, block_out=P, post_weight=P, gate=P, weight=P, rows=6, x_stride=64, block_stride=64, gates=2, n=64,
             x_dtype=hr.HR_BF16, dtype=hr.HR_BF16, post_norm=1, scale=1.0, eps=1e-6, residual=P, rs=64, h=P, order=64,
             signs=P, rule=0, codes=P, scales=P)
    a.update(kw)
    p = hr._NormStruct(**{k: a[k] for k, _ in hr._NormStruct._fields_})
    ref = ctypes.addressof(p)
    if mx:
        return hr.lib.hr_norm_residual_quant_mxfp4(ref, a["residual"], a["rs"], a["order"], a["signs"], a["rule"],
                                                   a["codes"], a["scales"], None)
    return hr.lib.hr_norm_residual(ref, a["residual"], a["rs"], a["h"], None)


ALONE = dict(block_out=None, post_weight=None, gate=None, post_norm=0, residual=None)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(x=None), hr.HR_EINVAL),
    (dict(x=P + 1), hr.HR_EINVAL),
    (dict(residual=None), hr.HR_EINVAL),
    (dict(residual=P + 1), hr.HR_EINVAL),
    (dict(weight=P + 2), hr.HR_EINVAL),
    (dict(x_stride=63), hr.HR_EINVAL),
    (dict(block_stride=63), hr.HR_EINVAL),
    (dict(rs=63), hr.HR_EINVAL),
    (dict(gates=4), hr.HR_EINVAL),
    (dict(gates=0), hr.HR_EINVAL),
    (dict(post_norm=0), hr.HR_EINVAL),           # a weight for no norm
    (dict(post_norm=2), hr.HR_EINVAL),
    (dict(eps=-1.0), hr.HR_EINVAL),
    (dict(eps=float("nan")), hr.HR_EINVAL),
    (dict(scale=float("inf")), hr.HR_EINVAL),
    (dict(rows=-1), hr.HR_EINVAL),
    (dict(x_dtype=4), hr.HR_EINVAL),
    (dict(dtype=hr.HR_F16), hr.HR_EUNSUPPORTED),
    (dict(n=0), hr.HR_EUNSUPPORTED),
    (dict(n=32800, x_stride=32800, block_stride=32800, rs=32800), hr.HR_EUNSUPPORTED),
    (dict(rows=(1 << 24) + 2), hr.HR_EUNSUPPORTED),
    (dict(block_out=None), hr.HR_EINVAL),        # a gate and a norm of nothing
    ({**ALONE, "residual": P}, hr.HR_EINVAL),
    (dict(rows=0), hr.HR_OK),
    ({**ALONE, "rows": 0, "x": None, "h": None, "codes": None, "scales": None}, hr.HR_OK),
])
def test_norm_refusals(mx, kw, status):
    assert _norm(mx, **kw) == status


def test_norm_needs_a_description():
    assert hr.lib.hr_norm_residual(None, P, 64, P, None) == hr.HR_EINVAL
    assert hr.lib.hr_norm_residual_quant_mxfp4(None, P, 64, 0, None, 0, P, P, None) == hr.HR_EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(h=P + 1), hr.HR_EINVAL),
    ({**ALONE, "h": None}, hr.HR_EINVAL),        # nothing to compute
])
def test_norm_plain_refusals(kw, status):
    assert _norm(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(codes=None), hr.HR_EINVAL),
    (dict(scales=None), hr.HR_EINVAL),
    (dict(codes=P + 4), hr.HR_EINVAL),
    (dict(rule=7), hr.HR_EINVAL),
    (dict(order=0), hr.HR_EINVAL),               # signs without an order
    (dict(order=128), hr.HR_EUNSUPPORTED),
    (dict(n=60, order=0, signs=None), hr.HR_EUNSUPPORTED),
])
def test_norm_quant_refusals(kw, status):
    assert _norm(True, **kw) == status


# ------------------------------------------------------------------ the binding

def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


@pytest.mark.parametrize("error,call", [
    (TypeError, lambda: hr.quant_mxfp4([1.0])),
    (TypeError, lambda: hr.quant_mxfp4(_cpu(2, 64, dtype=torch.int32))),
    (ValueError, lambda: hr.quant_mxfp4(_cpu(64))),
    (ValueError, lambda: hr.quant_mxfp4(_cpu(2, 48))),
    (ValueError, lambda: hr.quant_mxfp4(_cpu(2, 64), rule="up")),
    (ValueError, lambda: hr.quant_mxfp4(_cpu(64, 2).t())),
    (ValueError, lambda: hr.quant_mxfp4(_cpu(1, 64).expand(3, 64))),
    (ValueError, lambda: hr.quant_mxfp4(_cpu(2, 64))),                                   # not on the GPU
    (ValueError, lambda: hr.rotate_quant_mxfp4(_cpu(2, 64), 128)),
    (ValueError, lambda: hr.rotate_quant_mxfp4(_cpu(2, 64), 0)),
    (ValueError, lambda: hr.rotate_quant_mxfp4(_cpu(2, 64), 48)),
    (ValueError, lambda: hr.rotate_quant_mxfp4(_cpu(2, 64), 64, torch.ones(32, dtype=torch.int8))),
    (TypeError, lambda: hr.rotate_quant_mxfp4(_cpu(2, 64), 64, torch.ones(64))),
    (TypeError, lambda: hr.dequant_mxfp4(_cpu(2, 32), _u8(2, 2))),
    (ValueError, lambda: hr.dequant_mxfp4(_u8(2, 32), _u8(2, 4))),
    (ValueError, lambda: hr.dequant_mxfp4(_u8(2, 24), _u8(2, 2))),
    (ValueError, lambda: hr.dequant_mxfp4(_u8(2, 32), _u8(2, 2), signs=torch.ones(64, dtype=torch.int8))),
    (TypeError, lambda: hr.dequant_mxfp4(_u8(2, 32), _u8(2, 2), dtype=torch.int8)),
    (ValueError, lambda: hr.dequant_mxfp4(_u8(2, 32), _u8(2, 2))),
    (TypeError, lambda: hr.mxfp4_gemm(_cpu(2, 32), _u8(2, 2), _u8(3, 32), _u8(3, 2))),
    (ValueError, lambda: hr.mxfp4_gemm(_u8(2, 24), _u8(2, 1), _u8(3, 24), _u8(3, 1))),
    (ValueError, lambda: hr.mxfp4_gemm(_u8(2, 0), _u8(2, 0), _u8(3, 0), _u8(3, 0))),
    (ValueError, lambda: hr.mxfp4_gemm(_u8(2, 32), _u8(2, 2), _u8(3, 64), _u8(3, 4))),
    (ValueError, lambda: hr.mxfp4_gemm(_u8(2, 32), _u8(2, 1), _u8(3, 32), _u8(3, 2))),
    (ValueError, lambda: hr.mxfp4_gemm(_u8(2, 32), _u8(2, 2), _u8(3, 32), _u8(2, 2))),
    (TypeError, lambda: hr.mxfp4_gemm(_u8(2, 32), _u8(2, 2), _u8(3, 32), _u8(3, 2), dtype=torch.float64)),
    (ValueError, lambda: hr.mxfp4_gemm(_u8(2, 32), _u8(2, 2), _u8(3, 32), _u8(3, 2))),
    (TypeError, lambda: hr.norm_residual(None)),
    (ValueError, lambda: hr.norm_residual(_cpu(4, 0))),
    (TypeError, lambda: hr.norm_residual(_cpu(4, 8), dtype=torch.float16)),
    (TypeError, lambda: hr.norm_residual(_cpu(4, 8), dtype=torch.int8)),
    (ValueError, lambda: hr.norm_residual(_cpu(4, 8), want_h=False)),
    (ValueError, lambda: hr.norm_residual(_cpu(4, 8), post_norm=True)),
    (ValueError, lambda: hr.norm_residual(_cpu(4, 8))),
])
def test_binding_refusals(error, call):
    with pytest.raises(error):
        call()


@pytest.mark.parametrize("current", [0, 1])
def test_calls_go_to_the_tensors_device(monkeypatch, current):
    """Tensors on device 1: its stream, and device 1 the current one during the call."""
    import contextlib

    now, seen = [current], []

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], index
        yield
        now[0] = before

    def call(a, stream):
        seen.append((a, stream, now[0]))
        return 0

    monkeypatch.setattr(hr, "_get_device", lambda: now[0])
    monkeypatch.setattr(hr, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(hr, "_stream", lambda index: 100 + index)
    monkeypatch.setattr(torch.cuda, "device", device)
    hr._launch(1, call, 5)
    assert seen == [(5, 101, 1)] and now[0] == current


@pytest.mark.parametrize("current,fast", [(0, True), (1, True), (0, False)])
def test_outputs_are_made_on_the_tensors_device(monkeypatch, current, fast):
    made = []
    monkeypatch.setattr(hr, "_get_device", lambda: current)
    monkeypatch.setattr(hr, "_empty_cuda", (lambda *a: made.append(("fast", *a))) if fast else None)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(("empty", *a, k)))
    hr._new(0, 3, 5, torch.uint8)
    if fast and current == 0:
        assert made == [("fast", (3, 5), (5, 1), torch.uint8)]
    else:
        assert made == [("empty", (3, 5), {"dtype": torch.uint8, "device": torch.device("cuda", 0)})]


def test_a_call_that_fails_raises():
    def hr_call(stream):
        return hr.HR_EDEVICE

    with pytest.MonkeyPatch.context() as m:
        m.setattr(hr, "_get_device", lambda: 0)
        m.setattr(hr, "_raw_stream", lambda index: 0)
        with pytest.raises(hr.HRError):
            hr._launch(0, hr_call)


# ------------------------------------------------------------------ the oracle

def test_levels_and_their_codes():
    both = np.concatenate([mxfp4.LEVELS, -mxfp4.LEVELS])
    assert np.array_equal(mxfp4.encode(both), np.arange(16))
    for i in range(7):       # half way: the even code
        mid = (mxfp4.LEVELS[i] + mxfp4.LEVELS[i + 1]) / 2
        assert mxfp4.encode(mid) == (i if i % 2 == 0 else i + 1)
        assert mxfp4.encode(np.nextafter(mid, 0)) == i
        assert mxfp4.encode(np.nextafter(mid, 9)) == i + 1
    assert mxfp4.encode(7.99) == 7 and mxfp4.encode(-100.0) == 15 and mxfp4.encode(-0.0) == 8


@pytest.mark.parametrize("a,floor,ceil", [
    (4.0, 127, 127), (6.0, 127, 127), (np.nextafter(6.0, 7), 127, 128), (7.9, 127, 128), (8.0, 128, 128),
    (1.0, 125, 125), (2.0 ** -125, 0, 0), (2.0 ** -126, 0, 0), (2.0 ** -149, 0, 0), (0.0, 0, 0),
    (2.0 ** -124 * 1.75, 1, 2), (np.float64(np.finfo(np.float32).max), 252, 253), (np.inf, 255, 255),
    (np.nan, 255, 255),
])
def test_scale_bytes(a, floor, ceil):
    assert mxfp4.scale_bytes(a, "floor") == floor
    assert mxfp4.scale_bytes(a, "ceil") == ceil


def test_a_block_by_hand():
    y = np.zeros(64)
    y[:8] = [12, -8, 6, 5, -2.5, 1, 0.4, -0.1]       # scale 2: 6, -4, 3, 2.5 -> 2, -1.25 -> -1, .5, .2 -> 0, -0
    codes, b = mxfp4.quantize(y)
    assert list(b) == [128, 0]
    assert list(codes[:8]) == [7, 14, 5, 4, 10, 1, 0, 8] and not codes[8:].any()
    back = mxfp4.values(mxfp4.pack(codes), b)
    assert list(back[:8]) == [12, -8, 6, 4, -2, 1, 0, 0]
    assert np.array_equal(mxfp4.unpack(mxfp4.pack(codes)), codes)


def test_quantizing_what_was_read_back_changes_nothing():
    rng = np.random.Generator(np.random.PCG64(1))
    y = rng.standard_normal((5, 96)) * np.exp(3 * rng.standard_normal((5, 1)))
    codes, b = mxfp4.quantize(y, "ceil")
    back = mxfp4.values(mxfp4.pack(codes), b)
    again, b2 = mxfp4.quantize(back, "ceil")
    assert np.array_equal(mxfp4.values(mxfp4.pack(again), b2), back)
    assert np.abs(y - back).max() <= (np.repeat(np.ldexp(1.0, b.astype(int) - 127), 32, -1)).max()


@pytest.mark.parametrize("order", [32, 64, 128, 256])
def test_rotation_and_back(order):
    rng = np.random.Generator(np.random.PCG64(order))
    x = rng.standard_normal((3, 2 * order))
    signs = rng.integers(0, 2, 2 * order) * 2 - 1
    y = mxfp4.rotate(x, order, signs)
    assert np.allclose(mxfp4.unrotate(y, order, signs), x, atol=1e-12)
    i = np.arange(order)
    h = np.array([[(-1) ** bin(a & b).count("1") for b in i] for a in i]) / np.sqrt(order)
    assert np.allclose(y[:, order:], (x * signs)[:, order:] @ h, atol=1e-12)


def test_gemm_by_hand():
    rng = np.random.Generator(np.random.PCG64(2))
    a, w = (rng.integers(0, 256, (r, 32), dtype=np.uint8) for r in (2, 3))
    sa, sw = (rng.integers(120, 134, (r, 2), dtype=np.uint8) for r in (2, 3))
    c, size = mxfp4.gemm(a, sa, w, sw)
    for m in range(2):
        for n in range(3):
            t = 0.0
            for k in range(64):
                p = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
                qa = p[a[m, k // 2] >> 4 * (k % 2) & 15] * 2.0 ** (int(sa[m, k // 32]) - 127)
                qw = p[w[n, k // 2] >> 4 * (k % 2) & 15] * 2.0 ** (int(sw[n, k // 32]) - 127)
                t += qa * qw
            assert np.isclose(c[m, n], t, rtol=1e-13)
    assert (np.abs(c) <= size).all()


def test_norm_by_hand():
    x, o = np.array([[3.0, -4.0], [1.0, 1.0]]), np.array([[1.0, 7.0], [0.0, 0.0]])
    r, h, _ = norm.norm_residual(x, eps=0.0, weight=np.array([2.0, 1.0]))
    assert np.array_equal(r, x) and np.allclose(h, [[6 / np.sqrt(12.5), -4 / np.sqrt(12.5)], [2, 1]])
    r, h, _ = norm.norm_residual(x, o, post_norm=True, post_weight=np.array([5.0, 10.0]), gate=np.array([[2.0, 0.5]]),
                                 scale=0.1, eps=1e-30)
    assert np.allclose(r, [[3 + 0.1 * 2 * 5 / 5, -4 + 0.1 * 0.5 * 10 * 7 / 5], [1, 1]])
    r, _, _ = norm.norm_residual(x, o, gate=np.array([[1.0, 0.0], [3.0, 3.0]]), scale=2.0)
    assert np.array_equal(r, [[5, -4], [1, 1]])
