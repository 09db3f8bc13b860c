"""CPU-only checks of the 4-bit key/value cache calls: refusals of the C entry
points and of the binding (nothing here launches a kernel), and pins of the
oracle they are tested against."""
import ctypes

import numpy as np
import pytest
import torch

import hadamard_rotation_int4_amd as hr
import oracle

P = 0x10000      # a fake 16-byte aligned address, never dereferenced


def _cache(**kw):
    a = dict(k_codes=P, k_scales=P, v_codes=P, v_scales=P, signs=P, pages=4, heads=2, dim=128, page=64, group=128,
             rotate=1)
    a.update(kw)
    c = hr._CacheStruct(**a)
    return c, ctypes.addressof(c)


def _append(cache=None, **kw):
    c, ref = _cache(**(cache or {}))
    a = dict(ref=ref, k=P, v=P, dt=hr.HR_BF16, ks=256, vs=256, slots=P, tokens=4)
    a.update(kw)
    return hr.lib.hr_kv4_append(a["ref"], a["k"], a["v"], a["dt"], a["ks"], a["vs"], a["slots"], a["tokens"], None)


def _read(cache=None, **kw):
    c, ref = _cache(**(cache or {}))
    a = dict(ref=ref, slots=P, tokens=4, dt=hr.HR_BF16, k=P, v=P)
    a.update(kw)
    return hr.lib.hr_kv4_read(a["ref"], a["slots"], a["tokens"], a["dt"], a["k"], a["v"], None)


def _attend(cache=None, **kw):
    c, ref = _cache(**(cache or {}))
    a = dict(ref=ref, q=P, dt=hr.HR_BF16, qs=1024, total=4, starts=None, table=P, width=4, lens=P, batch=4,
             q_heads=8, max_new=1, max_len=256, scale=0.1, causal=1, window=0, out=P, ws=None, wsb=0)
    a.update(kw)
    return hr.lib.hr_kv4_attention(a["ref"], a["q"], a["dt"], a["qs"], a["total"], a["starts"], a["table"],
                                   a["width"], a["lens"], a["batch"], a["q_heads"], a["max_new"], a["max_len"],
                                   a["scale"], a["causal"], a["window"], a["out"], a["ws"], a["wsb"], None)


BAD_CACHES = [
    (dict(k_codes=None), hr.HR_EINVAL),
    (dict(v_scales=None), hr.HR_EINVAL),
    (dict(k_scales=P + 8), hr.HR_EINVAL),
    (dict(signs=P + 4), hr.HR_EINVAL),
    (dict(pages=-1), hr.HR_EINVAL),
    (dict(pages=1 << 31), hr.HR_EUNSUPPORTED),
    (dict(rotate=2), hr.HR_EINVAL),
    (dict(dim=96), hr.HR_EUNSUPPORTED),
    (dict(dim=512), hr.HR_EUNSUPPORTED),
    (dict(group=256), hr.HR_EUNSUPPORTED),
    (dict(group=16), hr.HR_EUNSUPPORTED),
    (dict(page=8), hr.HR_EUNSUPPORTED),
    (dict(page=48), hr.HR_EUNSUPPORTED),
    (dict(page=1 << 21), hr.HR_EUNSUPPORTED),
    (dict(heads=0), hr.HR_EUNSUPPORTED),
]


@pytest.mark.parametrize("call", [_append, _read, _attend])
@pytest.mark.parametrize("cache,status", BAD_CACHES)
def test_cache_refusals(call, cache, status):
    assert call(cache) == status
    assert hr.lib.hr_last_error() != b""


@pytest.mark.parametrize("call", [_append, _read, _attend])
def test_no_cache(call):
    assert call(ref=None) == hr.HR_EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), hr.HR_EINVAL),
    (dict(v=None), hr.HR_EINVAL),
    (dict(slots=None), hr.HR_EINVAL),
    (dict(k=P + 8), hr.HR_EINVAL),
    (dict(slots=P + 4), hr.HR_EINVAL),
    (dict(dt=3), hr.HR_EINVAL),
    (dict(ks=248), hr.HR_EINVAL),                # rows would overlap
    (dict(vs=260), hr.HR_EINVAL),                # not a multiple of 16 bytes
    (dict(tokens=-1), hr.HR_EINVAL),
    (dict(tokens=1 << 31), hr.HR_EUNSUPPORTED),
    (dict(tokens=0), hr.HR_OK),
    (dict(tokens=0, k=None, v=None, slots=None), hr.HR_OK),
])
def test_append_refusals(kw, status):
    assert _append(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), hr.HR_EINVAL),
    (dict(v=P + 4), hr.HR_EINVAL),
    (dict(slots=None), hr.HR_EINVAL),
    (dict(dt=-1), hr.HR_EINVAL),
    (dict(tokens=-2), hr.HR_EINVAL),
    (dict(tokens=0, k=None, v=None, slots=None), hr.HR_OK),
])
def test_read_refusals(kw, status):
    assert _read(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), hr.HR_EINVAL),
    (dict(out=None), hr.HR_EINVAL),
    (dict(lens=None), hr.HR_EINVAL),
    (dict(table=None), hr.HR_EINVAL),
    (dict(q=P + 2), hr.HR_EINVAL),
    (dict(lens=P + 2), hr.HR_EINVAL),
    (dict(dt=9), hr.HR_EINVAL),
    (dict(q_heads=7), hr.HR_EUNSUPPORTED),
    (dict(q_heads=0), hr.HR_EUNSUPPORTED),
    (dict(qs=1000), hr.HR_EINVAL),
    (dict(qs=1028), hr.HR_EINVAL),
    (dict(total=5), hr.HR_EINVAL),               # no starts, not batch * max_new
    (dict(causal=2), hr.HR_EINVAL),
    (dict(window=-1), hr.HR_EINVAL),
    (dict(scale=0.0), hr.HR_EINVAL),
    (dict(scale=float("nan")), hr.HR_EINVAL),
    (dict(scale=float("inf")), hr.HR_EINVAL),
    (dict(max_len=-1), hr.HR_EINVAL),
    (dict(max_len=(1 << 30) + 1), hr.HR_EUNSUPPORTED),
    (dict(batch=70000, total=70000), hr.HR_EUNSUPPORTED),
    (dict(max_len=100000), hr.HR_EINVAL),        # split over the tokens: needs a workspace
    (dict(max_len=100000, ws=P, wsb=64), hr.HR_EINVAL),
    (dict(total=0, batch=0, q=None, out=None, lens=None, table=None), hr.HR_OK),
])
def test_attention_refusals(kw, status):
    assert _attend(**kw) == status


def test_workspace_sizes():
    f = hr.lib.hr_kv4_attention_workspace
    assert f(8, 128, hr.HR_BF16, 1, 1, 32, 1, 200, 0) == 0
    big = f(8, 128, hr.HR_BF16, 1, 1, 32, 1, 131072, 0)
    assert big > 0 and big % (16 * (128 * 4 + 8)) == 0
    assert f(8, 128, hr.HR_BF16, 1, 1, 32, 1, 131072, 100) == 0           # a window leaves little to split
    for bad in ((0, 128, 1, 1, 1, 32, 1, 9, 0), (8, 128, 1, -1, 1, 32, 1, 9, 0), (8, 128, 1, 1, 1, 4, 1, 9, 0)):
        assert f(*bad) == 0


def _tensors(**kw):
    a = dict(pages=2, heads=2, page=16, dim=64, groups=1)
    a.update(kw)
    c = torch.zeros((a["pages"], a["heads"], a["page"], a["dim"] // 2), dtype=torch.uint8)
    s = torch.zeros((a["pages"], a["heads"], a["groups"], a["page"]), dtype=torch.float16)
    return [c, s, c.clone(), s.clone()]


def test_binding_refusals():
    good = _tensors()
    with pytest.raises(ValueError, match="GPU"):
        hr.KV4Cache(*good)
    for i, t, err in ((0, None, TypeError), (2, None, TypeError), (0, good[0].int(), TypeError),
                      (1, good[1].float(), TypeError), (2, good[2][:1], ValueError), (3, good[3][..., :8], ValueError),
                      (0, good[0][0], ValueError), (0, good[0][..., ::2], ValueError)):
        bad = list(good)
        bad[i] = t
        with pytest.raises(err):
            hr.KV4Cache(*bad)
    for kw in (dict(page=24), dict(page=8), dict(dim=96), dict(groups=4)):
        with pytest.raises(ValueError):
            hr.KV4Cache(*_tensors(**kw))
    with pytest.raises(ValueError, match="signs"):
        hr.KV4Cache(*good, rotate=False, signs=torch.ones(64, dtype=torch.int8))
    with pytest.raises(TypeError):
        hr.KV4Cache(*good, signs=torch.ones(64))
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: hr.kv4_append(good, x, x, torch.zeros(3, dtype=torch.int64)),
                 lambda: hr.kv4_read(None, torch.zeros(3, dtype=torch.int64)),
                 lambda: hr.kv4_attention(good[0], x, x, x)):
        with pytest.raises(TypeError):
            call()


class _Stub(hr.KV4Cache):
    """A cache object without a GPU, for the checks that come before any pointer is taken."""

    def __init__(self):
        self.pages, self.heads, self.page, self.dim, self.group, self.rotate = 2, 2, 16, 64, 64, True
        self.device = torch.device("cuda:0")
        self._index, self._ref = 0, None


def test_binding_argument_checks():
    c = _Stub()
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    for k, v, s, err in ((x.double(), x, slots, TypeError), (x, x.float(), slots, TypeError),
                         (x[:, :1], x, slots, ValueError), (x[..., :32], x, slots, ValueError),
                         (x, x[:2], slots, ValueError), (x, x, slots.int(), TypeError), (x, x, slots[:2], ValueError),
                         (x, x, None, TypeError), (x.transpose(0, 1)[:2].contiguous().transpose(0, 1), x, slots, ValueError),
                         (torch.zeros((3, 132), dtype=torch.bfloat16)[:, :128].view(3, 2, 64), x, slots, ValueError),
                         (torch.zeros((1, 2, 64), dtype=torch.bfloat16).expand(3, 2, 64), x, slots, ValueError)):
        with pytest.raises(err):
            hr.kv4_append(c, k, v, s)
    with pytest.raises(TypeError):
        hr.kv4_read(c, slots, dtype=torch.int8)
    with pytest.raises(ValueError):
        hr.kv4_read(c, slots, k=x[:2])
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((3, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for kw, err in ((dict(q=q[:, :3]), ValueError), (dict(table=table.long()), TypeError), (dict(table=table[0]), ValueError),
                    (dict(lens=lens[:2]), ValueError), (dict(starts=lens), ValueError), (dict(out=q.float()), TypeError),
                    (dict(workspace=lens), TypeError), (dict(table=table[:, ::2]), ValueError)):
        a = dict(q=q, table=table, lens=lens)
        a.update(kw)
        with pytest.raises(err):
            hr.kv4_attention(c, **a)
    with pytest.raises(ValueError, match="GPU"):
        hr.kv4_attention(c, q, table, lens, out=q)


@pytest.mark.parametrize("name,value,err", [
    (name, value, err) for name, bits in (("window", 31), ("max_new", 31), ("max_len", 63))
    for value, err in ((2 ** (bits + 1) + 5, ValueError), (2 ** (bits + 1), ValueError), (2 ** bits, ValueError),
                       (-1, ValueError), (1.5, TypeError), ("1", TypeError))])
def test_binding_integer_ranges(name, value, err):
    """Sizes past the C types are refused, not cut to them."""
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((3, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(err, match=name):
        hr.kv4_attention(_Stub(), q, table, lens, **{name: value})


def test_workspace_of_sizes_the_call_refuses():
    f = hr.lib.hr_kv4_attention_workspace
    top32, top64 = 2 ** 31 - 1, 2 ** 63 - 1
    for bad in ((1, 128, 1, 1 << 62, 1, 1, 1, 1 << 30, 0), (1, 128, 1, 1, 1, 1, 1, top64, 0),
                (top32, 128, 1, 1, top32, top32, top32, 1 << 20, 0), (1, top32, 1, 1, 1, 1, 1, 1 << 20, 0),
                (1, 128, 1, 1, 1, 1, top32, 1 << 20, 0), (1, 128, 7, 1, 1, 1, 1, 1 << 20, 0),
                (2, 128, 1, 1, 1, 3, 1, 1 << 20, 0)):
        assert f(*bad) == 0


def test_attention_width_past_32_bits():
    assert _attend(width=1 << 31) == hr.HR_EUNSUPPORTED
    assert _attend(width=1 << 62) == hr.HR_EUNSUPPORTED


def test_attention_query_heads_past_32_bits_of_elements():
    f = hr.lib.hr_kv4_attention_workspace
    for q_heads in (1 << 23, 1 << 26):
        assert _attend(q_heads=q_heads, qs=q_heads * 128, total=1, batch=1) == hr.HR_EUNSUPPORTED
        assert f(2, 128, hr.HR_BF16, 1, 1, q_heads, 1, 1 << 20, 0) == 0


# ------------------------------------------------------------------ the oracle

def test_oracle_rotation_is_orthogonal():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 64))
    s = (rng.integers(0, 2, 64) * 2 - 1).astype(np.int8)
    y = oracle.kv4.rotate(x, s)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    assert np.allclose(oracle.kv4.unrotate(y, s), x)


def test_oracle_attention_by_hand():
    """Two tokens, one head: the softmax of two scores, the causal row and the empty row."""
    vals = np.zeros((1, 1, 16, 64))
    vals[0, 0, 0, 0], vals[0, 0, 1, 1] = 1.0, 1.0
    q = np.zeros((3, 1, 64))
    q[:, 0, 1] = 2.0
    out = oracle.kv4.attention(q, vals, vals, [[0]], [2], [0, 3], 0.5, rotated=False)
    assert not out[0].any()                       # position -1 sees nothing
    assert np.allclose(out[1, 0, :2], [1.0, 0.0])
    e = np.exp(1.0)
    assert np.allclose(out[2, 0, :2], [1 / (1 + e), e / (1 + e)])


def test_oracle_rotated_attention_is_attention_on_unrotated_values():
    rng = np.random.default_rng(2)
    s = (rng.integers(0, 2, 64) * 2 - 1).astype(np.int8)
    k, v = rng.standard_normal((2, 2, 2, 16, 64))
    q = rng.standard_normal((4, 6, 64))
    args = ([[1, 0]], [20], [0, 4], 0.1)
    a = oracle.kv4.attention(q, k, v, *args, signs=s, rotated=True, window=7)
    b = oracle.kv4.attention(q, oracle.kv4.unrotate(k, s), oracle.kv4.unrotate(v, s), *args, rotated=False, window=7)
    assert np.allclose(a, b)


def test_oracle_values_undo_quantize():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 3, 16, 128)).astype(np.float32)
    q, s = oracle.kv4.quantize_plain(x, 32)
    codes = oracle.quant.pack_int4(q.reshape(-1, 128)).reshape(2, 3, 16, 64)
    back = oracle.kv4.values(codes, np.swapaxes(s, -1, -2))
    step = np.repeat(s.astype(np.float64), 32, -1)
    assert (np.abs(back - x) <= 0.5 * step * (1 + 1e-2)).all()
