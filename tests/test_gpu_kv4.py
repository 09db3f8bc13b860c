"""The 4-bit key/value cache on the GPU against the fp64 oracle: quantizing as it
is written, reading back, and attention over it.

Attention tolerances, relative 2-norm against fp64 on the same codes and scales.
The output's own rounding is 2^-9 / sqrt(3) = 1.1e-3 (bf16) or 2^-12 / sqrt(3) =
1.4e-4 (fp16) rms times at most sqrt(2) for where values fall in their binade.
16-bit queries, probabilities and scaled values are each rounded to fp16, 1.4e-4
rms apiece, the queries' error entering through scores whose sum of squares of
products stays within a few units here: 4e-4 together.  Allowed: 2^-8 (bf16),
2^-10 (fp16).  fp32 keeps products to 2^-24 and scores of size 2^4 to 2^-20 in
the exponent: 2^-17 allowed.  No element may be off by more than 32 times that
of max(its size, the rms).
"""
import numpy as np
import pytest
import torch

import hadamard_rotation_int4_amd as hr
import oracle
from parity import check_quant

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TOL = {"bf16": 2.0 ** -8, "f16": 2.0 ** -10, "f32": 2.0 ** -17}


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _signs(rng, dim):
    return (rng.integers(0, 2, dim) * 2 - 1).astype(np.int8)


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _num(t):
    return t.detach().float().cpu().numpy() if t.dtype == torch.bfloat16 else t.detach().cpu().numpy()


def _vectors(codes, scales, slots, page):
    """Codes [tokens][heads][dim/2] and scales [tokens][heads][groups] at slots."""
    return codes[slots // page, :, slots % page], scales[slots // page, :, :, slots % page]


def _close(got, want, tol):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    assert got.shape == want.shape
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    err, want = (got - want)[~nan], want[~nan]
    if not want.size:
        return
    rms = np.sqrt(np.mean(want * want))
    rel = np.sqrt(np.mean(err * err)) / rms if rms else np.abs(err).max()
    assert rel <= tol, f"relative error {rel:.3g} > {tol:.3g}"
    worst = (np.abs(err) / np.maximum(np.abs(want), max(rms, 1e-30))).max() if rms else np.abs(err).max()
    assert worst <= 32 * tol, f"one element {worst:.3g} off"


# ------------------------------------------------------------------ write and read

@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64),
                                       (256, 128), (256, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rotate,signed", [(False, False), (True, False), (True, True)])
def test_append_and_read(dim, group, dtype, rotate, signed):
    rng = _rng(dim * 1000 + group + len(dtype))
    heads, page, pages, tokens = 3, 16, 9, 77
    signs = _signs(rng, dim) if signed else None
    cache = hr.kv4_cache(pages, heads, dim, page, group, rotate, None if signs is None else _t(signs))
    # keys and values side by side, tokens strided, a few wide channels
    kv = rng.standard_normal((tokens, 2 * heads * dim + 8)) * np.where(rng.random(2 * heads * dim + 8) < 0.02, 20, 1)
    kv = _t(kv.astype(np.float32)).to(TYPES[dtype])
    k = kv[:, :heads * dim].view(tokens, heads, dim)
    v = kv[:, heads * dim:2 * heads * dim].view(tokens, heads, dim)
    slots = rng.permutation(pages * page)[:tokens]
    slots[5], slots[40] = -1, pages * page            # neither is written
    hr.kv4_append(cache, k, v, _t(slots))
    torch.cuda.synchronize()
    keep = np.array([t for t in range(tokens) if t not in (5, 40)])
    for x, codes, scales in ((k, cache.k_codes, cache.k_scales), (v, cache.v_codes, cache.v_scales)):
        x = _num(x.contiguous())
        c, s = _vectors(codes.cpu().numpy(), scales.cpu().numpy(), slots[keep], page)
        if rotate:
            y = oracle.kv4.rotate(x[keep], signs)
            check_quant(c.reshape(-1, dim // 2), s.reshape(-1, dim // group), y.reshape(-1, dim), group)
        else:
            q, want = oracle.kv4.quantize_plain(x[keep], group)
            assert np.array_equal(s.view(np.uint16), want.view(np.uint16))
            assert np.array_equal(oracle.quant.unpack_int4(c.reshape(-1, dim // 2)).reshape(q.shape), q)
        # nothing else was touched
        rest = np.setdiff1d(np.arange(pages * page), slots[keep])
        c, s = _vectors(codes.cpu().numpy(), scales.cpu().numpy(), rest, page)
        assert not c.any() and not s.any()
    # read back what is there
    for out in TYPES:
        gk, gv = hr.kv4_read(cache, _t(slots), dtype=TYPES[out])
        for got, codes, scales in ((gk, cache.k_codes, cache.k_scales), (gv, cache.v_codes, cache.v_scales)):
            vals = oracle.kv4.values(codes.cpu().numpy(), scales.cpu().numpy())
            want = vals[slots[keep] // page, :, slots[keep] % page]
            if rotate:
                want = oracle.kv4.unrotate(want, signs)
            got = _num(got)
            assert not got[[5, 40]].any()
            got = got[keep].astype(np.float64)
            # one rounding to the type, and fp32 sums of dim terms (8 levels, 2^-24 each) with the rotation
            u = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}[out]
            room = 16 * 2.0 ** -24 * np.sqrt((want ** 2).sum(-1, keepdims=True)) if rotate else 0.0
            assert (np.abs(got - want) <= u * np.abs(want) + room + 2.0 ** -24).all()


@pytest.mark.parametrize("tokens", [0, 1, 2, 15, 16, 17, 300])
@pytest.mark.parametrize("page", [16, 256])
def test_append_lengths(tokens, page):
    rng = _rng(tokens + page)
    heads, dim = 5, 128
    signs = _signs(rng, dim)
    cache = hr.kv4_cache(320 // min(page, 32) + 2, heads, dim, page, None, True, _t(signs))
    x = _t(rng.standard_normal((2, tokens, heads, dim)).astype(np.float32)).to(torch.bfloat16)
    slots = rng.permutation(300)[:tokens].astype(np.int64)
    hr.kv4_append(cache, x[0], x[1], _t(slots))
    c, s = _vectors(cache.v_codes.cpu().numpy(), cache.v_scales.cpu().numpy(), slots, page)
    if tokens:
        check_quant(c.reshape(-1, 64), s.reshape(-1, 1), oracle.kv4.rotate(_num(x[1]), signs).reshape(-1, dim), dim)
    k, v = hr.kv4_read(cache, _t(slots))
    assert k.shape == v.shape == (tokens, heads, dim)


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_values_that_are_not_finite(rotate, dtype):
    """A NaN, an infinity or (fp32) a scale past 9352 poisons its (token, head), key and value, and no other."""
    rng = _rng(8)
    heads, dim, group, tokens = 2, 128, 32, 12
    cache = hr.kv4_cache(2, heads, dim, 16, group, rotate)
    x = rng.standard_normal((2, tokens, heads, dim)).astype(np.float32)
    x[0, 1, 0, 100] = np.nan
    x[1, 3, 1, 0] = np.inf
    x[0, 5, 0, 127] = -np.inf
    bad = {(1, 0), (3, 1), (5, 0)}
    if dtype == "f32":
        x[1, 7, 1] *= 1e8
        bad.add((7, 1))
    x[:, 9] = 0.0                                     # an all-zero vector is fine
    x = _t(x).to(TYPES[dtype])
    hr.kv4_append(cache, x[0], x[1], torch.arange(tokens, device=DEV))
    for y in hr.kv4_read(cache, torch.arange(tokens, device=DEV), dtype=torch.float32):
        y = y.cpu().numpy()
        for t in range(tokens):
            for h in range(heads):
                assert np.isnan(y[t, h]).all() if (t, h) in bad else np.isfinite(y[t, h]).all()
        assert not y[9].any()
    codes = cache.k_codes.cpu().numpy()
    for t, h in bad:
        assert not codes[0, h, t].any()


def test_small_and_large_scales():
    """Scales in fp16's subnormal range and at its top, without a rotation: equal to the oracle's."""
    rng = _rng(9)
    x = rng.standard_normal((2, 40, 1, 64)).astype(np.float32) * (10.0 ** rng.uniform(-8, 5, (2, 40, 1, 1))).astype(np.float32)
    cache = hr.kv4_cache(3, 1, 64, 16, 32, rotate=False)
    hr.kv4_append(cache, _t(x[0]), _t(x[1]), torch.arange(40, device=DEV))
    for i, (codes, scales) in enumerate(((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))):
        c, s = _vectors(codes.cpu().numpy(), scales.cpu().numpy(), np.arange(40), 16)
        q, want = oracle.kv4.quantize_plain(x[i], 32)
        # a poisoned key poisons the value too: compare where both sides of the token are finite
        fine = np.isfinite(oracle.kv4.quantize_plain(x[0], 32)[1]).all(-1) & np.isfinite(
            oracle.kv4.quantize_plain(x[1], 32)[1]).all(-1)
        assert fine.sum() > 20
        assert np.array_equal(s[fine].view(np.uint16), want[fine].view(np.uint16))
        assert np.array_equal(oracle.quant.unpack_int4(c.reshape(-1, 32)).reshape(q.shape)[fine], q[fine])
        assert np.isnan(s[~fine].astype(np.float32)).all()


# ------------------------------------------------------------------ attention

class Filled:
    """A cache whose sequences' tokens hold near-Gaussian vectors.  Every slot that belongs to no sequence holds
    the worst there is: any bits in its codes, NaN and infinite scales."""

    def __init__(self, rng, lens, heads, dim, group, page, rotate, signed=True, size=1.0):
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + 3
        order = rng.permutation(self.pages)
        self.width = max(max(need, default=0) + 2, 1)
        self.table = np.full((len(lens), self.width), -7, dtype=np.int32)
        self.lens = np.asarray(lens, dtype=np.int32)
        at = 0
        codes = rng.integers(0, 256, (2, self.pages, heads, page, dim // 2)).astype(np.uint8)
        scales = rng.choice(np.array([np.nan, np.inf, -np.inf, 6e4, 0.0], dtype=np.float16),
                            (2, self.pages, heads, dim // group, page))
        for b, n in enumerate(lens):
            ids = order[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = ids
            if not n:
                continue
            j = np.arange(n)
            for kv in range(2):
                y = rng.standard_normal((n, heads, dim)) * np.exp(0.3 * rng.standard_normal((n, heads, 1))) * size
                q, s = oracle.kv4.quantize_plain(y.astype(np.float32), group)
                c = oracle.quant.pack_int4(q.reshape(-1, dim)).reshape(n, heads, dim // 2)
                codes[kv][ids[j // page], :, j % page] = c
                scales[kv][ids[j // page], :, :, j % page] = s
        self.codes, self.scales = codes, scales
        self.signs = _signs(rng, dim) if rotate and signed else None
        self.rotate, self.heads, self.dim, self.page = rotate, heads, dim, page
        self.cache = hr.KV4Cache(_t(codes[0]), _t(scales[0]), _t(codes[1]), _t(scales[1]), rotate=rotate,
                                 signs=None if self.signs is None else _t(self.signs))

    def want(self, q, starts, scale=None, causal=True, window=0):
        kv = [oracle.kv4.values(self.codes[i], self.scales[i]) for i in range(2)]
        return oracle.kv4.attention(q, kv[0], kv[1], self.table, self.lens, starts,
                                    self.dim ** -0.5 if scale is None else scale, self.signs, self.rotate, causal,
                                    window)


def _attend(f, rng, news, q_heads, dtype, causal=True, window=0, scale=None, max_len=None, extra=0):
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    total = int(starts[-1])
    qkv = _t(rng.standard_normal((total, q_heads * f.dim + extra)).astype(np.float32)).to(TYPES[dtype])
    q = qkv[:, :q_heads * f.dim].view(total, q_heads, f.dim)
    out = hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), starts=_t(starts), max_new=max(news, default=0),
                           max_len=max_len, causal=causal, window=window, scale=scale)
    assert out.dtype == q.dtype and out.shape == q.shape
    _close(_num(out), f.want(_num(q.contiguous()), starts, scale, causal, window), TOL[dtype])
    return out, q, starts


@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 128),
                                       (256, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rotate", [False, True])
def test_decode_types(dim, group, dtype, rotate):
    rng = _rng(dim + group)
    f = Filled(rng, [300, 1, 0, 47], 2, dim, group, 32, rotate)
    _attend(f, rng, [1] * 4, 6, dtype, extra=16)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 700, 1025])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_lengths(n, page):
    rng = _rng(n)
    f = Filled(rng, [n, max(1, n - 1)], 3, 128, 128, page, True)
    _attend(f, rng, [1, 1], 3 * 4, "bf16")
    _attend(f, rng, [1, 1], 3 * 4, "f16", max_len=n)


@pytest.mark.parametrize("rep", [1, 2, 3, 5, 8, 16, 17, 33])
def test_decode_heads(rep):
    rng = _rng(rep)
    f = Filled(rng, [90, 260], 2, 64, 64, 16, True)
    _attend(f, rng, [1, 1], 2 * rep, "f16")


@pytest.mark.parametrize("news", [[2, 3, 1], [5, 5, 5], [16, 1, 33], [40, 64, 20], [1, 0, 7], [130, 200, 129]])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,group,dtype", [(128, 128, "bf16"), (64, 32, "f16"), (128, 64, "f32"), (256, 64, "bf16")])
def test_several_new_tokens(news, causal, dim, group, dtype):
    rng = _rng(sum(news))
    lens = [max(news[0], 65), max(news[1], 200), max(news[2], 131)]
    f = Filled(rng, lens, 2, dim, group, 32, True)
    _attend(f, rng, news, 4, dtype, causal=causal)


@pytest.mark.parametrize("dim,group", [(64, 64), (64, 32), (128, 128), (128, 64)])
def test_fp16_prompt(dim, group):
    """Enough rows of two sequences to fill the chip 32 at a time; the first in two parts."""
    rng = _rng(dim + group)
    f = Filled(rng, [700, 290], 8, dim, group, 32, True)
    _attend(f, rng, [255, 131], 32, "f16")
    _attend(f, rng, [390, 131], 32, "f16")


@pytest.mark.parametrize("lens,news", [([3, 0, 40], [10, 4, 40]), ([1], [33]), ([100], [160])])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing(lens, news, dtype):
    """More new rows than cached tokens: the first rows' positions are negative, their outputs zero."""
    rng = _rng(3)
    f = Filled(rng, lens, 1, 128, 128, 16, True)
    out, _, starts = _attend(f, rng, news, 4, dtype)
    assert not _num(out)[:max(0, news[0] - lens[0])].any()


@pytest.mark.parametrize("window", [1, 2, 31, 64, 100, 5000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("news", [[1, 1], [9, 50], [70, 150]])
def test_window(window, causal, news):
    rng = _rng(window)
    f = Filled(rng, [400, 150], 2, 64, 64, 16, True)
    _attend(f, rng, news, 8, "bf16", causal=causal, window=window)


@pytest.mark.parametrize("batch,heads,n", [(1, 1, 5000), (1, 2, 9999), (3, 1, 2500)])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f32", 64), ("f16", 256)])
def test_decode_split_over_the_tokens(batch, heads, n, dtype, dim):
    rng = _rng(n)
    f = Filled(rng, [n - 700 * b for b in range(batch)], heads, dim, dim, 64, True)
    out, q, starts = _attend(f, rng, [1] * batch, heads * 4, dtype)
    # the same again, and with bounds that are too small or far too large
    again = hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), starts=_t(starts))
    assert torch.equal(out, again)
    for bound in (0, 100, 1 << 20):
        other = hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), max_len=bound)
        _close(_num(other), f.want(_num(q.contiguous()), starts), TOL[dtype])


@pytest.mark.parametrize("news", [1, 3, 150])
def test_poisoned_token(news):
    """A token that is not finite reaches the rows that see it, and only those."""
    rng = _rng(4)
    f = Filled(rng, [200], 2, 128, 128, 16, True)
    for h, j in ((0, 199), (1, 170)):
        page, place = f.table[0, j // 16], j % 16
        for kv, t in ((0, f.cache.k_scales), (1, f.cache.v_scales)):
            t[page, h, :, place] = float("nan")
            f.scales[kv][page, h, :, place] = np.nan
        for kv, t in ((0, f.cache.k_codes), (1, f.cache.v_codes)):
            t[page, h, place] = 0
            f.codes[kv][page, h, place] = 0
    out, _, _ = _attend(f, rng, [news], 4, "bf16")
    out = _num(out)
    assert np.isnan(out[-1]).all()
    if news == 150:
        assert np.isfinite(out[:100]).all()


@pytest.mark.parametrize("size,scale", [(1e-3, 1.0), (30.0, 0.0883883), (1.0, 3.0), (1000.0, 1e-5)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sizes_of_keys_and_scores(size, scale, dtype):
    """Tiny and large keys and values; scores from near equal to one token taking all."""
    rng = _rng(5)
    f = Filled(rng, [333], 2, 128, 128, 64, True, size=size)
    if size * scale > 2:      # a score's own rounding (2^-12 of its terms) moves the softmax of scores this large
        starts = np.array([0, 1], dtype=np.int32)
        q = _t(rng.standard_normal((1, 8, 128)).astype(np.float32)).to(TYPES[dtype])
        out = hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), scale=scale)
        want = f.want(_num(q), starts, scale)
        terms = scale * size * 128 * 4
        _close(_num(out), want, TOL[dtype] + terms * (2.0 ** -12 if dtype != "f32" else 2.0 ** -23) / 8)
    else:
        _attend(f, rng, [1], 8, dtype, scale=scale)


@pytest.mark.parametrize("qsize", [1e-30, 1e-6, 1e4, 1e30])
def test_sizes_of_queries(qsize):
    """bf16 queries far outside fp16's range (the scale undoes it)."""
    rng = _rng(6)
    f = Filled(rng, [100], 1, 128, 128, 64, True)
    q = _t((rng.standard_normal((1, 4, 128)) * qsize).astype(np.float32)).to(torch.bfloat16)
    out = hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), scale=0.088 / qsize)
    _close(_num(out), f.want(_num(q), np.array([0, 1]), 0.088 / qsize), TOL["bf16"])


# A max_len far above the sequences' lengths makes a call's work look large: many rows then take the form for prompts
# whatever their number of tokens.
FAR = 1 << 20


@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 128),
                                       (256, 256)])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("news", [[70], [40, 64, 20], [130, 200, 129], [1, 0, 97]])
def test_prompt_types(dim, group, rotate, news):
    rng = _rng(dim + group + len(news))
    f = Filled(rng, [n + int(rng.integers(0, 300)) for n in news], 2, dim, group, 16, rotate)
    _attend(f, rng, news, 4, "bf16", max_len=FAR, extra=64)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 31, 64, 100, 5000])
@pytest.mark.parametrize("dim,rep", [(128, 3), (64, 1), (128, 17)])
def test_prompt_masks(causal, window, dim, rep):
    rng = _rng(window + rep)
    f = Filled(rng, [150, 333, 90], 2, dim, dim, 64, True)
    _attend(f, rng, [70, 150, 90], 2 * rep, "bf16", causal, window, max_len=FAR)


@pytest.mark.parametrize("lens,news", [([3, 0, 40], [80, 90, 40]), ([33], [133]), ([100], [160])])
def test_prompt_rows_that_see_nothing(lens, news):
    rng = _rng(12)
    f = Filled(rng, lens, 2, 128, 64, 16, True)
    out, _, starts = _attend(f, rng, news, 4, "bf16", max_len=FAR)
    for b, n in enumerate(lens):
        if news[b] > n:
            assert not _num(out)[starts[b]:starts[b] + news[b] - n].any()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_poisoned_token(dim):
    rng = _rng(13)
    f = Filled(rng, [200], 2, dim, dim, 16, True)
    place = f.table[0, 170 // 16], 1, slice(None), 170 % 16
    for kv, t in ((0, f.cache.k_scales), (1, f.cache.v_scales)):
        t[place] = float("nan")
        f.scales[kv][place] = np.nan
    out, _, _ = _attend(f, rng, [150], 4, "bf16", max_len=FAR)
    out = _num(out)
    assert np.isnan(out[-1, 2:]).all() and np.isfinite(out[:, :2]).all() and np.isfinite(out[:120]).all()


@pytest.mark.parametrize("dim,batch,news,n", [(128, 1, 600, 3600), (64, 2, 300, 2000), (256, 1, 600, 4200),
                                              (128, 9, 24, 2500)])
def test_prompt_split_over_the_tokens(dim, batch, news, n):
    rng = _rng(14)
    f = Filled(rng, [n - 7 * b for b in range(batch)], 2, dim, dim, 64, True)
    _attend(f, rng, [news] * batch, 8, "bf16")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("news", [40, 150])
def test_prompt_rows_of_different_sizes(dim, news):
    """Rows side by side whose queries lie within fp16's range, above it and below it."""
    rng = _rng(8)
    f = Filled(rng, [news + 60], 2, dim, dim, 16, True, size=1e-6)
    q = rng.standard_normal((news, 4, dim)) * rng.choice([1e6, 1.0, 1e-6, 0.0], (news, 4, 1))
    q = _t(q.astype(np.float32)).to(torch.bfloat16)
    starts = np.array([0, news], dtype=np.int32)
    for bound in (None, FAR):
        out = hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), starts=_t(starts), max_new=news, max_len=bound)
        _close(_num(out), f.want(_num(q), starts), TOL["bf16"])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("side", [-1, 1])
@pytest.mark.parametrize("news", [1, 40, 150])
def test_running_maximum_far_from_zero(dim, side, news):
    """All scores of a row near -150 or 150 (in log2 units, 128 dims): only their differences count.  Keys are
    multiples of their scale, 1/2, so fp16 holds them; what rounding the queries does is alike for all tokens but for
    2^-12 / sqrt(3) of 3 times the 0.4 by which keys differ, 2e-4; fp32 sums of 2^7 are good to 2^-16."""
    rng = _rng(9)
    n, heads, page = news + 90, 2, 16
    base = rng.choice([-1.0, 1.0], (1, heads, dim))
    k = base * rng.choice([2.5, 3.0, 3.5], (n, heads, dim))
    v = rng.standard_normal((n, heads, dim))
    pages = -(-n // page)
    cache = hr.kv4_cache(pages, heads, dim, page, dim, rotate=False)
    at = [_t(x.astype(np.float32)).to(torch.bfloat16) for x in (k, v)]
    hr.kv4_append(cache, at[0], at[1], torch.arange(n, device=DEV))
    vals = [oracle.kv4.values(_num(c), _num(s)) for c, s in ((cache.k_codes, cache.k_scales),
                                                             (cache.v_codes, cache.v_scales))]
    assert np.array_equal(vals[0].transpose(0, 2, 1, 3).reshape(-1, heads, dim)[:n], k)
    q = 3 * side * np.repeat(base, 2, 1) + 0.3 * rng.standard_normal((news, 2 * heads, dim))
    q = _t(q.astype(np.float32)).to(torch.bfloat16)
    table, lens = np.arange(pages, dtype=np.int32)[None], np.array([n], dtype=np.int32)
    starts = np.array([0, news], dtype=np.int32)
    want = oracle.kv4.attention(_num(q), vals[0], vals[1], table, lens, starts, dim ** -0.5, None, False, True, 0)
    for bound in (None, FAR):
        out = hr.kv4_attention(cache, q, _t(table), _t(lens), starts=_t(starts), max_new=news, max_len=bound)
        _close(_num(out), want, TOL["bf16"])


def test_append_then_attend_end_to_end():
    """Attention over what append wrote is near attention over the keys and values themselves."""
    rng = _rng(7)
    heads, dim, page, n = 2, 128, 32, 400
    signs = _signs(rng, dim)
    cache = hr.kv4_cache(20, heads, dim, page, 32, True, _t(signs))
    kv = _t(rng.standard_normal((2, n, heads, dim)).astype(np.float32)).to(torch.bfloat16)
    table = torch.randperm(20, device=DEV).to(torch.int32)[:-(-n // page)].view(1, -1)
    j = torch.arange(n, device=DEV)
    slots = table[0].long()[j // page] * page + j % page
    hr.kv4_append(cache, kv[0, :390], kv[1, :390], slots[:390].contiguous())
    hr.kv4_append(cache, kv[0, 390:], kv[1, 390:], slots[390:].contiguous())
    q = _t(rng.standard_normal((1, 8, dim)).astype(np.float32)).to(torch.bfloat16)
    out = _num(hr.kv4_attention(cache, q, table.contiguous(), torch.tensor([n], dtype=torch.int32, device=DEV)))
    k, v = kv.double().cpu().numpy()
    z = np.einsum("hd,nhd->hn", _num(q)[0].astype(np.float64), np.repeat(k, 4, 1)) / np.sqrt(dim)
    p = np.exp(z - z.max(-1, keepdims=True))
    want = np.einsum("hn,nhd->hd", p / p.sum(-1, keepdims=True), np.repeat(v, 4, 1))
    # a group of 32 normal values has absmax 2.1: steps of 0.3, errors of 0.087 rms in keys and values, scores off
    # by 0.087 rms; both move the output by under 0.13 of its size
    assert np.linalg.norm(out[0] - want) <= 0.2 * np.linalg.norm(want)


def test_cache_above_4_gib():
    """Offsets that pass 32 bits: the last pages of a cache whose codes are over 4 GiB each."""
    rng = _rng(11)
    heads, dim, page = 8, 128, 64
    pages = (1 << 32) // (heads * page * dim // 2) + 40
    codes = torch.zeros((2, pages, heads, page, dim // 2), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((2, pages, heads, 1, page), dtype=torch.float16, device=DEV)
    cache = hr.KV4Cache(codes[0], scales[0], codes[1], scales[1])
    n = 150
    ids = np.array([pages - 1, pages - 7, pages - 30])
    j = np.arange(n)
    slots = ids[j // page] * page + j % page
    kv = _t(rng.standard_normal((2, n, heads, dim)).astype(np.float32)).to(torch.bfloat16)
    hr.kv4_append(cache, kv[0], kv[1], _t(slots))
    k, v = hr.kv4_read(cache, _t(slots), dtype=torch.float32)
    for got, x in ((k, kv[0]), (v, kv[1])):
        assert (torch.linalg.norm(got - x.float()) <= 0.2 * torch.linalg.norm(x.float())).item()
    vals = [oracle.kv4.values(codes[i][_t(ids)].cpu().numpy(), scales[i][_t(ids)].cpu().numpy()) for i in range(2)]
    q = _t(rng.standard_normal((2, heads, dim)).astype(np.float32)).to(torch.bfloat16)
    out = hr.kv4_attention(cache, q, _t(ids.astype(np.int32).reshape(1, -1)),
                           torch.tensor([n], dtype=torch.int32, device=DEV), max_new=2)
    want = oracle.kv4.attention(_num(q), vals[0], vals[1], np.array([[0, 1, 2]]), [n], [0, 2], dim ** -0.5)
    _close(_num(out), want, TOL["bf16"])


def test_other_stream_and_graph():
    """On a stream of its own, and captured: every replay equals the eager result, with eager work in between."""
    rng = _rng(12)
    f = Filled(rng, [3000, 1200], 2, 128, 128, 64, True)
    table, lens = _t(f.table), _t(f.lens)
    q = _t(rng.standard_normal((2, 8, 128)).astype(np.float32)).to(torch.bfloat16)
    want = hr.kv4_attention(f.cache, q, table, lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = hr.kv4_attention(f.cache, q, table, lens)
    side.synchronize()
    assert torch.equal(got, want)
    spare = hr.kv4_cache(2, 2, 128)
    x = _t(rng.standard_normal((2, 1, 2, 128)).astype(np.float32)).to(torch.bfloat16)
    slot = torch.tensor([70], device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hr.kv4_append(spare, x[0], x[1], slot)
        captured = hr.kv4_attention(f.cache, q, table, lens)
    for n in range(4):
        captured.zero_()
        spare.k_codes.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, want)
        assert spare.k_codes[1, :, 6].any()
        assert torch.equal(hr.kv4_attention(f.cache, q, table, lens), want)


def test_rows_of_no_sequence_are_left():
    rng = _rng(13)
    for n in (100, 4000):                 # one part, several parts
        f = Filled(rng, [n], 1, 128, 128, 64, True)
        q = _t(rng.standard_normal((6, 4, 128)).astype(np.float32)).to(torch.bfloat16)
        out = torch.full_like(q, 7.0)
        hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), starts=torch.tensor([2, 4], dtype=torch.int32, device=DEV),
                         max_new=2, out=out)
        assert (out[:2] == 7.0).all() and (out[4:] == 7.0).all()
        want = f.want(_num(q)[2:4], np.array([0, 2]))
        _close(_num(out)[2:4], want, TOL["bf16"])


def test_example_layer():
    """The example: W4A4 projections, cache and attention together, prompt and single tokens.  W4A4 products of
    Gaussian rows with groups of 128 are 0.16 off fp32 each (steps of 0.4 of the deviation: 0.116 rms an operand);
    three of them in a row and 4-bit keys and values stay under 0.5, where unrelated outputs are 1.4 off."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "kv4_decode.py")
    spec = importlib.util.spec_from_file_location("kv4_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    prompt, single, _, held = mod.run(batch=3, prompt=150, steps=5)
    assert prompt <= 0.5 and single <= 0.5
    assert held == 2 * 8 * 66


def test_more_rows_than_max_new():
    """Rows past max_new may be left, but nothing wrong is written, and nothing beyond the sequence's rows."""
    rng = _rng(14)
    for n in (100, 4000):
        f = Filled(rng, [n], 1, 128, 128, 64, True)
        q = _t(rng.standard_normal((40, 4, 128)).astype(np.float32)).to(torch.bfloat16)
        out = torch.full((40, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), starts=torch.tensor([0, 30], dtype=torch.int32, device=DEV),
                         max_new=1, out=out)
        assert (out[30:] == 7.0).all()
        want = f.want(_num(q)[:30], np.array([0, 30]))
        got = _num(out)[:30]
        done = ~(got == 7.0).all((1, 2))
        assert done[0]
        _close(got[done], want[done], TOL["bf16"])
