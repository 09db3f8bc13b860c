"""The 4-bit key/value cache on the GPU where the other tests of it do not reach: masks and arguments at the ends of
their ranges, softmax weights and values far apart, and every form of the attention kernels over many tokens.

Tolerances are those of test_gpu_kv4.py, whose oracle and comparison are used here too; what a test allows beyond them
is derived in its docstring.
"""
import numpy as np
import pytest
import torch

import hadamard_rotation_int4_amd as hr
import oracle
from test_gpu_kv4 import DEV, FAR, TOL, TYPES, Filled, _attend, _close, _num, _rng, _t

pytestmark = pytest.mark.gpu


class Held:
    """A cache (one sequence, pages in any order) that holds the given keys and values, fp32 [tokens][heads][dim],
    quantized without a rotation."""

    def __init__(self, rng, k, v, group, page):
        n, heads, dim = k.shape
        pages = -(-n // page)
        self.table = rng.permutation(pages).astype(np.int32)[None]
        self.lens = np.array([n], dtype=np.int32)
        self.heads, self.dim = heads, dim
        j = np.arange(n)
        at = self.table[0, j // page], slice(None), j % page
        parts, self.vals = [], []
        for x in (k, v):
            q, s = oracle.kv4.quantize_plain(x.astype(np.float32), group)
            codes = np.zeros((pages, heads, page, dim // 2), dtype=np.uint8)
            scales = np.zeros((pages, heads, dim // group, page), dtype=np.float16)
            codes[at] = oracle.quant.pack_int4(q.reshape(-1, dim)).reshape(n, heads, dim // 2)
            scales[self.table[0, j // page], :, :, j % page] = s
            parts += [_t(codes), _t(scales)]
            self.vals.append(oracle.kv4.values(codes, scales))
        self.cache = hr.KV4Cache(*parts, rotate=False)

    def attend(self, q, **kw):
        """(got, want) of the last q.shape[0] tokens' queries."""
        starts = np.array([0, len(q)], dtype=np.int32)
        out = hr.kv4_attention(self.cache, q, _t(self.table), _t(self.lens), starts=_t(starts), max_new=len(q), **kw)
        kw.pop("max_len", None)
        scale = kw.pop("scale", self.dim ** -0.5)
        return _num(out), dense(_num(q), *self.vals, self.table, self.lens, starts, scale, None, False, **kw)


def dense(q, kvals, vvals, table, lens, starts, scale, signs=None, rotated=True, causal=True, window=0):
    """oracle.kv4.attention with whole matrices of scores, for many rows (finite values only)."""
    q = np.asarray(q, dtype=np.float64)
    rep = q.shape[1] // kvals.shape[1]
    qr = oracle.kv4.rotate(q, signs) if rotated else q
    out = np.zeros_like(q)
    for b, n in enumerate(int(n) for n in lens):
        s0, s1 = int(starts[b]), int(starts[b + 1])
        if n == 0 or s0 == s1:
            continue
        k, v = oracle.kv4.gather(kvals, table[b], n), oracle.kv4.gather(vvals, table[b], n)
        pos, j = n - (s1 - s0) + np.arange(s1 - s0)[:, None], np.arange(n)
        see = np.ones((s1 - s0, n), dtype=bool)
        if causal:
            see &= j <= pos
        if window:
            see &= j > pos - window
        some = see.any(1)
        for h in range(q.shape[1]):
            z = np.where(see, scale * (qr[s0:s1, h] @ k[h // rep].T), -np.inf)
            p = np.exp(z - np.where(some, z.max(1), 0.0)[:, None])
            out[s0:s1, h] = p @ v[h // rep] / np.where(some, p.sum(1), 1.0)[:, None]
    return oracle.kv4.unrotate(out, signs) if rotated else out


@pytest.mark.parametrize("window", [2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,news", [([5], [16]), ([3, 40, 0], [10, 4, 9]), ([33, 100], [133, 160])])
def test_window_that_hides_nothing(window, causal, lens, news):
    """The largest windows hide nothing, also from rows whose positions are negative."""
    rng = _rng(21)
    f = Filled(rng, lens, 2, 128, 128, 16, True)
    for dtype in ("bf16", "f32"):
        _attend(f, rng, news, 4, dtype, causal=causal, window=window)
    _attend(f, rng, news, 4, "bf16", causal=causal, window=window, max_len=FAR)


@pytest.mark.parametrize("starts", [[4, -2 ** 31], [2 ** 31 - 1, 6], [2 ** 31 - 1, -2 ** 31], [5, 2], [-3, 0]])
@pytest.mark.parametrize("n,bound", [(100, None), (4000, None), (100, FAR)])
def test_starts_that_hold_no_rows(starts, n, bound):
    """Starts that decrease or lie outside the queries: nothing is read or written for them."""
    rng = _rng(27)
    f = Filled(rng, [n], 1, 128, 128, 64, True)
    for dtype in ("bf16", "f32"):
        q = _t(rng.standard_normal((6, 4, 128)).astype(np.float32)).to(TYPES[dtype])
        out = torch.full_like(q, 7.0)
        for max_new in (1, 100):
            hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
                             max_new=max_new, max_len=bound, out=out)
            assert (out == 7.0).all()


@pytest.mark.parametrize("dim,group", [(64, 64), (64, 32), (128, 128), (128, 32), (256, 256), (256, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", [2.5, 3.25, 3.75])
@pytest.mark.parametrize("n,news", [(600, 1), (3000, 1), (600, 150)])
def test_sink(dim, group, dtype, size, n, news):
    """One token takes nearly all of the softmax and its value is zero, so the output is what the small probabilities
    make of the others.  Its key is 7 size in dim 0, every query 8 there, the other keys 0: with a scale of 1/8 in log2
    units it is 7 size (12, 16 or 18 nats) above scores of 0 +- 1 nat, exactly in fp16 as well.  The outputs' weights
    are then those of scores near +1 nat, 2^-25 of the largest at the least; values of 1000 keep fp16 outputs (2e-3 to
    1) normal numbers.  fp32: the difference of scores, 26 in log2 units, is good to 26 times 2^-23, 2^-18.3 in the
    probabilities: 2^-17 + 2^-18 allowed."""
    rng = _rng(22)
    heads = 2
    k, v = rng.standard_normal((2, n, heads, dim))
    k *= np.sqrt(128 / dim)
    k[..., 0] = 0.0
    v *= 1000.0
    k[0], v[0] = 0.0, 0.0
    k[0, :, 0] = 7 * size
    f = Held(rng, k, v, group, 32)
    q = rng.standard_normal((news, 2 * heads, dim))
    q[..., 0] = 8.0
    q = _t(q.astype(np.float32)).to(TYPES[dtype])
    tol = TOL[dtype] + (2.0 ** -18 if dtype == "f32" else 0.0)
    for bound in (None, FAR) if news > 1 and dtype == "bf16" else (None,):
        got, want = f.attend(q, scale=0.125 / np.log2(np.e), max_len=bound)
        _close(got, want, tol)


@pytest.mark.parametrize("dim,group", [(64, 64), (128, 128), (128, 32), (256, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", [0.01, 1.0])
def test_huge_value_in_a_masked_place(dim, group, dtype, size):
    """The first row sees a token of the largest values there are, the window hides it from the others: theirs are as
    good as without it."""
    rng = _rng(23)
    n, news, heads, window = 700, 24, 2, 600
    k, v = rng.standard_normal((2, n, heads, dim))
    v *= size
    v[n - news - window + 1] = 6e4 * rng.choice([-1.0, 1.0], (heads, dim))      # the first that row 0 sees
    f = Held(rng, k, v, group, 64)
    q = _t(rng.standard_normal((news, 2 * heads, dim)).astype(np.float32)).to(TYPES[dtype])
    for bound in (None, FAR) if dtype == "bf16" else (None,):
        got, want = f.attend(q, window=window, max_len=bound)
        _close(got[1:], want[1:], TOL[dtype])
        _close(got[:1], want[:1], TOL[dtype])


@pytest.mark.parametrize("dtype,qsize,scale", [("f32", 1e-42, None), ("f32", 1e-8, 1e-38), ("f32", 1e-45, 1e-3),
                                               ("bf16", 1e-39, None), ("bf16", 1e-8, 1e-38), ("f16", 1e-7, 1e-38),
                                               ("bf16", 2e-39, 3e38), ("f32", 2e-39, 3e38)])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("news", [1, 3, 40])
def test_tiny_queries_and_scales(dtype, qsize, scale, rotate, news):
    """Scores that fp32 holds as subnormal numbers or not at all, beside masked ones: every visible token counts alike.
    Tiny queries under a huge scale are ordinary ones: rotated to 2^-150, scores move by 2^-19.5 (3e38 times 2^-150 /
    sqrt(3) times 11 for 128 dims)."""
    rng = _rng(24)
    f = Filled(rng, [news + 50], 2, 128, 128, 16, rotate)
    starts = np.array([0, news], dtype=np.int32)
    q = _t((rng.standard_normal((news, 4, 128)) * qsize).astype(np.float32)).to(TYPES[dtype])
    want = f.want(_num(q), starts, scale)
    for bound in (None, FAR):
        out = hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), starts=_t(starts), max_new=news, max_len=bound,
                               scale=scale)
        _close(_num(out), want, TOL[dtype])


@pytest.mark.parametrize("news", [[5], [40, 3], [1, 130]])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_starts_without_max_new(news, dtype):
    """With starts alone, every row of every sequence is computed."""
    rng = _rng(25)
    f = Filled(rng, [n + 100 for n in news], 2, 128, 128, 16, True)
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    q = _t(rng.standard_normal((starts[-1], 4, 128)).astype(np.float32)).to(TYPES[dtype])
    out = hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), starts=_t(starts))
    _close(_num(out), f.want(_num(q), starts), TOL[dtype])


# ------------------------------------------------------------------ every form, over many tokens

def _parts(f, total, q_heads, dtype, max_new, window=0):
    """Parts of the token axis that a call's workspace is for: which form a call takes shows in them."""
    need = hr.lib.hr_kv4_attention_workspace(f.heads, f.dim, hr.__dict__[f"HR_{dtype.upper()}"], total, len(f.lens), q_heads,
                                             max_new, f.width * f.page, window)
    return need // (total * q_heads * (4 * f.dim + 8)) if need else 1


def _attend_many(f, rng, news, q_heads, dtype, causal=True, window=0):
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    q = _t(rng.standard_normal((starts[-1], q_heads, f.dim)).astype(np.float32)).to(TYPES[dtype])
    out = hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), starts=_t(starts), max_new=max(news), causal=causal,
                           window=window)
    vals = [np.nan_to_num(oracle.kv4.values(f.codes[i], f.scales[i]), posinf=0, neginf=0) for i in range(2)]
    want = dense(_num(q), *vals, f.table, f.lens, starts, f.dim ** -0.5, f.signs, f.rotate, causal, window)
    _close(_num(out), want, TOL[dtype])


@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 128),
                                       (256, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("page", [16, 64])
def test_row_kernel_over_many_tokens(dim, group, dtype, page):
    """16 rows on four waves: several tiles a wave, parts, pages that end between parts; one row tile, then two."""
    rng = _rng(dim + group + page)
    f = Filled(rng, [2900, 1300, 0], 2, dim, group, page, True)
    assert _parts(f, 3, 8, dtype, 1) > 8
    _attend_many(f, rng, [1, 1, 1], 8, dtype)
    assert 1 < _parts(f, 13, 10, dtype, 5)
    _attend_many(f, rng, [5, 5, 3], 10, dtype)
    _attend_many(f, rng, [5, 5, 3], 10, dtype, causal=False)


@pytest.mark.parametrize("dim,group", [(64, 64), (128, 32), (256, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("causal,window", [(True, 2100), (False, 2100), (False, 3001), (False, 0)])
@pytest.mark.parametrize("news", [[1, 1], [6, 2]])
def test_masks_with_parts(dim, group, dtype, causal, window, news):
    rng = _rng(window + dim)
    f = Filled(rng, [4700, 2450], 1, dim, group, 32, True)
    assert _parts(f, sum(news), 4, dtype, max(news), window) > 4
    _attend_many(f, rng, news, 4, dtype, causal, window)


@pytest.mark.parametrize("dim,group,batch,heads,q_heads,news,n,parts", [
    (64, 64, 1, 2, 8, 600, 2000, 5),            # 128 rows
    (64, 32, 1, 2, 8, 600, 2000, 5),
    (128, 128, 3, 8, 32, 32, 6000, 12),         # 128 rows, joined 16 groups a row
    (128, 32, 3, 8, 32, 32, 6000, 12),
    (128, 128, 9, 2, 8, 96, 2500, 6),           # 256 rows
    (128, 64, 9, 2, 8, 96, 2500, 6),
    (256, 256, 1, 2, 8, 1100, 4400, 8),         # 128 rows
    (256, 64, 1, 2, 8, 1100, 4400, 8),
])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1500), (False, 0)])
def test_prompt_kernel_in_parts(dim, group, batch, heads, q_heads, news, n, parts, causal, window):
    """The number of parts is the prompt kernel's: the row kernel would divide these calls otherwise."""
    rng = _rng(dim + group)
    f = Filled(rng, [n - 70 * b for b in range(batch)], heads, dim, group, 64, True)
    if not window:
        assert _parts(f, batch * news, q_heads, "bf16", news) == parts
    _attend_many(f, rng, [news] * batch, q_heads, "bf16", causal, window)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 64), (128, 128), (128, 32), (256, 64)])
@pytest.mark.parametrize("n,news", [(200, 1), (200, 60), (2600, 1), (2600, 7)])
def test_poisoned_token_in_every_type(dtype, dim, group, n, news):
    rng = _rng(26)
    f = Filled(rng, [n], 2, dim, group, 16, True)
    for h, j in ((0, n - 1), (1, n - 1 - news // 2)):
        page, place = f.table[0, j // 16], j % 16
        for kv, t in ((0, f.cache.k_scales), (1, f.cache.v_scales)):
            t[page, h, :, place] = float("nan")
            f.scales[kv][page, h, :, place] = np.nan
    _attend(f, rng, [news], 4, dtype)


@pytest.mark.parametrize("dim,group", [(64, 64), (128, 128), (256, 256), (128, 32)])
def test_every_fp32_row(dim, group):
    """Each of 80000 rows by itself: one weight of a row off by half a unit of fp16 (2^-12), in one row of thousands, does
    not show in the whole.  The weights of 40 tokens, none above a half or so, are good to 2^-20 (scores of up to 10 in
    log2 units): 2^-17 allowed, as for the whole."""
    rng = _rng(28)
    n, batch, heads = 40, 64, 8
    f = Filled(rng, [n] * batch, heads, dim, group, 64, True)
    starts = n * np.arange(batch + 1, dtype=np.int32)
    q = _t(rng.standard_normal((n * batch, 4 * heads, dim)).astype(np.float32))
    got = _num(hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), starts=_t(starts), max_new=n, causal=False))
    vals = [np.nan_to_num(oracle.kv4.values(f.codes[i], f.scales[i]), posinf=0, neginf=0) for i in range(2)]
    want = dense(_num(q), *vals, f.table, f.lens, starts, dim ** -0.5, f.signs, True, False)
    off = np.linalg.norm(got - want, axis=-1) / np.linalg.norm(want, axis=-1)
    assert off.max() <= TOL["f32"], f"a row is {off.max():.3g} off, the median {np.median(off):.3g}"


@pytest.mark.parametrize("dim,group", [(64, 64), (64, 32), (128, 128), (128, 64)])
@pytest.mark.parametrize("news", [1, 4, 5])
def test_fp16_rows_of_many_sequences(dim, group, news):
    """Enough pairs of a sequence and a head for 32 rows a workgroup, around the 16 rows from which they are taken."""
    rng = _rng(29)
    f = Filled(rng, list(range(news, news + 64)), 8, dim, group, 16, True)
    _attend_many(f, rng, [news] * 64, 32, "f16")


@pytest.mark.parametrize("dim,group", [(64, 64), (128, 32), (256, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,news", [(90, 3), (200, 70), (3000, 3)])
@pytest.mark.parametrize("rotate", [False, True])
def test_queries_that_are_not_finite(dim, group, dtype, n, news, rotate):
    """A query that is not finite makes its own row NaN and leaves those beside it as they are."""
    rng = _rng(30)
    f = Filled(rng, [n], 2, dim, group, 16, rotate)
    x = rng.standard_normal((news, 4, dim)).astype(np.float32)
    starts = np.array([0, news], dtype=np.int32)
    want = f.want(_num(_t(x).to(TYPES[dtype])), starts)
    x[0, 1, 3], x[news - 1, 2] = np.nan, np.nan
    x[1, 0] = np.inf
    bad = np.zeros((news, 4), dtype=bool)
    bad[0, 1] = bad[news - 1, 2] = bad[1, 0] = True
    q = _t(x).to(TYPES[dtype])
    for bound in (None, FAR) if dtype == "bf16" and news > 3 else (None,):
        got = _num(hr.kv4_attention(f.cache, q, _t(f.table), _t(f.lens), starts=_t(starts), max_new=news, max_len=bound))
        assert np.isnan(got[bad].astype(np.float64)).all()
        _close(got[~bad], want[~bad], TOL[dtype])
