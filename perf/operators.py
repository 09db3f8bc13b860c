"""Operators of the 4-bit key/value cache: the cases they are measured on.

Two operators:

* ``write``: keys and values of some tokens are rotated per head (randomized Hadamard transform of the head
  dimension), quantized to int4 groups as they are written into a paged cache, and read back.
* ``attend``: softmax attention of queries over such a cache, in its 4-bit form, with grouped heads, ragged
  lengths, a causal and a window mask; the queries are rotated and the outputs rotated back on the way.

A cache has ``pages`` pages of ``page`` tokens each.  Codes [pages][heads][page][dim / 2] hold two int4 codes
a byte (two's complement, the even element in the low nibble), scales [pages][heads][dim / group][page] are
fp16.  A token's slot is its page times ``page`` plus its place in the page.

Where ``own`` is false, everything here is elementary torch operations in 32 bits; where it is true, ``run``
calls the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def _write(name, tokens, heads, dim, group, page, dtype, rotate):
    return {"name": name, "op": "write", "tokens": tokens, "heads": heads, "dim": dim, "group": group,
            "page": page, "dtype": dtype, "rotate": rotate}


def _attend(name, batch, queries, length, q_heads, heads, dim, group, page, dtype, rotate=True, ragged=True,
            causal=True, window=0):
    return {"name": name, "op": "attend", "batch": batch, "queries": queries, "length": length,
            "q_heads": q_heads, "heads": heads, "dim": dim, "group": group, "page": page, "dtype": dtype,
            "rotate": rotate, "ragged": ragged, "causal": causal, "window": window}


def listed():
    return [
        # one token of one sequence, the write of a single decode step: latency alone
        _write("write one token", 1, 8, 128, 128, 64, "bf16", True),
        # an odd prompt in fp32 without the rotation, small groups and pages: 2048-wide models' 64-wide heads
        _write("write 1237 fp32 plain", 1237, 8, 64, 32, 16, "f32", False),
        # a chunk of prompts in fp16 with wide heads and several groups a head
        _write("write 4099 fp16 wide", 4099, 4, 256, 64, 32, "f16", True),
        # a batch of long prompts at once: the largest write, bound by memory
        _write("write 32768 prompt", 32768, 8, 128, 128, 64, "bf16", True),
        # one sequence that has just begun, one new token: latency alone
        _attend("decode short", 1, 1, 129, 32, 8, 128, 128, 64, "bf16"),
        # a small serving batch of a 2048-wide model, ragged, one sequence of it empty
        _attend("decode 16 ragged", 16, 1, 2048, 32, 8, 64, 64, 16, "bf16"),
        # a full serving batch of a 4096-wide model at ragged lengths: bound by the cache's bytes
        _attend("decode 64 ragged", 64, 1, 8192, 32, 8, 128, 128, 64, "bf16"),
        # one long context: the work of few rows spread over the whole chip
        _attend("decode long", 1, 1, 131071, 32, 8, 128, 128, 256, "bf16"),
        # heads that share nothing, small groups, fp32 queries and outputs
        _attend("decode fp32 groups", 4, 1, 3001, 16, 16, 128, 32, 16, "f32"),
        # a few proposed tokens a sequence checked at once, 5120-wide model
        _attend("verify 5 tokens", 12, 5, 6000, 40, 8, 128, 64, 32, "bf16"),
        # a chunk of a long prompt over what is cached of it already: bound by the matrix products
        _attend("prompt chunk", 1, 2048, 8192, 32, 8, 128, 128, 64, "bf16", ragged=False),
        # ragged prompts of a 2048-wide model with a sliding window
        _attend("prompts window", 6, 1500, 2600, 32, 8, 64, 64, 16, "bf16", window=1024),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dim = rng.choice((64, 128, 128, 256))
    group = rng.choice([g for g in (32, 64, 128, 256) if g < dim] + 3 * [dim])
    page = rng.choice((16, 32, 64, 64, 128, 256))
    heads = rng.choice((1, 2, 4, 8, 8, 16))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if rng.random() < 0.3:
        tokens = _log_int(rng, 1, 32768 * 1024 // max(1024, heads * dim) // (2 if dtype == "f32" else 1))
        # fp32 values are read back unrounded, so a code that falls on the other side of a midpoint would show:
        # these are written without the rotation, whose sums have no one order
        case = _write("", tokens, heads, dim, group, page, dtype, dtype != "f32" and rng.random() < 0.75)
    else:
        q_heads = heads * rng.choice((1, 2, 4, 4, 5, 8))
        form = rng.random()
        wide = max(q_heads * dim, 1024)
        if form < 0.6:       # one new token a sequence
            batch, queries = _log_int(rng, 1, 64), 1
            most = 131071
        elif form < 0.8:     # a few new tokens a sequence
            batch, queries = _log_int(rng, 1, 24), rng.randint(2, 16)
            most = 24 * 8192 // batch
        else:                # prompts and chunks of prompts
            batch = rng.randint(1, 6)
            queries = _log_int(rng, 17, max(17, min(2048, math.isqrt(2048 * 8192 * 4096 // (2 * batch * wide)))))
            most = 8192
        # neither the cache nor the products are larger than the largest of the listed cases
        most = min(most, 64 * 4096 * 1024 // (batch * max(heads * dim, 1024)), 2048 * 7168 * 4096 // (batch * queries * wide))
        length = _log_int(rng, queries, max(queries, most))
        if dtype == "f32":
            length = max(queries, length // 2)
        case = _attend("", batch, queries, length, q_heads, heads, dim, group, page, dtype,
                       rotate=rng.random() < 0.75, ragged=rng.random() < 0.75, causal=rng.random() < 0.85,
                       window=rng.choice((0, 0, 0, _log_int(rng, 1, length))))
    del case["name"]
    return case


def _lengths(case):
    """(cached lengths, new tokens) of each sequence: ragged ones spread over [1/8, 1] of the largest, the last
    of a larger batch empty.  The cached length counts the new tokens; an empty one still asks one row."""
    n, b = case["length"], case["batch"]
    lens, news = [], []
    for i in range(b):
        f = 1.0 - 0.875 * ((i * 0.6180339887) % 1.0) if case["ragged"] else 1.0
        q = max(1, int(case["queries"] * f))
        lens.append(max(q, int(n * f)))
        news.append(q)
    if case["ragged"] and b >= 16:
        lens[-1] = 0
        news[-1] = 1
    return lens, news


# ------------------------------------------------------------------ inputs

def _quantize(y, group):
    """Codes (as fp32 integers) and fp16 scales of y [..., dim] in groups of `group`."""
    g = y.unflatten(-1, (-1, group))
    a = g.abs().amax(-1)
    s = (a / torch.full_like(a, 7.0)).half()
    f = s.float().unsqueeze(-1)
    k = torch.where(f > 0, 1.0 / f, torch.zeros_like(f))
    return (g * k).round().clamp(-7, 7), s


def _pack(codes):
    """fp32 integer codes [..., dim] -> bytes [..., dim / 2]."""
    c = codes.to(torch.int16) & 15
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def _filled(gen, pages, case):
    """Codes and scales of a filled cache: rotated values are near Gaussian, their size varies from token to
    token and by head."""
    h, p, d = case["heads"], case["page"], case["dim"]
    y = torch.randn((pages, h, p, d), generator=gen, device=DEV)
    y *= torch.exp(0.3 * torch.randn((pages, h, p, 1), generator=gen, device=DEV))
    codes, s = _quantize(y, case["group"])
    return _pack(codes.flatten(-2)), s.transpose(-1, -2).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    dim, heads, page, group = case["dim"], case["heads"], case["page"], case["group"]
    dtype = DTYPES[case["dtype"]]
    signs = None
    if case["rotate"]:
        signs = (torch.randint(0, 2, (dim,), generator=gen, device=DEV) * 2 - 1).to(torch.int8)
    if case["op"] == "write":
        tokens = case["tokens"]
        pages = -(-tokens // page) + 3
        # keys and values as one product leaves them, side by side; a few channels are far larger than the rest
        kv = torch.randn((tokens, 2 * heads * dim), generator=gen, device=DEV)
        wide = 1.0 + 19.0 * (torch.rand((2 * heads * dim,), generator=gen, device=DEV) < 0.01)
        kv = (kv * wide).to(dtype)
        order = torch.randperm(pages * page, generator=gen, device=DEV) if tokens < 256 else None
        if order is None:       # whole pages in any order, the last one of them part filled
            at = torch.arange(tokens, device=DEV)
            slots = torch.randperm(pages, generator=gen, device=DEV)[at // page] * page + at % page
        else:                   # new tokens of many sequences
            slots = order[:tokens].contiguous()
        k = kv[:, :heads * dim].view(tokens, heads, dim)
        v = kv[:, heads * dim:].view(tokens, heads, dim)
        codes = torch.zeros((2, pages, heads, page, dim // 2), dtype=torch.uint8, device=DEV)
        scales = torch.zeros((2, pages, heads, dim // group, page), dtype=torch.float16, device=DEV)
        state = {"case": case, "k": k, "v": v, "slots": slots, "signs": signs}
        parts = (codes[0], scales[0], codes[1], scales[1])
    else:
        lens, news = _lengths(case)
        need = [-(-n // page) for n in lens]
        width = max(1, max(need))
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
        first = torch.tensor(np.concatenate([[0], np.cumsum(need)[:-1]]), device=DEV).unsqueeze(1)
        at = torch.arange(width, device=DEV).unsqueeze(0)
        live = at < torch.tensor(need, device=DEV).unsqueeze(1)
        table = torch.where(live, order[torch.where(live, first + at, 0)], 0).to(torch.int32)
        starts = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32, device=DEV)
        total = sum(news)
        q_heads = case["q_heads"]
        qkv = torch.randn((total, (q_heads + 2 * heads) * dim), generator=gen, device=DEV).to(dtype)
        q = qkv[:, :q_heads * dim].view(total, q_heads, dim)
        parts = _filled(gen, pages, case) + _filled(gen, pages, case)
        state = {"case": case, "q": q, "table": table, "signs": signs, "starts": starts,
                 "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
                 "most_new": max(news), "most": max(max(lens), 1)}
    state["parts"] = parts
    if own:
        import hadamard_rotation_int4_amd as hr

        state["cache"] = hr.KV4Cache(*parts, rotate=case["rotate"], signs=signs)
    return state


# ------------------------------------------------------------------ plain forms

def _hadamard(dim, signs):
    """The rotation of a head as a matrix R [dim][dim], y = x R: R[j][i] = signs[j] H[i][j] / sqrt(dim)."""
    i = torch.arange(dim, device=DEV)
    bits = i.unsqueeze(0) & i.unsqueeze(1)
    for_parity = bits ^ (bits >> 4)
    for_parity = for_parity ^ (for_parity >> 2)
    for_parity = (for_parity ^ (for_parity >> 1)) & 1
    h = (1 - 2 * for_parity).float() / math.sqrt(dim)
    return h * signs.float().unsqueeze(1)


def _values(codes, scales, group):
    """fp32 values [..., page, dim] of codes [..., page, dim / 2] and scales [..., dim / group, page]."""
    lo = ((codes & 15) ^ 8).to(torch.int8) - 8
    hi = ((codes >> 4) ^ 8).to(torch.int8) - 8
    q = torch.stack((lo, hi), -1).flatten(-2).float()
    return (q.unflatten(-1, (-1, group)) * scales.transpose(-1, -2).float().unsqueeze(-1)).flatten(-2)


def _plain_write(state):
    case = state["case"]
    group, page, dim = case["group"], case["page"], case["dim"]
    page_of, place = state["slots"] // page, state["slots"] % page
    r = _hadamard(dim, state["signs"]) if case["rotate"] else None
    kc, ks, vc, vs = state["parts"]

    def one(x, codes, scales):
        y = x.float()
        y = y @ r if r is not None else y
        c, s = _quantize(y, group)
        codes[page_of, :, place] = _pack(c.flatten(-2))
        scales[page_of, :, :, place] = s
        back = _values(codes[page_of, :, place].unsqueeze(-2), scales[page_of, :, :, place].unsqueeze(-1), group)
        back = back.squeeze(-2)
        return (back @ r.t() if r is not None else back).to(x.dtype)

    return one(state["k"], kc, ks), one(state["v"], vc, vs)


def _plain_attend(state):
    case, q = state["case"], state["q"]
    total, q_heads, dim = q.shape
    heads, group = case["heads"], case["group"]
    rep = q_heads // heads
    table, lens, starts = state["table"].long(), state["lens"].long(), state["starts"].long()
    batch, new = table.shape[0], state["most_new"]
    r = _hadamard(dim, state["signs"]) if case["rotate"] else None

    def cached(codes, scales):      # [batch][heads][tokens][dim]
        c = codes[table].transpose(1, 2)
        s = scales[table].transpose(1, 2)
        return _values(c, s, group).flatten(2, 3)

    kc, ks, vc, vs = state["parts"]
    k, v = cached(kc, ks), cached(vc, vs)
    news = starts[1:] - starts[:-1]
    i = torch.arange(new, device=DEV)
    row = torch.minimum(starts[:-1].unsqueeze(1) + i, starts[1:].unsqueeze(1) - 1)    # padded with the last
    x = q.float()
    x = x @ r if r is not None else x
    x = x[row].view(batch, new, heads, rep, dim).permute(0, 2, 3, 1, 4).reshape(batch, heads, rep * new, dim)
    score = x @ k.transpose(-1, -2) * (1.0 / math.sqrt(dim))
    j = torch.arange(k.shape[2], device=DEV)
    pos = (lens - news).unsqueeze(1) + i                                              # [batch][new]
    seen = (j < lens[:, None, None]).expand(batch, new, -1)
    if case["causal"]:
        seen = seen & (j <= pos.unsqueeze(-1))
    if case["window"]:
        seen = seen & (j > pos.unsqueeze(-1) - case["window"])
    seen = seen[:, None, None].expand(batch, heads, rep, new, -1).reshape(score.shape)
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp_(score.sub_(top))
    norm = e.sum(-1, keepdim=True)
    out = e @ v / torch.where(norm > 0, norm, 1.0)
    out = out @ r.t() if r is not None else out
    out = out.view(batch, heads, rep, new, dim).permute(0, 3, 1, 2, 4).reshape(batch, new, q_heads, dim)
    t = torch.arange(total, device=DEV)
    b = torch.bucketize(t, starts[1:], right=True)
    return out[b, t - starts[b]].to(q.dtype)


def run(state):
    if not own:
        return _plain_write(state) if state["case"]["op"] == "write" else _plain_attend(state)
    import hadamard_rotation_int4_amd as hr

    case, cache = state["case"], state["cache"]
    if case["op"] == "write":
        hr.kv4_append(cache, state["k"], state["v"], state["slots"])
        return hr.kv4_read(cache, state["slots"], dtype=state["k"].dtype)
    return hr.kv4_attention(cache, state["q"], state["table"], state["lens"], starts=state["starts"],
                            max_new=state["most_new"], max_len=state["most"], causal=case["causal"],
                            window=case["window"])


# ------------------------------------------------------------------ work

def _seen_of(case, length, new):
    """(pairs of a row and a token it sees, tokens that any row sees) of one sequence, a head."""
    pairs, first, last = 0, length, 0
    for i in range(new):
        pos = length - new + i
        hi = min(length, pos + 1) if case["causal"] else length
        lo = max(0, pos - case["window"] + 1) if case["window"] else 0
        if hi > lo:
            pairs += hi - lo
            first, last = min(first, lo), max(last, hi)
    return pairs, max(0, last - first)


def work(case):
    dim, heads = case["dim"], case["heads"]
    size = 4 if case["dtype"] == "f32" else 2
    packed = dim // 2 + 2 * (dim // case["group"])       # bytes of one token's key or value, one head
    if case["op"] == "write":
        vectors = 2 * case["tokens"] * heads
        # values in, codes out, codes in, values out; a slot is read by each of the two calls
        turn = 4 * dim * int(math.log2(dim)) if case["rotate"] else 0
        return {"bytes": vectors * (2 * dim * size + 2 * packed) + 16 * case["tokens"],
                "flops": vectors * (turn // 2 + 4 * dim)}
    lens, news = _lengths(case)
    pairs = tokens = 0
    for n, q in zip(lens, news):
        a, b = _seen_of(case, n, q)
        pairs += a
        tokens += b
    rows = sum(news) * case["q_heads"]
    return {"bytes": 2 * tokens * heads * packed + 2 * rows * dim * size, "flops": 4 * pairs * case["q_heads"] * dim}


# ------------------------------------------------------------------ in 64 bits

def _sylvester(dim):
    h = np.ones((1, 1))
    while h.shape[0] < dim:
        h = np.block([[h, h], [h, -h]])
    return torch.from_numpy(h).to(DEV) / math.sqrt(dim)


def _decoded(codes, scales, group):
    """Every vector of a cache in 64 bits: codes [heads][tokens][dim / 2], scales [heads][dim / group][tokens]."""
    nibble = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1], dtype=torch.float64, device=DEV)
    b = codes.long()
    x = torch.empty((*b.shape[:-1], 2 * b.shape[-1]), dtype=torch.float64, device=DEV)
    x[..., 0::2] = nibble[b % 16]
    x[..., 1::2] = nibble[b // 16]
    return x * scales.double().repeat_interleave(group, 1).transpose(1, 2)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = was
    dim, group, page = case["dim"], case["group"], case["page"]
    turn = None
    if case["rotate"]:
        turn = _sylvester(dim) @ torch.diag(state["signs"].double())      # y = turn x
    if case["op"] == "write":
        got = []
        for x in (state["k"], state["v"]):
            y = x.double()
            if turn is not None:
                y = y @ turn.t()
            y = y.reshape(-1, group)
            top = y.abs().max(dim=1, keepdim=True).values
            s = (top / 7.0).half().double()
            c = torch.where(s > 0, torch.round(y / torch.where(s > 0, s, 1.0)), 0.0).clamp(-7.0, 7.0)
            y = (c * s).view(x.shape)
            got.append(y @ turn if turn is not None else y)
        return tuple(got)
    lens, news = _lengths(case)
    q = state["q"].double()
    rep = case["q_heads"] // case["heads"]
    kc, ks, vc, vs = state["parts"]
    out = torch.zeros_like(q)
    at = 0
    for b, (n, new) in enumerate(zip(lens, news)):
        if n:
            ids = state["table"][b, : -(-n // page)].long()
            k, v = (_decoded(c[ids].transpose(0, 1).flatten(1, 2)[:, :n],
                             s[ids].permute(1, 2, 0, 3).flatten(2, 3)[:, :, :n], group) for c, s in ((kc, ks), (vc, vs)))
            if turn is not None:      # back to the basis of the queries
                k, v = k @ turn, v @ turn
            pos = torch.arange(n - new, n, device=DEV).view(-1, 1)
            j = torch.arange(n, device=DEV).view(1, -1)
            hidden = torch.zeros((new, n), dtype=torch.bool, device=DEV)
            if case["causal"]:
                hidden |= j > pos
            if case["window"]:
                hidden |= j <= pos - case["window"]
            none = hidden.all(1, keepdim=True)
            for h in range(case["q_heads"]):
                logit = q[at:at + new, h] @ k[h // rep].t() / math.sqrt(dim)
                logit[hidden] = -1e300
                p = torch.softmax(logit, 1)
                out[at:at + new, h] = torch.where(none, 0.0, p @ v[h // rep])
        at += new
    return out
