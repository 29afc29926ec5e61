"""Measured cases of the operators between the projections of an attention
layer: the per-head norm and position rotation of queries and keys, the append
of new keys and values to a paged cache held in 4 bits, and the attention that
reads that cache.

A case is a dict of plain values; ``listed()`` names the fixed ones, ``draw``
makes one more of the same ranges, ``prepare`` makes its inputs on the GPU,
``run`` makes one pass (plain torch operations, or the library's calls where
``own`` is true), ``work`` counts what the pass cannot do without, and
``exact`` computes the outputs in 64 bits.

The cache is a pool of pages, ``[pages][page bytes]``; a sequence's tokens lie
in the pages its row of ``tables`` names.  A page holds, for each head, tiles of
16 tokens of 20 * D bytes:

* key codes, 8 * D bytes: lane (h, r), h = 0..3, of token r has the dims
  D/4 * h .. in 32-bit words of 8; code 8j + 2p of a word at bits [4p, 4p+4),
  code 8j + 2p + 1 at [16 + 4p, 20 + 4p);
* key headers, 2 * D bytes: for each group of 32 dims the 16 tokens' (scale,
  minimum), two fp16;
* value codes, 8 * D bytes: lane (h, n), n = 0..15, has the dims E * n .. E * n +
  E - 1 (E = D/16) of the tokens 4h .. 4h+3, two dims to a 32-bit word; dim parity
  b and token i at bits 4 * (2b + i/2) + 16 * (i%2);
* value headers, 2 * D bytes, as the keys'.

A value is code * scale + minimum, of values held to +-32768: minimum =
fp16(min of the group), scale = fp16((max - minimum) / 15), code = the nearest
of 0..15 to (x - minimum) / scale.
"""
import math
import random

import torch

#: False: ``run`` computes the plain forms; True: it calls the library
own = False

_DT = {"float16": torch.float16, "bfloat16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(name, **c):
    if name:
        c["name"] = name
    return c


def _rope(name, T, heads, kv_heads, D, rot, dtype, interleaved=False, norm=True):
    return _case(name, op="norm_rope", T=T, heads=heads, kv_heads=kv_heads, D=D, rot=rot, dtype=dtype,
                 interleaved=interleaved, norm=norm)


def _append(name, S, T, ctx, heads, kv_heads, D, page, rot, dtype, interleaved=False, norm=True, queries=True):
    """S sequences of up to `ctx` earlier tokens, T new ones together; with
    `queries`, the queries are normed and rotated in the same pass."""
    return _case(name, op="append", S=S, T=T, ctx=ctx, heads=heads, kv_heads=kv_heads, D=D, page=page, rot=rot,
                 dtype=dtype, interleaved=interleaved, norm=norm, queries=queries)


def _attn(name, S, T, ctx, heads, kv_heads, D, page, dtype, window=0):
    """S sequences of up to `ctx` earlier tokens, T new ones together, whose
    queries read the cache."""
    return _case(name, op="attn", S=S, T=T, ctx=ctx, heads=heads, kv_heads=kv_heads, D=D, page=page, dtype=dtype,
                 window=window)


def listed():
    """The fixed cases."""
    return [
        # one new token of a layer with 32 query and 8 key heads
        _rope("norm_rope_t1", 1, 32, 8, 128, 128, "float16"),
        # a long ragged prompt, half of each head rotated, neighbouring pairs
        _rope("norm_rope_t4099_partial", 4099, 32, 4, 128, 64, "bfloat16", interleaved=True),
        # one new token behind a 657-token prompt, its query in the same pass
        _append("append_s1_t1", 1, 1, 657, 32, 8, 128, 64, 128, "float16"),
        # sixty-four sequences decoding, small pages
        _append("append_s64_t64", 64, 64, 8191, 32, 8, 128, 16, 128, "bfloat16"),
        # a 658-token prompt into an empty cache
        _append("append_t658", 1, 658, 0, 32, 8, 128, 64, 128, "float16"),
        # five prompts' chunks behind earlier tokens, small heads, no norm
        _append("append_s5_t8192", 5, 8192, 4096, 16, 8, 64, 32, 64, "bfloat16", norm=False, queries=False),
        # one new token over the 658 it belongs to
        _attn("attn_s1_t1", 1, 1, 657, 32, 8, 128, 64, "float16"),
        # sixteen sequences decoding, three query heads to a key head, small heads
        _attn("attn_s16_t16_d64", 16, 16, 4095, 24, 8, 64, 16, "bfloat16"),
        # sixty-four sequences decoding over long contexts
        _attn("attn_s64_t64", 64, 64, 8191, 32, 8, 128, 64, "bfloat16"),
        # a 658-token prompt
        _attn("attn_t658", 1, 658, 0, 32, 8, 128, 64, "float16"),
        # chunks of three prompts behind long contexts
        _attn("attn_s3_t1100_chunks", 3, 1100, 8000, 32, 8, 128, 64, "bfloat16"),
        # a long prompt
        _attn("attn_t4096", 1, 4096, 0, 32, 8, 128, 64, "bfloat16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    D = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 8, 8, 16))
    heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 4, 5, 7, 8, 16) if kv_heads * g <= 40])
    dtype = rng.choice(("float16", "bfloat16"))
    page = rng.choice((16, 32, 64, 128, 256))
    rot = rng.choice((D, D, D // 2, 16))
    kind = rng.choice(("norm_rope", "append", "append", "attn", "attn", "attn"))
    if kind == "norm_rope":
        return _rope(None, _log(rng, 1, 4500), heads, kv_heads, D, rot, dtype, rng.random() < 0.4, rng.random() < 0.8)
    if rng.random() < 0.5:  # every sequence decodes
        S = _log(rng, 1, 64)
        T, ctx = S, _log(rng, 1, 8191)
    else:
        S = _log(rng, 1, 8)
        T, ctx = S + _log(rng, 1, 8192 if kind == "append" else 3000), rng.choice((0, _log(rng, 1, 8000)))
        while kind == "attn" and S * heads * T * (ctx + T) > 5e8:  # no dearer than the long prompt
            T, ctx = S + (T - S) * 3 // 4, ctx * 3 // 4
    if kind == "append":
        return _append(None, S, T, ctx, heads, kv_heads, D, page, rot, dtype, rng.random() < 0.4, rng.random() < 0.7,
                       rng.random() < 0.6)
    return _attn(None, S, T, ctx, heads, kv_heads, D, page, dtype, rng.choice((0, 0, 0, _log(rng, 1, 2000))))


def _lengths(c):
    """Each sequence's new tokens and its length with them."""
    S, T, ctx = c["S"], c["T"], c["ctx"]
    if S == 1:
        return [T], [ctx + T]
    rng = random.Random(f"{S} {T} {ctx} {c['page']}")
    if S == T:
        new = [1] * S
    else:
        cuts = sorted(rng.sample(range(1, T), S - 1))
        new = [b - a for a, b in zip([0] + cuts, cuts + [T])]
    return new, [n + rng.randint(ctx // 4, ctx) for n in new]


# ---------------------------------------------------------------------------
# the cache's format, in elementary operations
# ---------------------------------------------------------------------------

def _quantize(x):
    """x [..., D], float32 or float64 -> codes [..., D] uint8, scales and minima [..., D/32] fp16."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    g = torch.where(g == g, g, torch.zeros_like(g)).clamp(-32768.0, 32768.0)
    m = g.amin(-1).half()
    s = ((g.amax(-1) - m.to(x.dtype)) / 15).half()
    live = s > 0
    t = (g - m.to(x.dtype)[..., None]) / torch.where(live, s, torch.ones_like(s)).to(x.dtype)[..., None]
    q = torch.round(t).clamp(0, 15) * live[..., None]
    return q.to(torch.uint8).view(x.shape), s, m


def _header_bytes(s, m):
    """[..., tokens, groups] scales and minima -> [..., tokens, groups, 4] bytes."""
    return torch.stack([s, m], -1).contiguous().view(torch.uint8)


def _key_bytes(q):
    """Codes [..., D] of a token -> its bytes [..., 4 lanes, D/8]."""
    D = q.shape[-1]
    v = q.view(*q.shape[:-1], 4, D // 32, 2, 2, 2)  # [lane][word][half of the word][pair][parity]
    low, high = v[..., 0], v[..., 1]
    by = torch.cat([low[..., 0] | (low[..., 1] << 4), high[..., 0] | (high[..., 1] << 4)], -1)
    return by.view(*q.shape[:-1], 4, D // 8)


def _key_codes(by):
    """Bytes [..., 4 lanes, D/8] -> codes [..., D]."""
    w = by.reshape(*by.shape[:-1], -1, 4)  # [lane][word][byte]
    even = torch.stack([w & 15, w >> 4], -1)[..., :2, :]
    odd = torch.stack([w & 15, w >> 4], -1)[..., 2:, :]
    return torch.stack([even, odd], -1).reshape(*by.shape[:-2], -1)


def _pages(c):
    return sum((n + c["page"] - 1) // c["page"] for n in _lengths(c)[1]) + 3


def _pack_pages(kq, ks, km, vq, vs, vm):
    """Codes [P, heads, page, D] and headers [P, heads, page, D/32] -> [P, page bytes]."""
    P, H, page, D = kq.shape
    n = page // 16

    def heads(s, m):
        return _header_bytes(s, m).view(P, H, n, 16, D // 32, 4).permute(0, 1, 2, 4, 3, 5).reshape(P, H, n, -1)

    kb = _key_bytes(kq).view(P, H, n, 16, 4, D // 8).permute(0, 1, 2, 4, 3, 5).reshape(P, H, n, -1)
    v = vq.view(P, H, n, 4, 4, 16, D // 32, 2).permute(0, 1, 2, 3, 5, 6, 7, 4)  # [h][lane n][word][parity][token]
    vb = torch.cat([v[..., 0] | (v[..., 2] << 4), v[..., 1] | (v[..., 3] << 4)], -1).reshape(P, H, n, -1)
    return torch.cat([kb, heads(ks, km), vb, heads(vs, vm)], -1).view(P, -1).contiguous()


def _unpack_pages(by, H, page, D):
    """[N, page bytes] -> float32 keys and values [N, heads, page, D]."""
    N, n = by.shape[0], page // 16
    t = by.view(N, H, n, 20 * D)

    def heads(b):
        f = b.reshape(N, H, n, D // 32, 16, 4).contiguous().view(torch.float16).float()
        return f.permute(0, 1, 2, 4, 3, 5).reshape(N, H, page, D // 32, 1, 2)

    kq = _key_codes(t[..., :8 * D].reshape(N, H, n, 4, 16, D // 8).permute(0, 1, 2, 4, 3, 5))
    w = t[..., 10 * D:18 * D].reshape(N, H, n, 4, 16, D // 32, 2, 2)  # [h][lane n][word][token parity][dim parity]
    vq = torch.stack([w & 15, w >> 4], -1).permute(0, 1, 2, 3, 8, 6, 4, 5, 7).reshape(N, H, page, D)
    k, v = kq.view(N, H, page, D // 32, 32).float(), vq.reshape(N, H, page, D // 32, 32).float()
    kh, vh = heads(t[..., 8 * D:10 * D]), heads(t[..., 18 * D:])
    return ((k * kh[..., 0] + kh[..., 1]).view(N, H, page, D), (v * vh[..., 0] + vh[..., 1]).view(N, H, page, D))


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _normed(x, weight, eps):
    """x [T, H, D] in any float type: divided by the root mean square of each head, times the weight."""
    return x if weight is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.to(x.dtype)


def _rotated(x, table, positions, interleaved):
    """Pairs of each head turned by the angles of the token's position."""
    rot = table.shape[1]
    cs = table[positions.long()].to(x.dtype)[:, None, :]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_norm_rope(c, st):
    q = _rotated(_normed(st["q"].float(), st["q_weight"], 1e-6), st["rope"], st["positions"], c["interleaved"])
    k = _rotated(_normed(st["k"].float(), st["k_weight"], 1e-6), st["rope"], st["positions"], c["interleaved"])
    return q.to(st["q"].dtype), k.to(st["k"].dtype)


def _new_tokens(c, st):
    """Of each new token: its sequence and its place in it."""
    T = c["T"]
    t = torch.arange(T, device="cuda")
    if st["offsets"] is None:
        return t, st["lens"].long() - 1
    off = st["offsets"].long()
    s = torch.searchsorted(off, t, right=True) - 1
    return s, st["lens"].long()[s] - off[s + 1] + t


def _put_values(flat, at, words, place, i):
    """The 4-bit codes of the tokens whose place in their quad is i."""
    sel = (place == i).nonzero()[:, 0]
    shift = 4 * (i // 2)
    j = at[sel][..., [0, 1] if i % 2 == 0 else [2, 3]]
    flat[j] = (flat[j] & (0xF0 >> shift)) | (words[sel] << shift)


def _plain_append(c, st):
    """In 64 bits up to the codes, which a last bit could turn."""
    T, H, D, page = c["T"], c["kv_heads"], c["D"], c["page"]
    dt = st["k"].dtype
    s, place = _new_tokens(c, st)
    k = _rotated(_normed(st["k"].double(), st["k_weight"], 1e-6), st["rope"], st["positions"], c["interleaved"])
    kq, ks, km = _quantize(k)
    vq, vs, vm = _quantize(st["v"].double())
    cache = st["cache"]
    flat = cache.view(-1)
    ids = st["tables"].long()[s, place // page]
    row, quad, r = place % 16, place % 16 // 4, place % 4
    base = (ids[:, None] * cache.shape[1] + torch.arange(H, device="cuda") * (page // 16 * 20 * D)
            + (place % page // 16 * 20 * D)[:, None])
    ar = lambda n: torch.arange(n, device="cuda")
    k_at = (base[:, :, None, None] + (ar(4)[:, None] * 16 + row[:, None, None, None]) * (D // 8) + ar(D // 8))
    h_at = (base[:, :, None, None] + 8 * D + (ar(D // 32)[:, None] * 16 + row[:, None, None, None]) * 4 + ar(4))
    v_at = (base[:, :, None, None] + 10 * D + (quad[:, None, None, None] * 16 + ar(16)[:, None]) * (D // 8) + ar(D // 8))
    flat[k_at] = _key_bytes(kq)
    flat[h_at] = _header_bytes(ks, km)
    flat[h_at + 10 * D] = _header_bytes(vs, vm)
    quads = v_at.view(T, H, 16, D // 32, 4)
    words = vq.view(T, H, 16, D // 32, 2)
    _put_values(flat, quads, words, r, 0)
    _put_values(flat, quads, words, r, 1)
    _put_values(flat, quads, words, r, 2)
    _put_values(flat, quads, words, r, 3)
    # the new tokens as the cache holds them
    kh = flat[h_at].contiguous().view(torch.float16).float().view(T, H, D // 32, 1, 2)
    vh = flat[h_at + 10 * D].contiguous().view(torch.float16).float().view(T, H, D // 32, 1, 2)
    by = flat[quads]
    odd = (r % 2 == 1)[:, None, None, None, None]
    by = torch.where(odd, by[..., 2:], by[..., :2])
    by = torch.where((r // 2 == 1)[:, None, None, None, None], by >> 4, by & 15)
    kr = _key_codes(flat[k_at]).view(T, H, D // 32, 32).float() * kh[..., 0] + kh[..., 1]
    vr = by.reshape(T, H, D // 32, 32).float() * vh[..., 0] + vh[..., 1]
    out = (kr.view(T, H, D).to(dt), vr.view(T, H, D).to(dt))
    if c["queries"]:
        q = _rotated(_normed(st["q"].float(), st["q_weight"], 1e-6), st["rope"], st["positions"], c["interleaved"])
        out = (q.to(dt), *out)
    return out


def _plain_attn(c, st):
    S, T, H, D = c["S"], c["T"], c["kv_heads"], c["D"]
    G = c["heads"] // H
    tables, lens = st["tables"].long(), st["lens"].long()
    s, place = _new_tokens(c, st)
    k, v = _unpack_pages(st["cache"][tables.reshape(-1)], H, c["page"], D)
    k = k.view(S, -1, H, c["page"], D).transpose(1, 2).reshape(S * H, -1, D)
    v = v.view(S, -1, H, c["page"], D).transpose(1, 2).reshape(S * H, -1, D)
    L = k.shape[1]
    row = torch.arange(T, device="cuda") - (0 if st["offsets"] is None else st["offsets"].long()[s])
    if st["offsets"] is None:
        row = torch.zeros_like(row)
    most = st["most_new"]
    q = torch.zeros((S, most, H, G, D), device="cuda")
    q[s, row] = st["q"].float().view(T, H, G, D)
    at = torch.full((S, most), -1, dtype=torch.long, device="cuda")
    at[s, row] = place
    q = q.permute(0, 2, 1, 3, 4).reshape(S * H, most * G, D)
    keys = torch.arange(L, device="cuda")
    seen = (keys <= at[..., None]) & (keys < lens[:, None, None])
    if c["window"]:
        seen = seen & (keys > at[..., None] - c["window"])
    seen = seen[:, None, :, None, :]
    x = torch.matmul(q, k.transpose(1, 2)).mul_(D ** -0.5).view(S, H, most, G, L)
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    n = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(S * H, most * G, L), v).view(S, H, most, G, D)
    o = o / torch.where(n > 0, n, torch.ones_like(n))
    return o.transpose(1, 2)[s, row].reshape(T, c["heads"], D).to(st["q"].dtype)


# ---------------------------------------------------------------------------
# the measured calls
# ---------------------------------------------------------------------------

#: positions that the rotation's table covers
_POSITIONS = 32768


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _rope_table(rot):
    """[positions][rot]: the cosines of each pair's angle, then the sines."""
    a = torch.arange(_POSITIONS, dtype=torch.float64, device="cuda")[:, None] * torch.pow(
        1e6, -2.0 / rot * torch.arange(rot // 2, dtype=torch.float64, device="cuda"))
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float()


def _cache_fields(c, seed):
    """The logical contents of every page: keys with a preferred direction for
    each head, as trained ones have, and values around an offset."""
    g = _gen(seed, 5)
    shape = (_pages(c), c["kv_heads"], c["page"], c["D"])
    dev = dict(device="cuda", generator=g)
    bias = torch.randn((c["kv_heads"], 1, c["D"]), **dev)
    k = _quantize(torch.randn(shape, **dev).add_(bias))
    v = _quantize(torch.randn(shape, **dev).add_(bias, alpha=0.3))
    return (*k, *v)


def prepare(case, seed):
    """Inputs and the cache of one case on the GPU, from the seed alone."""
    c = case
    st = dict(case=c)
    g = _gen(seed, 1)
    dt = _DT[c["dtype"]]
    T, Hq, H, D = c["T"], c["heads"], c["kv_heads"], c["D"]
    dev = dict(device="cuda", generator=g)
    if c["op"] != "norm_rope":
        new, lens = _lengths(c)
        st["most_new"] = max(new)
        width = max((n + c["page"] - 1) // c["page"] for n in lens)
        free = torch.randperm(_pages(c), **dev).int()
        tables = torch.zeros((c["S"], width), dtype=torch.int32, device="cuda")
        first = 0
        for s, n in enumerate(lens):
            need = (n + c["page"] - 1) // c["page"]
            tables[s, :need] = free[first:first + need]
            first += need
        st["tables"] = tables
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["offsets"] = None
        if T != c["S"]:
            st["offsets"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    if c["op"] == "attn":
        st["cache"] = _pack_pages(*_cache_fields(c, seed))
        st["q"] = (1.5 * torch.randn((T, Hq, D), **dev)).to(dt)
        return st
    # one projection's output, its columns the query, key and value heads
    qkv = torch.randn((T, Hq + 2 * H, D), **dev)
    qkv = (qkv * (0.5 + torch.rand((Hq + 2 * H, D), **dev))).to(dt)
    st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    st["q_weight"] = 0.5 + torch.rand(D, **dev) if c["norm"] else None
    st["k_weight"] = 0.5 + torch.rand(D, **dev) if c["norm"] else None
    st["rope"] = _rope_table(c["rot"])
    if c["op"] == "norm_rope":
        start = torch.randint(0, _POSITIONS - T, (1,), **dev)
        st["positions"] = (start + torch.arange(T, device="cuda")).int()
    else:
        st["positions"] = _new_tokens(c, st)[1].int()
        n = H * c["page"] // 16 * 20 * D
        st["cache"] = torch.randint(0, 256, (_pages(c), n), dtype=torch.uint8, **dev)
    return st


def run(state):
    """One pass through the case's operator, and its outputs."""
    c = state["case"]
    if not own:
        if c["op"] == "norm_rope":
            return _plain_norm_rope(c, state)
        if c["op"] == "append":
            return _plain_append(c, state)
        return _plain_attn(c, state)
    import quantized_weight_prefill_amd as qg

    st = state
    if c["op"] == "norm_rope":
        return qg.qk_norm_rope(st["q"], st["k"], st["rope"], st["positions"], q_weight=st["q_weight"],
                               k_weight=st["k_weight"], eps=1e-6 if c["norm"] else None, interleaved=c["interleaved"])
    if c["op"] == "append":
        q = qg.kv_append(st["cache"], st["k"], st["v"], st["tables"], st["lens"], offsets=st["offsets"],
                         rope=st["rope"], positions=st["positions"], k_weight=st["k_weight"],
                         eps=1e-6 if c["norm"] else None, interleaved=c["interleaved"],
                         q=st["q"] if c["queries"] else None, q_weight=st["q_weight"] if c["queries"] else None)
        k, v = qg.kv_read(st["cache"], st["tables"], st["lens"], c["T"], c["kv_heads"], c["D"], offsets=st["offsets"],
                          dtype=st["k"].dtype)
        return (q, k, v) if c["queries"] else (k, v)
    return qg.kv_attention(st["q"], st["cache"], st["tables"], st["lens"], c["kv_heads"], offsets=st["offsets"],
                           window=c["window"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    """Bytes and operations of one pass: each input read once, each output
    written once; of the cache, the tokens that some query sees, and of the
    append's values the 16-bit copies that the pass returns."""
    c = case
    T, Hq, H, D = c["T"], c["heads"], c["kv_heads"], c["D"]
    cached = 2 * H * (D // 2 + D // 8)  # of one token
    if c["op"] == "norm_rope":
        by = 2 * 2 * T * (Hq + H) * D + T * (4 * c["rot"] + 4) + 8 * D * c["norm"]
        return {"bytes": by, "flops": 8.0 * T * (Hq + H) * D}
    new, lens = _lengths(c)
    width = max((n + c["page"] - 1) // c["page"] for n in lens)
    by = 4 * (c["S"] * min(width, sum(lens) // c["S"] // c["page"] + 1) + 2 * c["S"] + 1)
    if c["op"] == "append":
        q = 2 * 2 * T * Hq * D * c["queries"]
        by += 2 * T * H * D * 2 + T * cached + q + T * (4 * c["rot"] + 4) + 2 * T * H * D * 2 + 4 * D * c["norm"]
        return {"bytes": by, "flops": 12.0 * T * H * D * 2 + 8.0 * T * Hq * D * c["queries"]}
    seen = pairs = 0
    for n, length in zip(new, lens):
        w = c["window"] or length
        first = length - n
        seen += min(length, n - 1 + w)
        full = max(0, length - max(first, w - 1))  # queries whose window is full
        pairs += full * w + sum(range(first + 1, first + 1 + n - full))
    by += seen * cached + 2 * 2 * T * Hq * D
    return {"bytes": by, "flops": 4.0 * pairs * Hq * D}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _turn64(x, weight, table, positions, interleaved):
    """Norm and rotation of heads [T, H, D], by complex numbers."""
    x = x.double()
    if weight is not None:
        x = x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * weight.double()
    rot = table.shape[1]
    turn = torch.complex(*table.double()[positions.long()].split(rot // 2, 1))[:, None, :]
    head = x[..., :rot]
    pairs = head.unflatten(-1, (-1, 2)) if interleaved else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, x[..., rot:]], -1)


def _held64(x):
    """What the cache holds of x [T, H, D]."""
    g = x.double().unflatten(-1, (-1, 32))
    low = g.min(-1, keepdim=True)[0].half().double()
    step = ((g.max(-1, keepdim=True)[0] - low) / 15).half().double()
    code = torch.where(step > 0, ((g - low) / step).round().clamp(0, 15), torch.zeros_like(g))
    return (code * step + low).flatten(-2)


def exact(case, seed):
    """What ``run`` returns, from the definition in 64 bits."""
    c = case
    st = prepare(case, seed)
    if c["op"] != "attn":
        turn = lambda x, w: _turn64(x, w, st["rope"], st["positions"], c["interleaved"])
        if c["op"] == "norm_rope":
            return turn(st["q"], st["q_weight"]), turn(st["k"], st["k_weight"])
        out = (_held64(turn(st["k"], st["k_weight"])), _held64(st["v"]))
        return (turn(st["q"], st["q_weight"]), *out) if c["queries"] else out
    H, D, page = c["kv_heads"], c["D"], c["page"]
    G = c["heads"] // H
    kq, ks, km, vq, vs, vm = _cache_fields(c, seed)
    value = lambda q, s, m, p: (q[p].double().unflatten(-1, (-1, 32)) * s[p].double()[..., None]
                                + m[p].double()[..., None]).flatten(-2).transpose(0, 1).flatten(1, 2)
    out, first = [], 0
    for s, (n, length) in enumerate(zip(*_lengths(c))):
        p = st["tables"][s, :(length + page - 1) // page].long()
        k, v = value(kq, ks, km, p)[:, :length], value(vq, vs, vm, p)[:, :length]  # [H, length, D]
        at = torch.arange(length - n, length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")
        hidden = (key > at) | (key <= at - (c["window"] or length + 1))
        q = st["q"][first:first + n].double().unflatten(1, (H, G))
        heads = []
        for h in range(H):
            o = []
            for j in range(G):
                x = (q[:, h, j] @ k[h].t()) / math.sqrt(D)
                o.append(torch.softmax(x.masked_fill_(hidden, -math.inf), 1) @ v[h])
            heads.append(torch.stack(o, 1))
        out.append(torch.cat(heads, 1))
        first += n
    return torch.cat(out)
