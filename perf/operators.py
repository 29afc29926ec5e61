"""Measured cases of the fused feed-forward operators: the linear layer with
its epilogue, the mixture-of-experts routing, and the mixture-of-experts layer
for a few tokens.

A case is a dict of plain values; ``listed()`` names the fixed ones, ``draw``
makes one more of the same ranges, ``prepare`` makes its inputs on the GPU,
``run`` makes one pass (plain torch operations, or the library's calls where
``own`` is true), ``work`` counts what the pass cannot do without, and
``exact`` computes the outputs in 64 bits from the logical weight fields.

Weights are made as logical fields (codes, scales, mins) and laid out in the
packed panel format of ``include/qgemm.h``.  The plain forms and the kernels
both start from the packed bytes; ``exact`` starts from the fields.
"""
import math

import torch

#: False: ``run`` computes the plain forms; True: it calls the library
own = False

_DT = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}
_ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _linear(name, fmt, M, N, K, dtype, layout="row", act="none", gated=False, bias=False, residual=False,
            out_layout="row", group=128, zp=False):
    c = dict(op="linear", fmt=fmt, M=M, N=N, K=K, dtype=dtype, layout=layout, act=act, gated=gated, bias=bias,
             residual=residual, out_layout=out_layout, group=group if fmt == "w4a16" else 0,
             zp=bool(zp) if fmt == "w4a16" else False)
    if name:
        c["name"] = name
    return c


def _moe(name, fmt_up, fmt_down, T, E, k, H, I, dtype, act="silu", residual=False, drop=0.0, group=128, zp=False):
    w4 = "w4a16" in (fmt_up, fmt_down)
    c = dict(op="moe", fmt_up=fmt_up, fmt_down=fmt_down, T=T, E=E, k=k, H=H, I=I, dtype=dtype, act=act,
             residual=residual, drop=drop, group=group if w4 else 0, zp=bool(zp) if w4 else False)
    if name:
        c["name"] = name
    return c


def _route(name, T, E, k, dtype, score="softmax", renorm=True, scale=1.0):
    c = dict(op="route", T=T, E=E, k=k, dtype=dtype, score=score, renorm=renorm, scale=scale)
    if name:
        c["name"] = name
    return c


def _group(name, T, E, k, drop=0.0):
    c = dict(op="group", T=T, E=E, k=k, drop=drop)
    if name:
        c["name"] = name
    return c


def listed():
    """The fixed cases."""
    return [
        # one new token through an attention output projection, added to the residual stream
        _linear("linear_m1_q4k_residual", "q4k", 1, 4096, 4096, "float16", residual=True),
        # sixteen sequences decoding through a long down projection, added to the residual stream
        _linear("linear_m16_q6k_down", "q6k", 16, 4096, 12288, "bfloat16", residual=True),
        # a ragged batch through a biased layer whose width fills no whole panel
        _linear("linear_m33_w4a16_bias_gelu", "w4a16", 33, 4097, 4096, "bfloat16", act="gelu", bias=True, zp=True),
        # a 658-token prompt through gate and up, handed to the down projection in its own layout
        _linear("linear_m658_q4k_gated", "q4k", 658, 12288, 4096, "float16", layout="xf", act="silu", gated=True,
                out_layout="xf"),
        # a long prompt through a biased, tanh-GELU layer
        _linear("linear_m2048_w4a16_bias", "w4a16", 2048, 12288, 4096, "bfloat16", layout="xf", act="gelu_tanh",
                bias=True),
        # one new token's routing: 8 of 128 experts
        _route("route_t1_e128", 1, 128, 8, "float16"),
        # a 658-token prompt's routing, sigmoid scores, single-precision logits
        _route("route_t658_e128", 658, 128, 8, "float32", score="sigmoid", scale=2.5),
        # seven tokens routed elsewhere, a quarter of their pairs on another device's experts
        _group("group_t7_e128", 7, 128, 8, drop=0.25),
        # a long prompt's pairs grouped for the per-expert products
        _group("group_t8192_e128", 8192, 128, 8),
        # one new token through 8 of 128 experts
        _moe("moe_t1_e128", "q4k", "q6k", 1, 128, 8, 2048, 768, "float16"),
        # seven sequences over fewer, wider experts, some pairs on another device's experts
        _moe("moe_t7_e60_w4a16", "w4a16", "w4a16", 7, 60, 4, 2048, 1408, "bfloat16", residual=True, drop=0.25, zp=True),
        # sixty-four sequences: nearly every expert has a few rows
        _moe("moe_t64_e128", "q4k", "q6k", 64, 128, 8, 2048, 768, "bfloat16", residual=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(("linear", "linear", "linear", "moe", "moe", "route", "group"))
    if op == "linear":
        fmt = rng.choice(("q4k", "q6k", "w4a16"))
        step = 128 if fmt == "w4a16" else 256
        gated = rng.random() < 0.4
        M, N, K = _log(rng, 1, 2048), _log(rng, 16, 12288), step * _log(rng, 1, 12288 // step)
        if gated:
            N = 16 * max(1, N // 16)
        while M * N * K * (2 if gated else 1) > 1e11:  # no dearer than the largest listed case
            M = max(1, M // 2)
        out = "xf" if N >= 128 and rng.random() < 0.3 else "row"
        if out == "xf":
            N = 128 * (N // 128)
        return _linear(None, fmt, M, N, K, rng.choice(("float16", "bfloat16")), rng.choice(("row", "xf")),
                       rng.choice(_ACTS), gated, rng.random() < 0.5, rng.random() < 0.5, out,
                       rng.choice([g for g in (32, 64, 128, 256) if K % g == 0]), rng.random() < 0.5)
    if op == "moe":
        fu, fd = rng.choice((("q4k", "q6k"), ("q4k", "q4k"), ("q6k", "q6k"), ("w4a16", "w4a16"), ("w4a16", "q6k")))
        E = _log(rng, 2, 128)
        H = 256 * rng.randint(1, 16)
        I = (128 if fd == "w4a16" else 256) * rng.randint(1, 6)
        while E * H * I > 128 * 2048 * 768:
            E = max(2, E // 2)
        k = rng.randint(1, min(8, E))
        return _moe(None, fu, fd, _log(rng, 1, 64), E, k, H, I, rng.choice(("float16", "bfloat16")),
                    rng.choice(("silu", "silu", "gelu_tanh", "gelu", "relu")), rng.random() < 0.5,
                    rng.choice((0.0, 0.0, 0.3)), rng.choice((32, 64, 128)), rng.random() < 0.5)
    E = _log(rng, 2, 512)
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, 8192 * 8 // k // 2)
    if op == "route":
        return _route(None, min(T, 8192), E, k, rng.choice(("float16", "bfloat16", "float32")),
                      rng.choice(("softmax", "sigmoid")), rng.random() < 0.7, rng.choice((1.0, 2.5)))
    return _group(None, T, E, k, rng.choice((0.0, 0.25)))


# ---------------------------------------------------------------------------
# weights: logical fields, and their packed form
# ---------------------------------------------------------------------------

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _fields(fmt, N, K, group, zp, g):
    """Logical weight fields of N columns over K, drawn so that a product
    with N(0,1) activations has a spread of about two."""
    dev = dict(device="cuda", generator=g)
    amp = 2.0 / math.sqrt(K)
    if fmt == "q4k":
        nb = K // 256
        d = ((0.7 + 0.6 * torch.rand((N, nb), **dev)) * (amp / 184.0)).half()
        sc = torch.randint(16, 64, (N, nb, 8), dtype=torch.uint8, **dev)
        m = (sc.int() + torch.randint(-2, 3, (N, nb, 8), **dev)).clamp(0, 63).to(torch.uint8)
        return dict(d=d, dmin=(d.float() * 7.5).half(), sc=sc, m=m,
                    q=torch.randint(0, 16, (N, K), dtype=torch.uint8, **dev))
    if fmt == "q6k":
        nb = K // 256
        d = ((0.7 + 0.6 * torch.rand((N, nb), **dev)) * (amp / 1369.0)).half()
        return dict(d=d, s=torch.randint(-128, 128, (N, nb, 16), dtype=torch.int8, **dev),
                    q=torch.randint(0, 64, (N, K), dtype=torch.uint8, **dev))
    s = ((0.7 + 0.6 * torch.rand((K // group, N), **dev)) * (amp / 4.6)).half()
    z = torch.randint(6, 10, (K // group, N), dtype=torch.uint8, **dev) if zp else None
    return dict(s=s, z=z, q=torch.randint(0, 16, (N, K), dtype=torch.uint8, **dev))


def _pad_cols(t, dim=0):
    """Columns padded with zeros to whole panels of 16."""
    n = t.shape[dim]
    if n % 16 == 0:
        return t
    shape = list(t.shape)
    shape[dim] = 16 - n % 16
    return torch.cat([t, torch.zeros(shape, dtype=t.dtype, device=t.device)], dim)


def _code_words(q, N, K):
    """4-bit codes [Np*16][K] -> pair-order bytes [Np][K/128][4 runs][16 columns][16]."""
    Np = q.shape[0] // 16
    v = q.view(Np, 16, K // 128, 4, 4, 4, 2)  # [panel][col][chunk][run][word][pair][half]
    lo, hi = v[..., 0], v[..., 1]             # bits [4p, 4p+4) and [16+4p, 20+4p) of the word
    by = torch.stack([lo[..., 0] | (lo[..., 1] << 4), lo[..., 2] | (lo[..., 3] << 4),
                      hi[..., 0] | (hi[..., 1] << 4), hi[..., 2] | (hi[..., 3] << 4)], -1)
    return by.permute(0, 2, 3, 1, 4, 5).reshape(Np, K // 128, 4, 16, 16)


def _bytes(t):
    return t.contiguous().view(torch.uint8)


def _pack(fmt, f, N, K, group, zp):
    """The packed panel layout of one weight, a flat byte tensor."""
    if fmt == "w4a16":
        q = _pad_cols(f["q"])
        Np = q.shape[0] // 16
        parts = [_code_words(q, N, K).reshape(-1)]
        s = _pad_cols(f["s"], 1).view(K // group, Np, 16).permute(1, 0, 2)
        parts.append(_bytes(s).reshape(-1))
        if zp:
            z = _pad_cols(f["z"], 1).view(K // group, Np, 8, 2).permute(1, 0, 2, 3)
            parts.append((z[..., 0] | (z[..., 1] << 4)).reshape(-1))
        return torch.cat(parts)
    nb = K // 256
    q = _pad_cols(f["q"])
    Np = q.shape[0] // 16
    d = _bytes(_pad_cols(f["d"])).view(Np, 16, nb, 2)
    if fmt == "q4k":
        dmin = _bytes(_pad_cols(f["dmin"])).view(Np, 16, nb, 2)
        sc, m = (_pad_cols(f[n]).view(Np, 16, nb, 8) for n in ("sc", "m"))
        s12 = torch.cat([sc[..., :4] | ((sc[..., 4:] >> 4) << 6), m[..., :4] | ((m[..., 4:] >> 4) << 6),
                         (sc[..., 4:] & 15) | ((m[..., 4:] & 15) << 4)], -1)
        head = torch.cat([d, dmin, s12], -1).permute(0, 2, 1, 3).reshape(Np, nb, 256)
        codes = _code_words(q, N, K).reshape(Np, nb, 2048)
        return torch.cat([head, codes], -1).reshape(-1)
    s = _bytes(_pad_cols(f["s"])).view(Np, 16, nb, 16).permute(0, 2, 1, 3).reshape(Np, nb, 256)
    dd = d.permute(0, 2, 1, 3).reshape(Np, nb, 32)
    lo = _code_words(q & 15, N, K).reshape(Np, nb, 2048)
    # high pairs: word e of a run covers codes 16e .. 16e+15; code 8(2e+u)+2p+t at bit 16t + 2(4u+p)
    h = (q >> 4).view(Np, 16, K // 128, 4, 2, 2, 4, 2)  # [panel][col][chunk][run][e][u][p][t]
    by = h[..., 0, :] | (h[..., 1, :] << 2) | (h[..., 2, :] << 4) | (h[..., 3, :] << 6)  # [..][e][u][t]
    hi = by.transpose(-1, -2).permute(0, 2, 3, 1, 4, 5, 6).reshape(Np, nb, 1024)
    return torch.cat([dd, s, lo, hi], -1).reshape(-1)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _codes(by, Np, K):
    """Pair-order bytes -> codes [Np][16 columns][K]."""
    v = by.view(Np, K // 128, 4, 16, 4, 4)  # [panel][chunk][run][col][word][byte]
    lo = torch.stack([v[..., 0] & 15, v[..., 0] >> 4, v[..., 1] & 15, v[..., 1] >> 4], -1)
    hi = torch.stack([v[..., 2] & 15, v[..., 2] >> 4, v[..., 3] & 15, v[..., 3] >> 4], -1)
    q = torch.stack([lo, hi], -1)           # [..][word][pair][half]
    return q.permute(0, 3, 1, 2, 4, 5, 6).reshape(Np, 16, K)


def _unpack(fmt, wp, N, K, group, zp, dtype):
    """Packed weights of any number of leading matrices [B][bytes] -> float32
    [B][N][K], each weight rounded once into dtype."""
    B = wp.shape[0]
    n16 = (N + 15) // 16
    Np = B * n16
    if fmt == "w4a16":
        nc, ns = n16 * K * 8, n16 * (K // group) * 32
        q = _codes(wp[:, :nc].reshape(-1), Np, K)
        s = wp[:, nc:nc + ns].contiguous().view(torch.float16).view(Np, K // group, 16).permute(0, 2, 1).float()
        if zp:
            zb = wp[:, nc + ns:].reshape(Np, K // group, 8)
            z = torch.stack([zb & 15, zb >> 4], -1).view(Np, K // group, 16).permute(0, 2, 1).float()
        else:
            z = torch.full_like(s, 8.0)
        w = q.view(Np, 16, K // group, group).float().sub_(z[..., None]).mul_(s[..., None])
    elif fmt == "q4k":
        nb = K // 256
        rec = wp.view(Np, nb, 2304)
        head = rec[..., :256].reshape(Np, nb, 16, 16).permute(0, 2, 1, 3).contiguous()
        dm = head[..., :4].contiguous().view(torch.float16).float()
        s12 = head[..., 4:]
        sc = torch.cat([s12[..., :4] & 63, (s12[..., 8:] & 15) | ((s12[..., :4] >> 6) << 4)], -1).float()
        m = torch.cat([s12[..., 4:8] & 63, (s12[..., 8:] >> 4) | ((s12[..., 4:8] >> 6) << 4)], -1).float()
        q = _codes(rec[..., 256:].reshape(-1), Np, K).view(Np, 16, nb, 8, 32)
        w = q.float().mul_((dm[..., 0:1] * sc)[..., None]).sub_((dm[..., 1:2] * m)[..., None])
    else:
        nb = K // 256
        rec = wp.view(Np, nb, 3360)
        d = rec[..., :32].contiguous().view(torch.float16).permute(0, 2, 1).float()
        s = rec[..., 32:288].contiguous().view(torch.int8).view(Np, nb, 16, 16).permute(0, 2, 1, 3).float()
        lo = _codes(rec[..., 288:2336].reshape(-1), Np, K)
        hb = rec[..., 2336:].reshape(Np, nb * 2, 4, 16, 2, 2, 2)  # [panel][chunk][run][col][e][t][u]
        h = torch.stack([hb & 3, (hb >> 2) & 3, (hb >> 4) & 3, hb >> 6], -1)  # [..][e][t][u][p]
        h = h.permute(0, 3, 1, 2, 4, 6, 7, 5).reshape(Np, 16, K)
        q = (lo | (h << 4)).view(Np, 16, nb, 16, 16)
        w = q.float().sub_(32.0).mul_((d[..., None] * s)[..., None])
    w = w.reshape(B, n16 * 16, K)[:, :N]
    return w.to(dtype).float()


def _act(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _from_xf(xf, M, K):
    """Fragment-major copy -> row-major [M][K]."""
    v = xf.view(-1, K // 128, 8, 2, 32, 8)  # [block][chunk][k-step][half][row][8]
    return v.permute(0, 4, 1, 2, 3, 5).reshape(-1, K)[:M]


def _to_xf(x):
    """Row-major [M][K] -> fragment-major copy (rows padded with zeros to whole 32-row blocks)."""
    M, K = x.shape
    pad = -M % 32
    if pad:
        x = torch.cat([x, torch.zeros((pad, K), dtype=x.dtype, device=x.device)])
    return x.view(-1, 32, K // 128, 8, 2, 8).permute(0, 2, 3, 4, 1, 5).reshape(-1)


def _plain_linear(c, st):
    dt = _DT[c["dtype"]]
    N, K = c["N"], c["K"]
    x = (_from_xf(st["x"], c["M"], K) if c["layout"] == "xf" else st["x"]).float()
    nt = 2 * N if c["gated"] else N
    w = _unpack(c["fmt"], st["wp"].view(1, -1), nt, K, c["group"], c["zp"], dt)[0]
    y = x @ w.t()
    if c["bias"]:
        y = y + st["bias"].float()
    y = _act(y[:, :N], c["act"]) * y[:, N:] if c["gated"] else _act(y, c["act"])
    if c["residual"]:
        y = y + st["residual"].float()
    y = y.to(dt)
    return _to_xf(y) if c["out_layout"] == "xf" else y


def _plain_group(ids, E):
    flat = ids.reshape(-1)
    P = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E)).long()
    order = torch.sort(key, stable=True)[1]
    cnt = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offs = torch.cat([torch.zeros(1, dtype=torch.int64, device=ids.device), torch.cumsum(cnt[:E], 0)])
    live = torch.arange(P, device=ids.device) < offs[E]
    return offs.int(), torch.where(live, order, torch.full_like(order, -1)).int()


def _plain_route(c, logits):
    v = logits.float()
    top, ids = torch.sort(v, dim=1, descending=True, stable=True)
    top, ids = top[:, :c["k"]], ids[:, :c["k"]]
    if c["score"] == "softmax":
        mx = v.max(1, keepdim=True)[0]
        w = torch.exp(top - mx) / torch.exp(v - mx).sum(1, keepdim=True)
    else:
        w = 1 / (1 + torch.exp(-top))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    offs, rows = _plain_group(ids, c["E"])
    return ids.int(), w, offs, rows


def _plain_moe(c, st):
    dt = _DT[c["dtype"]]
    T, E, k, H, I = (c[n] for n in ("T", "E", "k", "H", "I"))
    x, ids, wt = st["x"].float(), st["ids"].long(), st["weights"]
    wu, wd = st["w_up"].view(E, -1), st["w_down"].view(E, -1)
    live = (ids >= 0) & (ids < E)
    wt = torch.where(live, wt, torch.zeros_like(wt))
    ids = torch.where(live, ids, torch.zeros_like(ids))
    if T * k <= E:  # each pair with its own expert's weights
        flat = ids.reshape(-1)
        g = _unpack(c["fmt_up"], wu[flat], 2 * I, H, c["group"], c["zp"], dt)
        h = torch.matmul(g, x.repeat_interleave(k, 0)[:, :, None])[..., 0]
        h = _act(h[:, :I], c["act"]) * h[:, I:]
        w = _unpack(c["fmt_down"], wd[flat], H, I, c["group"], c["zp"], dt)
        y = torch.matmul(w, h[:, :, None]).view(T, k, H)
        y = (y * wt[:, :, None]).sum(1)
    else:           # every token through every expert, weighted by its routing
        g = _unpack(c["fmt_up"], wu, 2 * I, H, c["group"], c["zp"], dt)
        h = torch.matmul(g, x.t().contiguous())  # [E][2I][T]
        h = _act(h[:, :I], c["act"]) * h[:, I:]
        w = _unpack(c["fmt_down"], wd, H, I, c["group"], c["zp"], dt)
        cw = torch.zeros((T, E), device=x.device).scatter_add_(1, ids, wt)
        y = torch.matmul(w, h * cw.t()[:, None, :]).sum(0).t()
    if c["residual"]:
        y = y + st["residual"].float()
    return y.to(dt)


# ---------------------------------------------------------------------------
# the measured calls
# ---------------------------------------------------------------------------

def _choose(T, E, k, drop, g):
    """k distinct experts per token, in falling order of a random preference;
    with drop, that share of the pairs has no expert here (-1)."""
    ids = torch.rand((T, E), device="cuda", generator=g).sort(1, descending=True)[1][:, :k].int()
    if drop:
        gone = torch.rand((T, k), device="cuda", generator=g) < drop
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.contiguous()


def prepare(case, seed):
    """Inputs and weights of one case on the GPU, from the seed alone."""
    c = case
    st = dict(case=c)
    g = _gen(seed, 1)
    if c["op"] == "linear":
        dt = _DT[c["dtype"]]
        nt = 2 * c["N"] if c["gated"] else c["N"]
        st["wp"] = _pack(c["fmt"], _fields(c["fmt"], nt, c["K"], c["group"], c["zp"], _gen(seed, 2)), nt, c["K"],
                         c["group"], c["zp"])
        x = torch.randn((c["M"], c["K"]), device="cuda", generator=g).to(dt)
        st["x"] = _to_xf(x) if c["layout"] == "xf" else x
        st["bias"] = torch.randn(nt, device="cuda", generator=g).mul_(0.5).to(dt) if c["bias"] else None
        st["residual"] = torch.randn((c["M"], c["N"]), device="cuda", generator=g).to(dt) if c["residual"] else None
    elif c["op"] == "moe":
        dt = _DT[c["dtype"]]
        E, H, I = c["E"], c["H"], c["I"]
        for key, fmt, N, K, salt in (("w_up", c["fmt_up"], 2 * I, H, 2), ("w_down", c["fmt_down"], H, I, 3)):
            gw = _gen(seed, salt)
            st[key] = torch.cat([_pack(fmt, _fields(fmt, N, K, c["group"], c["zp"], gw), N, K, c["group"], c["zp"])
                                 for _ in range(E)])
        st["x"] = torch.randn((c["T"], H), device="cuda", generator=g).to(dt)
        st["residual"] = torch.randn((c["T"], H), device="cuda", generator=g).to(dt) if c["residual"] else None
        st["ids"] = _choose(c["T"], E, c["k"], c["drop"], g)
        w = torch.rand((c["T"], c["k"]), device="cuda", generator=g) + 0.1
        st["weights"] = w / w.sum(1, keepdim=True)
        st["offsets"], st["rows"] = _plain_group(st["ids"], E)
    elif c["op"] == "route":
        # some experts are preferred by every token, as in a trained router
        v = 1.5 * torch.randn((c["T"], c["E"]), device="cuda", generator=g)
        v += 0.7 * torch.randn(c["E"], device="cuda", generator=g)
        st["logits"] = v.to(_DT[c["dtype"]])
    else:
        st["ids"] = _choose(c["T"], c["E"], c["k"], c["drop"], g)
    return st


def run(state):
    """One pass through the case's operator, and its outputs."""
    c = state["case"]
    if not own:
        if c["op"] == "linear":
            return _plain_linear(c, state)
        if c["op"] == "moe":
            return _plain_moe(c, state)
        if c["op"] == "route":
            return _plain_route(c, state["logits"])
        return _plain_group(state["ids"], c["E"])
    import quantized_weight_prefill_amd as qg

    if c["op"] == "linear":
        kw = dict(bias=state["bias"], residual=state["residual"], act=c["act"], gated=c["gated"], group=c["group"],
                  has_zp=c["zp"], out_layout=qg.X_FRAG if c["out_layout"] == "xf" else qg.X_ROW)
        if c["layout"] == "xf":
            return qg.linear_xf(c["fmt"], state["x"], state["wp"], c["M"], c["N"], c["K"], **kw)
        return qg.linear(c["fmt"], state["x"], state["wp"], c["N"], **kw)
    if c["op"] == "moe":
        return qg.moe(c["fmt_up"], c["fmt_down"], state["x"], state["w_up"], state["w_down"], state["weights"],
                      state["offsets"], state["rows"], c["I"], group=c["group"], has_zp=c["zp"], act=c["act"],
                      residual=state["residual"])
    if c["op"] == "route":
        return qg.moe_route(state["logits"], c["k"], score=c["score"], renorm=c["renorm"], scale=c["scale"])
    return qg.moe_group(state["ids"], c["E"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _weight_bytes(fmt, N, K, group, zp):
    if fmt == "q4k":
        return N * K * 144 / 256
    if fmt == "q6k":
        return N * K * 210 / 256
    return N * K / 2 + N * (K // group) * (2.5 if zp else 2)


def work(case):
    """Bytes and operations of one pass: each input read once, each output
    written once; of the experts' weights, those that some pair uses (the
    expected number, for uniform choices)."""
    c = case
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        nt = 2 * N if c["gated"] else N
        by = _weight_bytes(c["fmt"], nt, K, c["group"], c["zp"]) + 2 * M * K + 2 * M * N
        by += 2 * nt * c["bias"] + 2 * M * N * c["residual"]
        return {"bytes": by, "flops": 2.0 * M * nt * K}
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "moe":
        H, I = c["H"], c["I"]
        keep = 1.0 - c["drop"]
        active = E * (1.0 - (1.0 - keep * k / E) ** T)
        per = (_weight_bytes(c["fmt_up"], 2 * I, H, c["group"], c["zp"])
               + _weight_bytes(c["fmt_down"], H, I, c["group"], c["zp"]))
        by = active * per + 2 * T * H * (2 + c["residual"]) + T * k * 8 + 4 * (E + 1)
        return {"bytes": by, "flops": 6.0 * T * k * keep * H * I}
    if c["op"] == "route":
        size = 4 if c["dtype"] == "float32" else 2
        return {"bytes": T * E * size + 12 * T * k + 4 * (E + 1), "flops": 4.0 * T * E}
    return {"bytes": 8 * T * k + 4 * (E + 1), "flops": 2.0 * T * k}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _weights64(fmt, f, K, group, dtype):
    """float64 [N][K]: the format's formula on the logical fields, rounded into dtype."""
    q = f["q"].double()
    if fmt == "q4k":
        w = (q * (f["d"].double()[:, :, None] * f["sc"].double()).reshape(q.shape[0], -1).repeat_interleave(32, 1)
             - (f["dmin"].double()[:, :, None] * f["m"].double()).reshape(q.shape[0], -1).repeat_interleave(32, 1))
    elif fmt == "q6k":
        w = (q - 32) * (f["d"].double()[:, :, None] * f["s"].double()).reshape(q.shape[0], -1).repeat_interleave(16, 1)
    else:
        z = 8.0 if f["z"] is None else f["z"].double().t().repeat_interleave(group, 1)
        w = (q - z) * f["s"].double().t().repeat_interleave(group, 1)
    return w.to(dtype).double()


def _act64(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.erfc(v / -math.sqrt(2.0)) / 2
    if act == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8 / math.pi) * v * (1 + 0.044715 * v ** 2))
    return v


def _grouped64(ids, E):
    """Pairs by expert, in pair order, from host lists."""
    by = [[] for _ in range(E)]
    flat = ids.reshape(-1).tolist()
    for p, e in enumerate(flat):
        if 0 <= e < E:
            by[e].append(p)
    rows = [p for b in by for p in b]
    offs = [0]
    for b in by:
        offs.append(offs[-1] + len(b))
    rows += [-1] * (len(flat) - len(rows))
    as_int = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    return as_int(offs), as_int(rows)


def exact(case, seed):
    """What ``run`` returns, from the definition in 64 bits."""
    c = case
    st = prepare(case, seed)
    if c["op"] == "group":
        return _grouped64(st["ids"], c["E"])
    if c["op"] == "route":
        v = st["logits"].double().cpu()
        order = [sorted(range(c["E"]), key=lambda e, r=r: (-r[e], e))[:c["k"]] for r in v.tolist()]
        ids = torch.tensor(order, dtype=torch.int32)
        s = torch.softmax(v, 1) if c["score"] == "softmax" else torch.sigmoid(v)
        w = torch.gather(s, 1, ids.long())
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        offs, rows = _grouped64(ids, c["E"])
        return ids.cuda(), (w * c["scale"]).cuda(), offs, rows
    dt = _DT[c["dtype"]]
    if c["op"] == "linear":
        N, K = c["N"], c["K"]
        nt = 2 * N if c["gated"] else N
        w = _weights64(c["fmt"], _fields(c["fmt"], nt, K, c["group"], c["zp"], _gen(seed, 2)), K, c["group"], dt)
        x = (_from_xf(st["x"], c["M"], K) if c["layout"] == "xf" else st["x"]).double()
        y = x @ w.t()
        if c["bias"]:
            y = y + st["bias"].double()
        y = _act64(y[:, :N], c["act"]) * y[:, N:] if c["gated"] else _act64(y, c["act"])
        if c["residual"]:
            y = y + st["residual"].double()
        return _to_xf(y) if c["out_layout"] == "xf" else y
    T, E, H, I = c["T"], c["E"], c["H"], c["I"]
    y = st["residual"].double() if c["residual"] else torch.zeros((T, H), dtype=torch.float64, device="cuda")
    gu, gd = _gen(seed, 2), _gen(seed, 3)
    ids = st["ids"].tolist()
    for e in range(E):
        fu = _fields(c["fmt_up"], 2 * I, H, c["group"], c["zp"], gu)
        fd = _fields(c["fmt_down"], H, I, c["group"], c["zp"], gd)
        pairs = [(t, j) for t in range(T) for j in range(c["k"]) if ids[t][j] == e]
        if not pairs:
            continue
        t = torch.tensor([p[0] for p in pairs], device="cuda")
        j = torch.tensor([p[1] for p in pairs], device="cuda")
        h = st["x"].double()[t] @ _weights64(c["fmt_up"], fu, H, c["group"], dt).t()
        h = _act64(h[:, :I], c["act"]) * h[:, I:]
        o = h @ _weights64(c["fmt_down"], fd, I, c["group"], dt).t()
        y.index_add_(0, t, o * st["weights"].double()[t, j][:, None])
    return y
