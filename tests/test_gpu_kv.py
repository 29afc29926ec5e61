"""Head norms with rotation, the append to the 4-bit cache and its read-back on
the GPU, against the 64-bit forms of tests/kv_ref.py."""
from __future__ import annotations

import random

import numpy as np
import pytest
import torch

import quantized_weight_prefill_amd as qg
from tests import kv_ref as R

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(shape, seed, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen(seed)) * scale).to(dtype).cuda()


def table(positions, rot, base=1e4):
    return torch.from_numpy(qg.rope_table(positions, rot, base)).cuda()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def assert_within(got, want, bound, what=""):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst {float((got - want).abs().max())}"


@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 128, True), (128, 64, False), (128, 16, True), (64, 64, False),
                                               (64, 16, False), (64, 64, True), (128, 0, False), (64, 48, False)])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T,heads,kv", [(1, 32, 8), (5, 3, 1), (37, 7, 7)])
def test_norm_rope(D, rot, interleaved, dtype, T, heads, kv):
    q, k = randn((T, heads, D), 1, dtype, 2.0), randn((T, kv, D), 2, dtype, 0.1)
    rope = table(300, rot) if rot else None
    pos = i32([(7 * t + 3) % 300 if t % 5 != 4 else (-1, 300, -2 ** 31, 2 ** 31 - 1)[t % 4] for t in range(T)]) if rot else None
    for weights, eps in ((True, 1e-6), (False, 1e-2), (True, None)):
        wq, wk = ((0.5 + torch.rand(D, generator=gen(3))).cuda(), torch.randn(D, generator=gen(4)).cuda()) if weights else (None, None)
        yq, yk = qg.qk_norm_rope(q, k, rope, pos, q_weight=wq, k_weight=wk, eps=eps, interleaved=interleaved)
        for x, w, y in ((q, wq, yq), (k, wk, yk)):
            want, mag = R.turn64(x, w, rope, pos, eps, interleaved)
            assert y.shape == x.shape and y.dtype == dtype
            assert_within(y, want, R.store_err(want, 24 * R.U32 * mag, dtype), f"weights={weights} eps={eps}")


@pytest.mark.parametrize("D", [64, 128])
def test_norm_rope_merged_rows_in_place(D):
    """Parts of one product's rows, rewritten where they are: the value columns stay."""
    T, heads, kv = 19, 6, 2
    qkv = randn((T, (heads + 2 * kv) * D), 5, BF16)
    before = qkv.clone()
    part = lambda b, lo, n: b[:, lo * D:(lo + n) * D].view(T, n, D)
    rope, pos = table(64, D), i32(list(range(T)))
    w = torch.ones(D, device="cuda")
    yq, yk = qg.qk_norm_rope(part(before, 0, heads), part(before, heads, kv), rope, pos, q_weight=w, k_weight=w)
    oq, ok = qg.qk_norm_rope(part(qkv, 0, heads), part(qkv, heads, kv), rope, pos, q_weight=w, k_weight=w,
                             q_out=part(qkv, 0, heads), k_out=part(qkv, heads, kv))
    assert torch.equal(oq, yq) and torch.equal(ok, yk) and oq.data_ptr() == qkv.data_ptr()
    assert torch.equal(part(qkv, heads + kv, kv), part(before, heads + kv, kv))
    only, none = qg.qk_norm_rope(part(before, 0, heads), None, rope, pos, q_weight=w)
    assert none is None and torch.equal(only, yq)
    with pytest.raises(ValueError, match="shares memory"):
        qg.qk_norm_rope(part(qkv, 0, heads), part(qkv, heads, kv), rope, pos, q_out=part(qkv, 1, heads))
    with pytest.raises(ValueError, match="positions"):
        qg.qk_norm_rope(part(qkv, 0, heads), None, rope)


def test_norm_rope_special_values():
    """Zero rows, subnormal, huge and non-finite elements: as the formula, row by row."""
    D = 128
    x = torch.zeros((6, 1, D), dtype=BF16)
    x[1] = 1e-40
    x[2, 0, 3] = 3e38
    x[3, 0, 5] = float("nan")
    x[4, 0, 7] = float("inf")
    x[5] = 1.0
    y, _ = qg.qk_norm_rope(x.cuda(), None, eps=1e-6)
    y = y.float().cpu()
    assert (y[0] == 0).all() and y[3].isnan().all() and y[4, 0, 7].isnan()
    assert y[1].abs().max() <= 1e-36 and (y[5] == 1).all()
    z, _ = qg.qk_norm_rope(x.cuda(), None, eps=None)
    assert torch.equal(z.cpu().view(torch.int16), x.view(torch.int16))


class Pool:
    """A cache whose pages are dealt out to sequences in a shuffled order."""

    def __init__(self, S, lens, kv, D, page, seed=0, spare=2, fill=0xA5):
        self.kv, self.D, self.page = kv, D, page
        need = [(n + page - 1) // page for n in lens]
        pages = sum(need) + spare
        order = list(range(pages))
        random.Random(seed).shuffle(order)
        width = max(need + [1])
        rows = []
        for n in need:
            rows.append([order.pop() for _ in range(n)] + [-1] * (width - n))
        self.tables = i32(rows).view(S, width)
        self.cache = qg.kv_cache(pages, kv, D, page).fill_(fill)

    def tokens(self, s, places):
        """Fields of some tokens, all heads: dict of arrays by (place, head)."""
        by, tb = self.cache.cpu().numpy(), self.tables.cpu().numpy()
        return {(p, h): R.token_fields(by, tb[s, p // self.page], self.kv, self.page, self.D, p, h) for p in places
                for h in range(self.kv)}


def check_tokens(pool, s, places, k64, v64):
    """The cache's fields of sequence s at `places` are the 64-bit form's of k64, v64 [n, kv, D]."""
    want = [R.quantize64(k64), R.quantize64(v64)]
    for (p, h), f in pool.tokens(s, places).items():
        i = places.index(p)
        for (c, sc, m, edge), (gc, gs, gm), what in ((want[0], f[:3], "key"), (want[1], f[3:], "value")):
            assert np.array_equal(gs, sc[i, h]) and np.array_equal(gm, m[i, h]), f"{what} header at {p}, head {h}"
            bad = (gc != c[i, h]) & (edge[i, h] > 1e-9)
            assert not bad.any(), f"{what} codes at {p}, head {h}: {np.argwhere(bad).ravel()[:8]}"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_append_prompt(D, dtype, page):
    """Ragged prompts into an empty cache, an empty one among them: fields, queries, read-back."""
    kv, heads = 2, 4
    new = [37, 0, 5, 1]
    T = sum(new)
    pool = Pool(4, new, kv, D, page)
    qkv = randn((T + 3, (heads + 2 * kv) * D), 11, dtype)  # three rows of no sequence behind the last
    part = lambda lo, n: qkv[:, lo * D:(lo + n) * D].view(T + 3, n, D)
    q, k, v = part(0, heads), part(heads, kv), part(heads + kv, kv)
    rope = table(64, D)
    wq, wk = (0.5 + torch.rand(D, generator=gen(6))).cuda(), (0.5 + torch.rand(D, generator=gen(7))).cuda()
    offs = i32(np.cumsum([0] + new).tolist())
    mark = torch.full((T + 3, heads, D), 7.0, dtype=dtype, device="cuda")
    y = qg.kv_append(pool.cache, k, v, pool.tables, i32(new), offsets=offs, rope=rope, k_weight=wk, eps=1e-6, q=q, q_weight=wq,
                     q_out=mark)
    pos = torch.tensor([p for n in new for p in range(n)])
    assert (y[T:] == 7).all()
    want, mag = R.turn64(q[:T], wq, rope, pos, 1e-6, False)
    assert_within(y[:T], want, R.store_err(want, 24 * R.U32 * mag, dtype), "queries")
    k64 = R.turn64(k[:T], wk, rope, pos, 1e-6, False)[0]
    v64 = v[:T].double().cpu()
    row = 0
    for s, n in enumerate(new):
        if n:
            check_tokens(pool, s, list(range(n)), k64[row:row + n], v64[row:row + n])
        row += n
    for dt in (torch.float32, F16, BF16):
        kr, vr = qg.kv_read(pool.cache, pool.tables, i32(new), T + 3, kv, D, offsets=offs, dtype=dt)
        for got, w in ((kr, R.held64(k64)), (vr, R.held64(v64))):
            assert got.dtype == dt and (got[T:] == 0).all()
            # the value itself is rounded to binary32 first
            assert_within(got[:T], w, R.store_err(w, 2.0 ** -24 * w.abs() + 2.0 ** -40, dt), f"read {dt}")


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, F16)])
def test_append_in_steps_is_append_at_once(D, dtype):
    """Chunks of every size mod 4, at every place mod 4, leave the bytes that one append leaves, and
    touch nothing else."""
    kv, page, n = 3, 32, 61
    k, v = randn((n, kv, D), 21, dtype), randn((n, kv, D), 22, dtype)
    rope = table(n, D)
    one = Pool(1, [n], kv, D, page)
    many = Pool(1, [n], kv, D, page)
    offs = i32([0, n])
    qg.kv_append(one.cache, k, v, one.tables, i32([n]), offsets=offs, rope=rope, eps=1e-6)
    done = 0
    for step in (1, 1, 2, 3, 4, 5, 1, 6, 7, 2, 8, 1, 1, 1, 9, 9):
        if step == 1:
            qg.kv_append(many.cache, k[done:done + 1], v[done:done + 1], many.tables, i32([done + 1]), rope=rope, eps=1e-6)
        else:
            qg.kv_append(many.cache, k[done:done + step], v[done:done + step], many.tables, i32([done + step]),
                         offsets=i32([0, step]), rope=rope, eps=1e-6)
        done += step
    assert done == n and torch.equal(one.cache, many.cache)
    # what no token of the sequence owns is as it was: spare pages, the tail of the last tile
    used = set(one.tables.cpu().view(-1).tolist())
    for p in range(one.cache.shape[0]):
        if p not in used:
            assert (one.cache[p] == 0xA5).all()
    last = one.cache[int(one.tables[0, -1])].view(kv, page // 16, 20 * D)[:, -1]
    for r in range(13, 16):  # 61 = 3 * 16 + 13
        for h in range(4):
            assert (last[:, (16 * h + r) * (D // 8):(16 * h + r + 1) * (D // 8)] == 0xA5).all()


def test_append_special_values():
    """NaN, infinities, groups of equal values, ties, subnormal spreads, values at the limits."""
    D, kv = 128, 1
    g = gen(33)
    x = torch.randn((14, kv, D), generator=g)
    x[0, 0, 5] = float("nan")
    x[1, 0, 6], x[1, 0, 70] = float("inf"), float("-inf")
    x[2] = 3.25
    x[3] = 0.0
    x[4] = torch.arange(D) % 16 + 0.5           # scale 1: codes exactly
    x[5] = (torch.arange(D) % 31) * 0.5         # scale 1, ties at every second value
    x[6] *= 1e-7
    x[7] *= 1e30
    x[8] = torch.where(torch.arange(D) % 2 == 0, 40000.0, -40000.0)
    x[9, 0, 31] = 1000.0
    x[10] = 1000.0 + torch.arange(D) % 16
    x[11] = -torch.arange(D).float()
    x[12] = torch.where(torch.arange(D) == 64, 1.0, 0.0)
    for dtype in (BF16, F16):
        y = x.to(dtype).cuda()
        pool = Pool(1, [14], kv, D, 16, fill=0xFF)
        qg.kv_append(pool.cache, y, y.flip(0).contiguous(), pool.tables, i32([14]), offsets=i32([0, 14]))
        check_tokens(pool, 0, list(range(14)), y.double().cpu(), y.flip(0).double().cpu())
        k, v = qg.kv_read(pool.cache, pool.tables, i32([14]), 14, kv, D, offsets=i32([0, 14]))
        assert k.isfinite().all() and v.isfinite().all() and k.abs().max() <= 32816


def test_append_header_rounding():
    """A minimum that binary32 rounds onto an fp16 tie: rounded twice, as the header says."""
    D, kv = 64, 1
    tiny = 2.0 ** -11 + 2.0 ** -31
    rope = torch.zeros((1, D), device="cuda")
    rope[:, :D // 2], rope[:, D // 2:] = 1.0, tiny
    k = torch.zeros((1, kv, D), dtype=F16, device="cuda")
    k[0, 0, 0], k[0, 0, 1] = -1.0, 1.0      # dim 0 becomes -(1 + tiny), the first group's minimum
    pool = Pool(1, [1], kv, D, 16)
    qg.kv_append(pool.cache, k, k, pool.tables, i32([1]), rope=rope, interleaved=True)
    k64 = R.turn64(k, None, rope, i32([0]), None, True)[0]
    assert float(k64[0, 0, 0]) == -1.0 - tiny
    check_tokens(pool, 0, [0], k64, k.double().cpu())
    assert float(pool.tokens(0, [0])[(0, 0)][2][0]) == -1.0


def test_append_places_outside():
    """Positions outside the rotation's table, pages that are none, lengths beyond the table, rows before
    the first place, offsets of any contents: left out, nothing else touched."""
    D, kv, page, T = 128, 2, 16, 24
    k = randn((T, kv, D), 41, F16)
    base = qg.kv_cache(6, kv, D, page).fill_(0x5A)

    def left(tables, lens, offsets, **kw):
        c = base.clone()
        qg.kv_append(c, k, k, i32(tables), i32(lens), offsets=i32(offsets), **kw)
        kr, vr = qg.kv_read(c, i32(tables), i32(lens), T, kv, D, offsets=i32(offsets))
        return c, kr, vr

    held = R.held64(k.double().cpu()).float().cuda()
    # the second page is none
    c, kr, vr = left([[3, 6]], [24], [0, 24])
    assert torch.equal(kr[:16], held[:16]) and (kr[16:] == 0).all() and torch.equal(vr[:16], held[:16])
    assert all((c[p] == 0x5A).all() for p in range(6) if p != 3)
    for bad in (-1, 2 ** 31 - 1, -2 ** 31):
        c, _, _ = left([[bad, bad]], [24], [0, 24])
        assert torch.equal(c, base)
    # length beyond the table: only the places inside are written; before the first place: left out
    c, kr, _ = left([[2]], [20], [0, 24])
    assert (kr[:4] == 0).all() and torch.equal(kr[4:20], held[4:20]) and (kr[20:] == 0).all()
    for lens in ([0], [-5], [2 ** 31 - 1], [-2 ** 31]):
        c, _, _ = left([[2]], lens, [0, 24])
        assert torch.equal(c, base)
    # rows of no sequence; offsets that are no offsets
    c, kr, _ = left([[2], [4]], [3, 2], [0, 3, 5])
    assert torch.equal(kr[:5], held[:5]) and (kr[5:] == 0).all()
    for offsets in ([-7, 2 ** 31 - 1, -2 ** 31], [30, 3, 40], [5, 5, 5]):
        left([[2], [4]], [3, 2], offsets)
    # a position without a line in the table
    pos = i32([0, 1, 64, -1] + list(range(4, T)))
    c, kr, _ = left([[0, 1]], [24], [0, 24], rope=table(64, D), positions=pos)
    clean, _, _ = left([[0, 1]], [24], [0, 24], rope=table(65, D), positions=i32(list(range(T))))
    by = lambda cache: [R.token_fields(cache.cpu().numpy(), p // 16, kv, page, D, p, 1) for p in range(T)]
    for p, (a, b, old) in enumerate(zip(by(c), by(clean), by(torch.cat([base, base])))):
        for f, w in zip(a, old if p in (2, 3) else b):
            assert f.tobytes() == w.tobytes(), p


def test_kv_refusals():
    D, kv = 128, 2
    k = randn((4, kv, D), 51, F16)
    pool = Pool(4, [1] * 4, kv, D, 16)
    lens = i32([1] * 4)
    ok = lambda **kw: qg.kv_append(**{**dict(cache=pool.cache, k=k, v=k, tables=pool.tables, lens=lens), **kw})
    ok()
    for kw, what in ((dict(v=k[:, :1]), "shape"), (dict(v=k.to(BF16)), "dtype"), (dict(lens=lens[:3]), "lens"),
                     (dict(lens=lens.long()), "lens"), (dict(tables=pool.tables[:3]), "offsets"), (dict(cache=pool.cache[0]), "cache"),
                     (dict(offsets=i32([0, 4])), "offsets"), (dict(k=k.transpose(0, 1)), ""), (dict(q=k[:3]), "rows"),
                     (dict(q_out=k), "without q"), (dict(q=k, q_out=k[:, :1]), "shape"), (dict(q=k, q_out=k), "shares memory"),
                     (dict(positions=lens[:2]), "positions"), (dict(k_weight=torch.ones(64, device="cuda")), "k_weight"),
                     (dict(k=pool.cache.view(F16).view(-1)[:4 * kv * D].view(4, kv, D)), "shares memory"),
                     (dict(rope=torch.ones((4, 100), device="cuda")), "")):
        with pytest.raises((ValueError, qg.QGemmError), match=what):
            ok(**kw)


def test_append_captured_and_on_streams():
    """A captured decode step replayed as the lengths grow; calls on an explicit stream."""
    D, kv, S = 128, 2, 3
    n = 9
    k, v, q = (randn((n, S, h, D), 61 + h, BF16) for h in (kv, kv, 4)[0:3])
    v = randn((n, S, kv, D), 70, BF16)
    rope = table(64, D)
    eager, cap = Pool(S, [n] * S, kv, D, 16), Pool(S, [n] * S, kv, D, 16)
    ks, vs, qs, lens = k[0].clone(), v[0].clone(), q[0].clone(), i32([1] * S)
    step = lambda: qg.kv_append(cap.cache, ks, vs, cap.tables, lens, rope=rope, eps=1e-6, q=qs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step()
    for i in range(n):
        ks.copy_(k[i]), vs.copy_(v[i]), qs.copy_(q[i]), lens.fill_(i + 1)
        g.replay()
        want = qg.kv_append(eager.cache, k[i], v[i], eager.tables, i32([i + 1] * S), rope=rope, eps=1e-6, q=q[i], stream=0)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(cap.cache, eager.cache), i
    raw = torch.cuda.Stream()
    raw.wait_stream(torch.cuda.current_stream())
    a = qg.qk_norm_rope(q[0], k[0], rope, i32([5] * S), stream=raw.cuda_stream)
    r = qg.kv_read(eager.cache, eager.tables, i32([n] * S), S, kv, D, stream=raw.cuda_stream)
    raw.synchronize()
    b = qg.qk_norm_rope(q[0], k[0], rope, i32([5] * S))
    w = qg.kv_read(eager.cache, eager.tables, i32([n] * S), S, kv, D)
    assert all(torch.equal(x, y) for x, y in zip(a + r, b + w))


def test_nothing_to_do():
    D, kv = 64, 2
    pool = Pool(1, [1], kv, D, 16)
    z = torch.empty((0, kv, D), dtype=F16, device="cuda")
    none = torch.empty((0, 1), dtype=torch.int32, device="cuda")
    before = pool.cache.clone()
    assert qg.qk_norm_rope(z, z)[0].shape == (0, kv, D)
    assert qg.kv_append(pool.cache, z, z, none, none[:, 0], q=z).shape == (0, kv, D)
    assert qg.kv_append(pool.cache, z, z, pool.tables, i32([1]), offsets=i32([0, 0])) is None
    assert qg.kv_read(pool.cache, none, none[:, 0], 0, kv, D)[0].shape == (0, kv, D)
    assert qg.kv_attention(z, pool.cache, none, none[:, 0], kv).shape == (0, kv, D)
    assert torch.equal(pool.cache, before)
