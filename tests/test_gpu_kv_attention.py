"""Attention over the 4-bit cache on the GPU, against the 64-bit form of
tests/kv_ref.py on the values that the cache holds."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import quantized_weight_prefill_amd as qg
from tests import kv_ref as R
from tests.test_gpu_kv import BF16, F16, Pool, assert_within, i32, randn, table

pytestmark = pytest.mark.gpu


class Batch:
    """Sequences of `lens` tokens in a cache, `new` of each as queries."""

    def __init__(self, new, lens, heads, kv, D, page, dtype, seed=0, qscale=1.5, fill=0xA5, extra=0):
        S = len(lens)
        self.new, self.lens, self.kv, self.D, self.dtype = new, lens, kv, D, dtype
        self.pool = Pool(S, lens, kv, D, page, seed, fill=fill)
        n = sum(lens)
        self.k, self.v = randn((n, kv, D), seed + 1, dtype), randn((n, kv, D), seed + 2, dtype)
        off = np.cumsum([0] + lens).tolist()
        if n:
            qg.kv_append(self.pool.cache, self.k, self.v, self.pool.tables, i32(lens), offsets=i32(off))
        self.k64, self.v64 = R.held64(self.k), R.held64(self.v)
        self.start = off
        T = sum(new)
        self.q = randn((T + extra, heads, D), seed + 3, dtype, qscale)
        self.offsets = None if new == [1] * S and not extra else i32(np.cumsum([0] + new).tolist())

    def run(self, **kw):
        return qg.kv_attention(self.q, self.pool.cache, self.pool.tables, i32(self.lens), self.kv, offsets=self.offsets, **kw)

    def check(self, y, window=0, scale=None, what="", rows=None):
        row = 0
        for s, (n, length) in enumerate(zip(self.new, self.lens)):
            at = self.start[s]
            pick = list(range(n)) if rows is None else [i for i in range(n) if (row + i) in rows]
            if pick:
                want, err = R.attention64(self.q[row:row + n][pick], self.k64[at:at + length], self.v64[at:at + length],
                                          [length - n + i for i in pick], self.D ** -0.5 if scale is None else scale, window, self.dtype)
                assert_within(y[row:row + n][pick], want, err, f"{what} sequence {s}")
            row += n


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("heads,kv", [(8, 2), (3, 3), (6, 2), (5, 1), (16, 1), (40, 1), (7, 1), (17, 1)])
def test_decode_head_layouts(D, dtype, heads, kv):
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 65, 130, 0]
    b = Batch([1] * len(lens), lens, heads, kv, D, 32, dtype, seed=3)
    y = b.run()
    b.check(y)
    assert (y[-1] == 0).all()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 7, 16, 100])
def test_decode_pages_and_windows(page, window):
    b = Batch([1] * 5, [3, 50, 129, 300, 257], 8, 2, 128, page, F16, seed=5)
    b.check(b.run(window=window), window=window)


@pytest.mark.parametrize("lens", [[5000], [4096, 1, 700], [2049, 3100]])
@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F16)])
def test_decode_long(lens, D, dtype):
    """Lengths that are split over workgroups; a bound on the lengths changes the split, not the result's bound."""
    b = Batch([1] * len(lens), lens, 8, 2, D, 64, dtype, seed=7)
    for max_len in (0, 100, 1 << 20):
        b.check(b.run(max_len=max_len), what=f"max_len {max_len}")
    b.check(b.run(window=1500), window=1500)
    assert torch.equal(b.run(), b.run())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("heads,kv", [(8, 2), (4, 4), (6, 2), (14, 2)])
def test_prompts(D, dtype, heads, kv):
    """Ragged prompts and chunks behind earlier tokens, single tokens and empty sequences among them."""
    new = [1, 33, 0, 64, 5, 130, 1]
    lens = [1, 33, 20, 100, 205, 130, 77]
    b = Batch(new, lens, heads, kv, D, 32, dtype, seed=9, extra=5)
    out = torch.full_like(b.q, 9.0)
    y = b.run(out=out)
    assert y is out and (y[sum(new):] == 9).all()
    b.check(y)
    b.check(b.run(window=40), window=40)


@pytest.mark.parametrize("n", [2, 3, 4, 7, 8, 9, 16, 31, 65, 127, 257, 300])
def test_one_prompt_lengths(n):
    b = Batch([n], [n], 8, 2, 128, 64, F16, seed=11)
    b.check(b.run(), rows=set(range(0, n, 3)) | {n - 1, n - 2})


def test_long_prompt_rows():
    """A prompt of many tiles and a chunk behind a long context: some rows of each."""
    b = Batch([1500, 70], [1500, 4170], 4, 1, 128, 64, BF16, seed=13)
    rows = {0, 1, 63, 64, 65, 511, 512, 700, 1023, 1024, 1498, 1499, 1500, 1533, 1569}
    b.check(b.run(), rows=rows)
    b.check(b.run(window=600), window=600, rows=rows)
    one = Batch([40], [6000], 8, 1, 64, 128, F16, seed=14)
    one.check(one.run(), rows={0, 7, 38, 39})
    assert torch.equal(one.run(), one.run())


@pytest.mark.parametrize("new", [[1, 1, 1], [4, 1, 40]])
def test_rows_that_see_nothing(new):
    """Lengths of zero, shorter than the new tokens, pages that are none: zeros, and no neighbour is disturbed."""
    lens = [max(n, 20) for n in new]
    b = Batch(new, lens, 4, 2, 128, 16, F16, seed=15)
    want = b.run()
    cut = [0, 1, 1]
    y = qg.kv_attention(b.q, b.pool.cache, b.pool.tables, i32([lens[0], cut[1], cut[2]]), 2, offsets=b.offsets)
    assert torch.equal(y[:new[0]], want[:new[0]])
    row = new[0] + new[1]
    assert (y[row:row + new[2] - 1] == 0).all()
    assert (qg.kv_attention(b.q, b.pool.cache, torch.full_like(b.pool.tables, -1), i32(lens), 2, offsets=b.offsets) == 0).all()
    for bad in ([-3] * 3, [0] * 3, [-2 ** 31] * 3):
        assert (qg.kv_attention(b.q, b.pool.cache, b.pool.tables, i32(bad), 2, offsets=b.offsets) == 0).all()
    # the middle page of a sequence is none: its keys are not seen
    t = b.pool.tables.clone()
    t[2, 0] = 2 ** 31 - 1
    y = qg.kv_attention(b.q, b.pool.cache, t, i32(lens), 2, offsets=b.offsets)
    last = sum(new) - 1
    at = b.start[2]
    w, err = R.attention64(b.q[last:last + 1], b.k64[at + 16:at + lens[2]], b.v64[at + 16:at + lens[2]], [lens[2] - 17], 128 ** -0.5, 0, F16)
    assert_within(y[last:last + 1], w, err, "a page that is none")


@pytest.mark.parametrize("new,lens", [([1, 1], [19, 5]), ([19, 40], [19, 85])])
@pytest.mark.parametrize("fill", [0xFF, 0x7C])
def test_unwritten_cache_is_not_read(new, lens, fill):
    """Bytes behind the last token that read as NaN and infinities do not reach the result."""
    a, b = Batch(new, lens, 4, 2, 128, 64, F16, seed=17, fill=0), Batch(new, lens, 4, 2, 128, 64, F16, seed=17, fill=fill)
    y = b.run()
    assert torch.equal(y, a.run()) and y.isfinite().all()
    b.check(y)


def test_non_finite_queries_stay_in_their_rows():
    b = Batch([1, 30], [40, 50], 4, 2, 128, 32, BF16, seed=19)
    want = b.run()
    b.q[3, 1, 7] = float("nan")
    b.q[12, 2, 9] = float("inf")
    y = b.run()
    assert y[3, 1].isnan().all()
    keep = torch.ones(y.shape[:2], dtype=torch.bool)
    keep[3, 1] = keep[12, 2] = False
    assert torch.equal(y[keep], want[keep])


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("n", [1, 90])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_that_picks_one_token(dtype, n, D):
    """Keys of one direction each and sharp queries: the result is the picked token's value, rounded
    once, so that every code, header and order of dims is seen alone."""
    kv, heads, L = 2, 4, 90
    g = torch.Generator().manual_seed(23)
    k = torch.where(torch.rand((L, kv, D), generator=g) < 0.5, -1.0, 1.0)
    v = torch.randn((L, kv, D), generator=g)
    pool = Pool(1, [L], kv, D, 32)
    qg.kv_append(pool.cache, k.to(dtype).cuda(), v.to(dtype).cuda(), pool.tables, i32([L]), offsets=i32([0, L]))
    pick = torch.arange(L - n, L) if n > 1 else torch.tensor([37])
    pick = torch.stack([torch.randint(0, int(p) + 1, (heads,), generator=g) if n > 1 else torch.tensor([37, 0, 89, 16]) for p in pick])
    q = torch.stack([torch.stack([k[pick[i, h], h // 2] * 32 for h in range(heads)]) for i in range(n)]).to(dtype).cuda()
    y = qg.kv_attention(q, pool.cache, pool.tables, i32([L]), kv, offsets=None if n == 1 else i32([0, n]), scale=1.0)
    held = R.held64(v.to(dtype))
    want = torch.stack([torch.stack([held[pick[i, h], h // 2] for h in range(heads)]) for i in range(n)])
    # a key's own product is 32 D, another's at most 32 (D - 2 * the dims that differ): less than e^-40 of it in weight
    assert_within(y, want, R.store_err(want, 2.0 ** -11 * want.abs() + 2.0 ** -25, dtype))


def test_huge_and_tiny_queries():
    """Logits far beyond the exponential's range, and queries below fp16's."""
    for scale in (1e4, 1e-6, 1e30, 1e-30):
        b = Batch([1, 40], [50, 60], 4, 2, 128, 32, BF16, seed=25, qscale=scale)
        y = b.run()
        assert y.isfinite().all()
        if scale < 1:
            b.check(y, what=str(scale))


def test_strided_queries_and_streams():
    """Queries as columns of a merged product; explicit streams; a captured step replayed as lengths grow."""
    D, kv, heads, S = 128, 2, 8, 3
    b = Batch([1] * S, [70, 300, 1200], heads, kv, D, 64, F16, seed=27)
    merged = torch.zeros((S, (heads + 2 * kv) * D), dtype=F16, device="cuda")
    merged[:, :heads * D] = b.q.view(S, -1)
    y = b.run()
    args = (b.pool.cache, b.pool.tables)
    assert torch.equal(qg.kv_attention(merged[:, :heads * D].view(S, heads, D), *args, i32(b.lens), kv), y)
    raw = torch.cuda.Stream()
    raw.wait_stream(torch.cuda.current_stream())
    z = b.run(stream=raw.cuda_stream)
    raw.synchronize()
    assert torch.equal(z, y)
    lens = i32([1, 1, 1])
    call = lambda: qg.kv_attention(b.q, *args, lens, kv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):  # two graphs, each with its own workspace, replayed at once
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for length in (1, 70, 15, 64):
        lens.fill_(length)
        want = qg.kv_attention(b.q, *args, i32([length] * S), kv)
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out, want), length


def test_refusals():
    b = Batch([1, 1], [5, 6], 4, 2, 128, 16, F16, seed=29)
    for kw, what in ((dict(out=b.q), "shares memory"), (dict(out=b.q[:1]), "out"), (dict(out=b.q.to(BF16)), "out"),
                     (dict(window=-1), ""), (dict(max_len=-1), ""), (dict(scale=float("nan")), "")):
        with pytest.raises((ValueError, qg.QGemmError), match=what):
            b.run(**kw)
    with pytest.raises((ValueError, qg.QGemmError)):
        qg.kv_attention(b.q[:, :3], b.pool.cache, b.pool.tables, i32([5, 6]), 2)
    with pytest.raises(ValueError, match="device"):
        qg.kv_attention(b.q.cpu(), b.pool.cache, b.pool.tables, i32([5, 6]), 2)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
def test_attention_layer_in_a_run(dtype):
    """q/k/v product, append with norm and rotation, attention and output product: a prompt and then
    single tokens, as a whole against the same steps in 64 bits on the kernels' own intermediate
    values, and step by step against the whole sequence at once."""
    H, heads, kv, D, n, steps = 256, 4, 2, 128, 45, 6
    g = torch.Generator().manual_seed(31)

    def weight(N, K):
        s = (torch.rand((K // 64, N), generator=g) * 0.02 + 0.01).half().numpy().view(np.uint16)
        q = torch.randint(0, 16, (N, K), generator=g, dtype=torch.uint8).numpy()
        return torch.from_numpy(qg.w4a16_pack(q, s, None, N, K, 64)).cuda()

    nq = (heads + 2 * kv) * D
    wqkv, wo = weight(nq, H), weight(H, heads * D)
    x = randn((n + steps, H), 32, dtype)
    wq, wk = torch.ones(D, device="cuda"), (0.5 + torch.rand(D, generator=g)).cuda()
    rope = table(128, D)

    def layer(pool, rows, length, offsets):
        qkv = qg.linear("w4a16", rows, wqkv, nq, group=64)
        part = lambda lo, m: qkv[:, lo * D:(lo + m) * D].view(-1, m, D)
        q = qg.kv_append(pool.cache, part(heads, kv), part(heads + kv, kv), pool.tables, length, offsets=offsets, rope=rope,
                         k_weight=wk, eps=1e-6, q=part(0, heads), q_weight=wq)
        a = qg.kv_attention(q, pool.cache, pool.tables, length, kv, offsets=offsets)
        return qg.linear("w4a16", a.view(-1, heads * D), wo, H, group=64, residual=rows), q, a

    whole, stepped = (Pool(1, [n + steps], kv, D, 16) for _ in range(2))
    y, q, a = layer(whole, x, i32([n + steps]), i32([0, n + steps]))
    ks, vs = qg.kv_read(whole.cache, whole.tables, i32([n + steps]), n + steps, kv, D, offsets=i32([0, n + steps]))
    want, err = R.attention64(q, ks, vs, list(range(n + steps)), D ** -0.5, 0, dtype)
    assert_within(a, want, err)
    outs = [layer(stepped, x[:n], i32([n]), i32([0, n]))[0]]
    for i in range(steps):
        outs.append(layer(stepped, x[n + i:n + i + 1], i32([n + i + 1]), None)[0])
    got = torch.cat(outs).double()
    # products of other row counts add in another order, and a code may turn: within a few steps of the type's rounding of the whole
    rel = float((got - y.double()).norm() / y.double().norm())
    assert rel <= 8 * R.HALF[dtype], rel
