"""Attention over the 4-bit cache, its append and their binding at the ends of tables, windows, batches and number
ranges, against the 64-bit forms of tests/kv_ref.py."""
from __future__ import annotations

import pytest
import torch

import quantized_weight_prefill_amd as qg
from tests import kv_ref as R
from tests.test_gpu_kv import BF16, F16, Pool, assert_within, i32, randn, table
from tests.test_gpu_kv_attention import Batch

pytestmark = pytest.mark.gpu


def check_behind_table(q, y, k64, v64, cap, length, window, dtype, rows, what):
    """Rows of one sequence of `length` tokens, of which the table has places for `cap`."""
    n = q.shape[0]
    for i in rows:
        p = length - n + i
        lo = max(0, p - window + 1) if window else 0
        if p < 0 or lo >= min(p + 1, cap):
            assert (y[i] == 0).all(), f"{what} row {i}"
            continue
        want, err = R.attention64(q[i:i + 1], k64[:cap], v64[:cap], [p], q.shape[2] ** -0.5, window, dtype)
        assert_within(y[i:i + 1], want, err, f"{what} row {i}")


@pytest.mark.parametrize("page,width,n,heads,kv", [
    (16, 5, 40, 8, 2), (32, 3, 40, 8, 2), (16, 3, 300, 4, 2), (32, 1, 40, 4, 1),  # four waves of 32 rows
    (16, 21, 40, 8, 2), (32, 27, 300, 8, 2),                                      # two waves to 32 rows
    (16, 189, 70, 8, 2),                                                          # and parts of the keys
    (16, 45, 700, 96, 12),                                                        # eight waves
    (16, 5, 6, 8, 2), (32, 3, 1, 8, 2),                                           # a few rows
])
@pytest.mark.parametrize("D,dtype", [(128, F16), (64, BF16)])
def test_lengths_past_the_table(page, width, n, heads, kv, D, dtype):
    """Places behind the table are not seen, wherever a tile of keys ends; a single token of the same place agrees."""
    cap = page * width
    b = Batch([n], [cap], heads, kv, D, page, dtype, seed=81)
    assert b.pool.tables.shape == (1, width)
    b.q = randn((n, heads, D), 82, dtype, 1.5)
    off = i32([0, n])
    rows = sorted({0, 1, n // 3, n // 2, n - 2, n - 1} & set(range(n)))
    for length in (cap - 1, cap, cap + 1, cap + 17, cap + n // 2, cap + n + 9, cap + 63, cap + 5000):
        for window in (0, n + 30):
            call = lambda q, o: qg.kv_attention(q, b.pool.cache, b.pool.tables, i32([length]), kv, offsets=o, window=window)
            check_behind_table(b.q, call(b.q, off), b.k64, b.v64, cap, length, window, dtype, rows, f"length {length}, window {window}")
            check_behind_table(b.q[-1:], call(b.q[-1:], None), b.k64, b.v64, cap, length, window, dtype, [0], f"single token, length {length}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv_heads", [2 ** 58, 2 ** 60, 2 ** 61, 2 ** 62, 2 ** 63 - 1, 65537, 0, -1, -2 ** 61])
def test_numbers_of_key_heads_that_wrap_around(kv_heads, D):
    """Refused, whatever their product with the bytes of a head comes to in 64 bits."""
    pool = Pool(1, [5], 2, D, 16)
    q = randn((1, 4, D), 83, F16)
    with pytest.raises(ValueError, match="page"):
        qg.kv_read(pool.cache, pool.tables, i32([5]), 1, kv_heads, D)
    with pytest.raises(ValueError, match="page"):
        qg.kv_attention(q, pool.cache, pool.tables, i32([5]), kv_heads)
    for head_dim in (2 ** 62, 2 ** 59, 0, -D):
        with pytest.raises((ValueError, qg.QGemmError)):
            qg.kv_read(pool.cache, pool.tables, i32([5]), 1, 2, head_dim)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 2 ** 31 - 30, 2 ** 40])
@pytest.mark.parametrize("n,heads", [(8, 4), (40, 4), (300, 8)])
def test_windows_wider_than_any_length(n, heads, window):
    """Also behind rows that have no place in their sequence: what no window gives."""
    b = Batch([n], [n], heads, 2, 128, 16, BF16, seed=84)
    b.offsets = i32([0, n])
    for length in (5, n - 1, n):
        call = lambda **kw: qg.kv_attention(b.q, b.pool.cache, b.pool.tables, i32([length]), 2, offsets=b.offsets, **kw)
        want = call()
        assert (want[n - 1] != 0).any() and (want[:n - length] == 0).all()
        assert torch.equal(call(window=window), want), length


@pytest.mark.parametrize("D,dtype", [(128, F16), (64, BF16)])
@pytest.mark.parametrize("new,window,length", [(1, 20, 100), (1, 500, 3000), (6, 30, 133), (40, 20, 150), (40, 100, 3050), (300, 77, 700)])
def test_places_before_the_window_need_not_be_written(D, dtype, new, window, length):
    """A sequence of which only what some window sees was appended, in a cache of bytes that read as NaN."""
    whole = Batch([new], [length], 8, 2, D, 64, dtype, seed=85)
    first = length - new - window + 1  # the first place that a row sees
    part = Pool(1, [length], 2, D, 64, 85, fill=0xFF)
    qg.kv_append(part.cache, whole.k[first:], whole.v[first:], part.tables, i32([length]), offsets=i32([0, length - first]))
    whole.offsets = None if new == 1 else i32([0, new])
    want = whole.run(window=window)
    whole.check(want, window=window, rows={0, new // 2, new - 1})
    y = qg.kv_attention(whole.q, part.cache, part.tables, i32([length]), 2, offsets=whole.offsets, window=window)
    assert torch.equal(y, want)


def poison(shape, dtype):
    """Free memory of a result's size that reads as NaN, for the allocator to hand out next."""
    x = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    del x


# rows before the first sequence, of each, and behind the last; lengths
RESTS = [
    (0, [1], 3, [20]), (2, [1, 2], 3, [30, 20]),       # a few rows
    (0, [40], 9, [40]), (5, [40, 1, 0], 70, [90, 30, 9]),  # prompts and single tokens
    (0, [700], 324, [700]), (300, [1], 20, [50]),
    (3, [70], 90, [3000]), (1, [1, 1], 62, [5000, 700]),   # parts of the keys
]


@pytest.mark.parametrize("before,new,behind,lens", RESTS)
@pytest.mark.parametrize("D,dtype", [(128, F16), (64, BF16)])
def test_rows_of_no_sequence_are_zeros_in_new_results(before, new, behind, lens, D, dtype):
    """What the library allocates is written whole; a result that the caller brings keeps those rows."""
    b = Batch(new, lens, 8, 2, D, 32, dtype, seed=86)
    T = before + sum(new) + behind
    off = [before]
    for m in new:
        off.append(off[-1] + m)
    b.offsets, b.q = i32(off), randn((T, 8, D), 87, dtype)
    own = slice(before, T - behind)
    marked = torch.full_like(b.q, 9.0)
    b.run(out=marked)
    assert (marked[:before] == 9).all() and (marked[own] != 9).any() and (marked[T - behind:] == 9).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in ({}, dict(stream=side.cuda_stream)):
        poison(b.q.shape, dtype)
        y = b.run(**kw)
        side.synchronize()
        assert torch.equal(y[own], marked[own]) and (y[:before] == 0).all() and (y[T - behind:] == 0).all()
    k, v = randn((T, 2, D), 88, dtype), randn((T, 2, D), 89, dtype)
    rope = table(6000, D)
    call = lambda **kw: qg.kv_append(b.pool.cache, k, v, b.pool.tables, i32(lens), offsets=b.offsets, rope=rope, eps=1e-6, q=b.q, **kw)
    marked = torch.full_like(b.q, 9.0)
    call(q_out=marked)
    assert (marked[:before] == 9).all() and (marked[own] != 9).any() and (marked[T - behind:] == 9).all()
    for kw in ({}, dict(stream=side.cuda_stream)):
        poison(b.q.shape, dtype)
        y = call(**kw)
        side.synchronize()
        assert torch.equal(y[own], marked[own]) and (y[:before] == 0).all() and (y[T - behind:] == 0).all()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
def test_no_sequence_at_all_gives_zeros(dtype):
    pool = Pool(1, [20], 2, 64, 16)
    none = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    x = randn((37, 2, 64), 90, dtype)
    for o in (i32([0]), i32([37])):
        poison(x.shape, dtype)
        assert (qg.kv_attention(x, pool.cache, none, none[:, 0], 2, offsets=o) == 0).all()
        poison(x.shape, dtype)
        assert (qg.kv_append(pool.cache, x, x, none, none[:, 0], offsets=o, q=x) == 0).all()
    empty = i32([0, 0])  # a sequence without new rows
    poison(x.shape, dtype)
    assert (qg.kv_attention(x, pool.cache, pool.tables, i32([20]), 2, offsets=empty) == 0).all()
    poison(x.shape, dtype)
    assert (qg.kv_append(pool.cache, x, x, pool.tables, i32([20]), offsets=empty, q=x) == 0).all()


def test_captured_batches_that_shrink():
    """A padded step in a graph, replayed with fewer rows each time: no row of an earlier replay is left."""
    D, T = 128, 96
    b = Batch([60, 30], [600, 300], 8, 2, D, 32, BF16, seed=91)
    b.q = randn((T, 8, D), 92, BF16)
    k, v = randn((T, 2, D), 93, BF16), randn((T, 2, D), 94, BF16)
    off, lens = i32([0, 60, 90]), i32([600, 300])

    def step():
        q = qg.kv_append(b.pool.cache, k, v, b.pool.tables, lens, offsets=off, eps=1e-6, q=b.q)
        return q, qg.kv_attention(q, b.pool.cache, b.pool.tables, lens, 2, offsets=off)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for o in ([0, 60, 90], [0, 50, 51], [4, 5, 6], [0, 0, 0], [0, 1, 96]):
        off.copy_(i32(o))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        torch.cuda.synchronize()
        for x, w in zip(got, want):
            assert torch.equal(x, w) and (x[o[2]:] == 0).all() and (x[:o[0]] == 0).all(), o


def equal_weights(L, n, heads, D, seed):
    """A sequence whose keys are 48 vectors in turn, and queries at right angles to all their differences: every key that a
    row sees weighs the same, while one fp16 rounding of the keys would move the products by many times what the result's own
    rounding leaves."""
    b = Batch([n], [L], heads, 1, D, 32, F16, seed=seed)
    b.k = b.k[:48][torch.arange(L, device="cuda") % 48].contiguous()
    qg.kv_append(b.pool.cache, b.k, b.v, b.pool.tables, i32([L]), offsets=i32([0, L]))
    b.k64 = R.held64(b.k)
    basis = torch.linalg.svd(b.k64[1:48, 0] - b.k64[:1, 0])[2][47:]
    g = torch.Generator().manual_seed(seed + 1)
    b.q = (12 * torch.randn((n, heads, len(basis)), generator=g, dtype=torch.float64) @ basis).to(F16).cuda()
    return b


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L,n,window,rows", [
    (900, 300, 512, range(0, 300, 7)),    # every row sees 512 keys, a tile of rows more
    (900, 300, 500, range(0, 300, 7)),
    (900, 9, 510, range(9)),
    (530, 40, 0, range(0, 22)),           # a tile of rows that see up to 512 keys, and of others
    (516, 9, 0, range(0, 5)),
])
def test_rows_of_few_keys_keep_fp16_precision_beside_any_others(D, L, n, window, rows):
    """What a row sees decides, not what its tile's other rows see: the bound of 512 keys is the row's own. Values and
    weights are each off by at most the relative half step that the result's rounding has at worst, twice the least that it
    has: the error is below sqrt(1 + 4 + 4) of the result's own rounding."""
    b = equal_weights(L, n, 4, D, 95)
    y = b.run(window=window).double().cpu()
    rows = list(rows)
    want, _ = R.attention64(b.q[rows], b.k64, b.v64, [L - n + i for i in rows], D ** -0.5, window, F16)
    own = (want.to(F16).double() - want).norm()
    assert (y[rows] - want).norm() < 3 * own


def test_one_result_for_every_row_is_refused():
    """Rows that share one place cannot be written."""
    q, k = randn((3, 4, 64), 96, F16), randn((3, 2, 64), 97, F16)
    one = torch.empty((1, 4, 64), dtype=F16, device="cuda").expand(3, 4, 64)
    for x in (q, q[:1].expand(3, 4, 64), one):
        with pytest.raises((ValueError, qg.QGemmError)):
            qg.qk_norm_rope(x, k, q_out=one)
    pool = Pool(3, [1] * 3, 2, 64, 16)
    for x in (q, q[:1].expand(3, 4, 64), one):
        with pytest.raises((ValueError, qg.QGemmError)):
            qg.kv_append(pool.cache, k, k, pool.tables, i32([1] * 3), q=x, q_out=one)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 6, 90])
@pytest.mark.parametrize("scale", [2.0 ** 12, 2.0 ** 18, 2.0 ** 40])
def test_products_far_beyond_the_exponential(dtype, D, n, scale):
    """Keys of +-1 and queries that are one of them, with products from 2^21 to 2^50 in log2 units: every other key's weight is 0
    in any arithmetic, so the result is the picked key's value, or where two keys are alike the mean of their values, each
    rounded once. Values are off by 2^-11 of each and half a subnormal step, the sum and its quotient by 2^-22."""
    kv, heads, L = 2, 4, 300
    g = torch.Generator().manual_seed(98)
    k = torch.where(torch.rand((L, kv, D), generator=g) < 0.5, -1.0, 1.0)
    twins = {L - 1: 17, 40: 3}
    for a, b in twins.items():
        k[a] = k[b]
    twins.update({b: a for a, b in list(twins.items())})
    v = torch.randn((L, kv, D), generator=g)
    pool = Pool(1, [L], kv, D, 32)
    qg.kv_append(pool.cache, k.to(dtype).cuda(), v.to(dtype).cuda(), pool.tables, i32([L]), offsets=i32([0, L]))
    held = R.held64(v.to(dtype))
    place = [L - n + i for i in range(n)]
    pick = [[(7 * i + 31 * h) % (p + 1) for h in range(heads)] for i, p in enumerate(place)]
    pick[-1] = [L - 1, 40, 3, 17]
    for sign in (1.0, -1.0):  # a negative scale turns the order around: the same result of negated queries
        q = torch.stack([torch.stack([sign * 8 * k[pick[i][h], h // 2] for h in range(heads)]) for i in range(n)])
        y = qg.kv_attention(q.to(dtype).cuda(), pool.cache, pool.tables, i32([L]), kv, offsets=None if n == 1 else i32([0, n]),
                            scale=sign * scale)
        want, mag = torch.zeros((n, heads, D), dtype=torch.float64), torch.zeros((n, heads, D), dtype=torch.float64)
        for i in range(n):
            for h in range(heads):
                a = pick[i][h]
                both = [a] + ([twins[a]] if twins.get(a, L) <= place[i] else [])
                want[i, h] = held[both, h // 2].mean(0)
                mag[i, h] = held[both, h // 2].abs().mean(0)
        assert_within(y, want, R.store_err(want, (2.0 ** -11 + 2.0 ** -22) * mag + 2.0 ** -25, dtype), f"sign {sign}")


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("n", [1, 6, 90])
def test_products_far_below_zero(dtype, n):
    """Every product is the same, from -2^21 to -2^50 in log2 units: all keys weigh the same. A weight is the same number for all
    keys of a row, so the result is off by the values' roundings, 2^-23 for each key's sums and the store's."""
    D, kv, heads, L = 128, 2, 4, 150
    pool = Pool(1, [L], kv, D, 32)
    k = torch.ones((L, kv, D), dtype=dtype, device="cuda")
    v = randn((L, kv, D), 99, dtype)
    qg.kv_append(pool.cache, k, v, pool.tables, i32([L]), offsets=i32([0, L]))
    held = R.held64(v)
    q = torch.full((n, heads, D), -1.0, dtype=dtype, device="cuda")
    for scale in (2.0 ** 14, 2.0 ** 21, 2.0 ** 43):
        y = qg.kv_attention(q, pool.cache, pool.tables, i32([L]), kv, offsets=None if n == 1 else i32([0, n]), scale=scale)
        for i in range(n):
            m = L - n + i + 1
            want, mag = (x[:m].mean(0).repeat_interleave(heads // kv, 0)[None] for x in (held, held.abs()))
            bound = R.store_err(want, (2.0 ** -11 + m * 2.0 ** -23) * mag + 2.0 ** -25, dtype)
            assert_within(y[i:i + 1], want, bound, f"scale {scale} row {i}")


@pytest.mark.parametrize("new,lens,heads", [([1] * 4, [300, 1, 700, 2100], 8), ([40], [40], 8), ([300, 1, 5], [300, 90, 1200], 8),
                                            ([658], [700], 32), ([600], [2600], 64)])
@pytest.mark.parametrize("D,dtype", [(128, F16), (64, BF16)])
def test_tables_wider_than_the_lengths(new, lens, heads, D, dtype):
    """Entries behind a sequence's pages are not followed, whatever they name; the split that their number leads to, and the
    one that max_len gives, keep the result within its bound."""
    kv = heads // 4
    b = Batch(new, lens, heads, kv, D, 64, dtype, seed=111)
    rows = set(range(0, sum(new), 1 + sum(new) // 24)) | {sum(new) - 1}
    narrow = b.pool.tables
    for entry in (-1, 0, 2 ** 31 - 1):
        b.pool.tables = torch.cat([narrow, torch.full((len(lens), 512 - narrow.shape[1]), entry, dtype=torch.int32, device="cuda")], 1)
        for s, n in enumerate(lens):
            b.pool.tables[s, (n + 63) // 64:] = entry
        for kw in ({}, dict(max_len=max(lens)), dict(window=70)):
            b.check(b.run(**kw), window=kw.get("window", 0), what=f"entries {entry}, {kw}", rows=rows)
