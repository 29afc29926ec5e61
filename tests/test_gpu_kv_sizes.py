"""Norm, rotation, 4-bit cache and attention at sizes that take other splits of the work than small ones do
(several heads a look-up, wide row tiles, two waves to a row tile, keys in parts), against the 64-bit forms
of tests/kv_ref.py; long tails, shared pages, workspaces and a cache beyond 32-bit offsets."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import quantized_weight_prefill_amd as qg
from tests import kv_ref as R
from tests.test_gpu_kv import BF16, F16, Pool, assert_within, check_tokens, i32, randn, table
from tests.test_gpu_kv_attention import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 64, True), (64, 48, False), (64, 64, True)])
def test_norm_rope_of_many_heads(D, rot, interleaved):
    """An odd number of heads, many rows; a padded row; the keys' weight is none."""
    T, heads, kv = 820, 35, 5
    q, k = randn((T, heads, D), 1, BF16), randn((T, kv, D), 2, BF16)
    w = randn((D,), 3, torch.float32)
    rope = table(T, rot)
    pos = list(range(T))[::-1]
    pos[411] = T
    y = qg.qk_norm_rope(q, k, rope, i32(pos), q_weight=w, interleaved=interleaved)
    pick = list(range(0, T, 29)) + [411, T - 1]
    for x, got, weight in ((q, y[0], w), (k, y[1], None)):
        want, mag = R.turn64(x[pick], weight, rope, torch.tensor([pos[t] for t in pick]), 1e-6, interleaved)
        assert_within(got[pick], want, R.store_err(want, 24 * R.U32 * mag, BF16), "turned")
    assert (y[0][411] == 0).all() and (y[1][411] == 0).all()


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, F16)])
def test_append_and_read_of_many_heads(D, dtype):
    """Ragged sequences, some rows without a place, queries in the same launch, then everything read back."""
    kv, page = 5, 32
    new, lens = [3001, 0, 7, 2992], [3050, 5, 7, 2990]  # the last sequence's first two rows have no place
    T = sum(new)
    pool = Pool(4, lens, kv, D, page, 7)
    pool.tables[0, 60] = -1
    k, v, q = (randn((T + 3, kv, D), i, dtype) for i in (11, 12, 13))
    off = i32(np.cumsum([0] + new).tolist())
    rope = table(3050, D)
    y = qg.kv_append(pool.cache, k, v, pool.tables, i32(lens), offsets=off, rope=rope, eps=1e-6, q=q)
    row = 0
    for s, (n, length) in enumerate(zip(new, lens)):
        first = length - n
        places = [p for p in range(max(first, 0), length, 173) if not (s == 0 and p // page == 60)] + ([length - 1] if n else [])
        rows = [row + p - first for p in places]
        if rows:
            pos = torch.tensor(places)
            k64, _ = R.turn64(k[rows], None, rope, pos, 1e-6, False)
            check_tokens(pool, s, places, k64, v[rows].double().cpu())
            want, mag = R.turn64(q[rows], None, rope, pos, 1e-6, False)
            assert_within(y[rows], want, R.store_err(want, 24 * R.U32 * mag, dtype), f"queries of {s}")
        row += n
    for keep in (slice(0, T + 3), slice(0, 40)):  # many heads, and few
        n = len(range(T + 3)[keep])
        o, ln = (off, i32(lens)) if n > 40 else (i32([0, n]), i32([lens[0] - new[0] + n]))
        tb = pool.tables if n > 40 else pool.tables[:1].contiguous()
        rk, rv = qg.kv_read(pool.cache, tb, ln, n, kv, D, offsets=o)
        held = R.held64(v[:n])
        place = torch.full((n,), True)
        row = 0
        for s, m in enumerate(new):
            for t in range(m):
                p = lens[s] - m + t
                if row + t < n:
                    place[row + t] = p >= 0 and not (s == 0 and p // page == 60)
            row += m
        place[T:] = False
        held[~place] = 0
        assert_within(rv, held, R.store_err(held, 0.0 * held, torch.float32), "values read back")
        assert (rk[~place.cuda()] == 0).all() and rk[place.cuda()].abs().sum(-1).min() > 0


# rows of heads/kv query heads; which split each takes is beside it
SPLITS = [
    ([700], [800], 96, 12, 64, F16),         # tiles of 256 rows
    ([701], [701], 96, 12, 128, BF16),
    ([290], [900], 64, 8, 128, F16),         # four waves, two parts
    ([600], [2600], 64, 8, 64, BF16),        # four waves, parts of 2048
    ([600], [600], 64, 8, 128, BF16),        # two waves to 32 rows, one part
    ([70], [3000], 8, 2, 128, F16),          # two waves to 32 rows, parts of 512
    ([70], [3000], 8, 2, 64, BF16),
    ([2000], [2000], 2, 1, 64, F16),         # a prompt's triangle in two parts
    ([33], [700], 1, 1, 128, BF16),
]


@pytest.mark.parametrize("new,lens,heads,kv,D,dtype", SPLITS)
def test_prompt_splits(new, lens, heads, kv, D, dtype):
    b = Batch(new, lens, heads, kv, D, 64, dtype, seed=41)
    n = new[0]
    rows = {0, 1, 31, 32, n // 2, n - 2, n - 1}
    b.check(b.run(), rows=rows)
    b.check(b.run(window=90), window=90, rows=rows, what="window 90")
    b.check(b.run(window=650, max_len=300), window=650, rows=rows, what="window 650")
    assert torch.equal(b.run(), b.run())


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F16)])
def test_short_and_long_sequences_together(D, dtype):
    """Single tokens, a few rows, prompts and chunks, each with its own parts of the keys."""
    new, lens = [1, 3, 90, 1, 0, 40, 8, 9], [5000, 2500, 2100, 10, 0, 40, 600, 601]
    b = Batch(new, lens, 8, 2, D, 64, dtype, seed=43)
    b.check(b.run())
    b.check(b.run(window=300, max_len=5000), window=300)


@pytest.mark.parametrize("lens", [[384, 1, 300], [385, 383], [4096], [4160]])
def test_decode_parts(lens):
    """Lengths around those at which single tokens' keys are split in another way."""
    b = Batch([1] * len(lens), lens, 8, 2, 128, 32, F16, seed=45)
    b.check(b.run())


@pytest.mark.parametrize("n", [1, 40, 300])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
def test_long_tail(n, dtype):
    """One key of weight 1 and thousands of 2^-18, wherever the one is: they add up to 2 %."""
    D, L = 128, 6000
    for at in (0, 3001, L - n):
        pool = Pool(1, [L], 1, D, 64, 3)
        k = torch.zeros((L, 1, D), dtype=dtype)
        k[at, 0, 0] = 18 * math.log(2) / 8
        v = randn((L, 1, D), 47, dtype).abs()
        v[at] = 0
        k = k.cuda()
        qg.kv_append(pool.cache, k, v, pool.tables, i32([L]), offsets=i32([0, L]))
        q = torch.zeros((n, 2, D), dtype=dtype, device="cuda")
        q[:, :, 0] = 8
        y = qg.kv_attention(q, pool.cache, pool.tables, i32([L]), 1, offsets=None if n == 1 else i32([0, n]), scale=1.0)
        pick = [0, n // 2, n - 1]
        want, err = R.attention64(q[pick], R.held64(k), R.held64(v), [L - n + i for i in pick], 1.0, 0, dtype)
        assert float(want.abs().max()) > 0.01
        assert_within(y[pick], want, err, f"the one at {at}")


@pytest.mark.parametrize("new", [[1, 1], [60, 1]])
def test_negative_and_zero_scales(new):
    b = Batch(new, [200, 90], 4, 2, 128, 16, BF16, seed=49)
    for scale in (-0.2, 0.0):
        b.check(b.run(scale=scale), scale=scale, what=str(scale))


def test_a_page_named_twice_is_read_twice():
    b = Batch([1], [16], 4, 2, 64, 16, F16, seed=51)
    page = int(b.pool.tables[0, 0])
    y = qg.kv_attention(b.q, b.pool.cache, i32([page, page, page]).view(1, 3), i32([45]), 2)
    k, v = (torch.cat([x, x, x])[:45] for x in (b.k64, b.v64))
    want, err = R.attention64(b.q, k, v, [44], 64 ** -0.5, 0, F16)
    assert_within(y, want, err, "a page three times")


@pytest.mark.parametrize("new,lens", [([1, 1], [3000, 40]), ([70], [3000])])
def test_own_workspace(new, lens):
    """Of any contents, of the size that is asked for; a smaller one or one that shares memory is refused."""
    b = Batch(new, lens, 8, 2, 128, 64, F16, seed=53)
    want = b.run()
    S, width = b.pool.tables.shape
    need = qg.kv_attention_workspace_bytes(sum(new), S, 8, 2, 128, width * 64, b.offsets is not None)
    assert need > 0
    for fill in (0xFF, 0x00, 0x7E):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(b.run(workspace=ws), want)
    with pytest.raises((ValueError, qg.QGemmError)):
        b.run(workspace=ws[:need - 16])
    out = torch.empty_like(b.q)
    with pytest.raises(ValueError, match="shares memory"):
        b.run(workspace=b.pool.cache.view(-1), out=out)
    big = torch.zeros(need + out.nbytes, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="shares memory"):
        b.run(workspace=big, out=big[:out.nbytes].view(F16).view(out.shape))
    assert torch.equal(b.run(out=out), want) and torch.equal(b.run(out=out, workspace=big), want)


def test_rows_of_no_sequence_read_as_zeros():
    pool = Pool(1, [20], 2, 64, 16)
    none = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    for dtype in (F16, BF16, torch.float32):
        for r in qg.kv_read(pool.cache, none, none[:, 0], 3, 2, 64, offsets=i32([0]), dtype=dtype):
            assert r.dtype == dtype and r.shape == (3, 2, 64) and (r == 0).all()


def test_cache_beyond_32_bit_offsets():
    """Pages whose bytes lie past 2^32 give what pages of a small cache give."""
    kv, D, page, lens = 8, 128, 256, [1, 700]
    per = qg.kv_page_bytes(kv, D, page)
    pages = 2 ** 32 // per + 12
    cache = qg.kv_cache(pages, kv, D, page)
    small = qg.kv_cache(4, kv, D, page)
    tables = i32([3, -1, -1, 0, 2, 1]).view(2, 3)
    far = torch.where(tables < 0, tables, tables + (pages - 4))
    k, v = randn((sum(lens), kv, D), 55, F16), randn((sum(lens), kv, D), 56, F16)
    off, ln = i32([0, 1, 701]), i32(lens)
    new = i32([0, 1, 71])
    q = randn((71, 16, D), 57, F16)
    got = []
    for c, t in ((small, tables), (cache, far)):
        qg.kv_append(c, k, v, t, ln, offsets=off)
        got.append((*qg.kv_read(c, t, ln, 701, kv, D, offsets=off), qg.kv_attention(q, c, t, ln, kv, offsets=new),
                    qg.kv_attention(q[:2], c, t, ln, kv)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert_within(got[0][1], R.held64(v), R.store_err(R.held64(v), 0.0 * R.held64(v), torch.float32), "values")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 40])
def test_few_keys_keep_fp16_precision(D, new):
    """Large queries at right angles to the differences of the keys: all weights alike, while one fp16
    rounding of the keys would move the products by 12 times what the result's own rounding leaves.  What else is
    rounded, values and weights, is off by at most the relative half step that the result's rounding has
    at worst, twice the least that it has: the error is below sqrt(1 + 4 + 4) of the result's rounding."""
    L, heads = 48, 4
    b = Batch([new], [L], heads, 1, D, 32, F16, seed=61)
    basis = torch.linalg.svd(b.k64[1:, 0] - b.k64[:1, 0])[2][L - 1:]
    g = torch.Generator().manual_seed(62)
    b.q = (12 * torch.randn((new, heads, len(basis)), generator=g, dtype=torch.float64) @ basis).to(F16).cuda()
    y = b.run().double().cpu()
    want, _ = R.attention64(b.q, b.k64, b.v64, [L - new + i for i in range(new)], D ** -0.5, 0, F16)
    own = (want.to(F16).double() - want).norm()
    assert (y - want).norm() < 3 * own


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, F16), (128, BF16)])
@pytest.mark.parametrize("heads", [4, 16])
def test_decode_in_one_part(D, dtype, heads):
    """Enough sequences that lengths up to 1024 stay in one part, of eight waves; few that do up to 512."""
    lens = [1000, 1, 500, 777, 33, 257, 0, 999, 640, 255]
    b = Batch([1] * len(lens), lens, heads, 4, D, 16, dtype, seed=71)
    assert qg.kv_attention_workspace_bytes(10, 10, heads, 4, D, 1008, False) == 0
    b.check(b.run())
    b.check(b.run(window=300), window=300)
    few = Batch([1, 1], [511, 300], heads, 4, D, 256, dtype, seed=72)
    assert qg.kv_attention_workspace_bytes(2, 2, heads, 4, D, 512, False) == 0
    few.check(few.run())


@pytest.mark.parametrize("new", [[1, 1], [40, 3]])
@pytest.mark.parametrize("ks,vs", [(1e-5, 1e-6), (1.0, 3e-5), (200.0, 5000.0)])
def test_small_and_large_cache_values(new, ks, vs):
    """Scales and minima that are subnormal in fp16, and values near the largest that the cache holds."""
    b = Batch(new, [130, 60], 4, 2, 64, 16, BF16, seed=73)
    b.k, b.v = (b.k.float() * ks).to(BF16), (b.v.float() * vs).to(BF16)
    qg.kv_append(b.pool.cache, b.k, b.v, b.pool.tables, i32(b.lens), offsets=i32(b.start))
    b.k64, b.v64 = R.held64(b.k), R.held64(b.v)
    y = b.run()
    assert y.abs().max() > vs * 0.05
    b.check(y)


@pytest.mark.parametrize("new", [[5, 8, 6], [1, 8, 1, 1, 0, 5], [1] * 6, [8] * 4])
@pytest.mark.parametrize("D,dtype", [(128, F16), (64, BF16)])
def test_a_few_tokens_of_each_sequence(new, D, dtype):
    """Up to 32 rows of a key head in one block of rows or two."""
    lens = [2000, 8, 700, 90, 33, 1500][:len(new)]
    b = Batch(new, lens, 8, 2, D, 32, dtype, seed=75)
    b.offsets = i32(np.cumsum([0] + new).tolist())
    b.check(b.run())
    b.check(b.run(window=64, max_len=2000), window=64)


@pytest.mark.parametrize("heads", [4, 16])
def test_offsets_of_any_contents(heads):
    """Offsets that are none give rows inside the batch or none at all; rows of no sequence stay as they were."""
    b = Batch([20, 20], [600, 40], heads, 2, 128, 32, BF16, seed=77)
    args = (b.pool.cache, b.pool.tables, i32(b.lens), 2)
    for offsets, outside in (([5, 5, 5], range(40)), ([2 ** 31 - 1, 40, -7], range(40)), ([0, -2 ** 31, 3], range(3, 40)),
                             ([30, 3, 40], range(3)), ([-7, 2 ** 31 - 1, -2 ** 31], ())):
        out = torch.full_like(b.q, 9.0)
        qg.kv_attention(b.q, *args, offsets=i32(offsets), out=out)
        assert (out[list(outside)] == 9).all(), offsets
    b.check(b.run())
