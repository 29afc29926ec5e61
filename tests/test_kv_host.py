"""The attention layer's entry points without a GPU: every argument error comes
back before any launch, the rotation's table and the page size."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import quantized_weight_prefill_amd as qg

P = ctypes.c_void_p(1 << 20)  # never dereferenced: every call here fails before a launch
M8 = ctypes.c_void_p((1 << 20) + 8)
M2 = ctypes.c_void_p((1 << 20) + 2)


def test_rope_table():
    t = qg.rope_table(513, 64, base=1e6, scale=0.5)
    assert t.shape == (513, 64) and t.dtype == np.float32
    p, i = np.meshgrid(np.arange(513.0), np.arange(32.0), indexing="ij")
    a = p * (0.5 * 1e6 ** (-2.0 * i / 64))
    # the angle and its cosine are within a few 2^-53 of the definition's, the entry rounds by 2^-24
    assert np.abs(t[:, :32] - np.cos(a)).max() <= 2.0 ** -24 and np.abs(t[:, 32:] - np.sin(a)).max() <= 2.0 ** -24
    for kw in (dict(positions=0, rot=64), dict(positions=4, rot=0), dict(positions=4, rot=7),
               dict(positions=4, rot=64, base=0.0), dict(positions=4, rot=64, base=math.nan), dict(positions=4, rot=64, scale=math.inf)):
        with pytest.raises((qg.QGemmError, ValueError)):
            qg.rope_table(**kw)
    assert qg.lib().qgemm_rope_table(4, 64, 1e4, 1.0, None) == -1


def test_page_bytes():
    assert qg.kv_page_bytes(8, 128, 64) == 8 * 64 * 160
    assert qg.kv_page_bytes(1, 64, 16) == 16 * 80
    for a in ((8, 96, 64), (0, 128, 64), (8, 128, 48), (8, 128, 8), (8, 128, 512), (65537, 128, 64)):
        assert qg.kv_page_bytes(*a) == 0
    with pytest.raises(qg.QGemmError):
        qg.kv_cache(4, 8, 96, device="cpu")
    assert qg.kv_cache(3, 2, 64, 32, device="cpu").shape == (3, 2 * 32 * 80)


def rope_call(Q=P, qs=4096, K=P, ks=1024, wq=P, wk=P, rope=P, rl=100, rot=128, il=0, pos=P, eps=1e-6, Qo=P, qos=4096, Ko=P,
              kos=1024, T=4, heads=32, kv=8, D=128, dtype=0):
    return qg.lib().qgemm_qk_norm_rope(Q, qs, K, ks, wq, wk, rope, rl, rot, il, pos, eps, Qo, qos, Ko, kos, T, heads, kv, D,
                                       dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -3), (dict(D=96), -2), (dict(T=-1), -2), (dict(T=1 << 23), -2), (dict(heads=-1), -2),
    (dict(heads=0, kv=0), -2), (dict(heads=65537), -2), (dict(rot=120), -2), (dict(rot=144), -2), (dict(rot=0), -2),
    (dict(rl=0), -2), (dict(eps=math.nan), -2), (dict(rope=M8), -4), (dict(pos=M2), -4), (dict(pos=None), -1),
    (dict(Q=None), -1), (dict(Qo=None), -1), (dict(K=None), -1), (dict(Ko=None), -1), (dict(Q=M8), -4), (dict(Ko=M8), -4),
    (dict(qs=4100), -2), (dict(qos=4000), -2), (dict(kos=1016), -2), (dict(ks=-1024), -2), (dict(wq=M8), -4), (dict(wk=M8), -4),
    (dict(T=0, Q=None), 0),
])
def test_norm_rope_argument_errors(kw, status):
    assert rope_call(**kw) == status


def append_call(cache=P, pages=10, page=64, tables=P, width=4, lens=P, offs=P, S=2, K=P, ks=1024, V=P, vs=1024, wk=P, rope=P,
                rl=100, rot=128, il=0, pos=P, eps=1e-6, Q=P, qs=4096, wq=P, Qo=P, qos=4096, T=4, heads=32, kv=8, D=128, dtype=0):
    return qg.lib().qgemm_kv_append(cache, pages, page, tables, width, lens, offs, S, K, ks, V, vs, wk, rope, rl, rot, il, pos,
                                    eps, Q, qs, wq, Qo, qos, T, heads, kv, D, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -3), (dict(D=256), -2), (dict(kv=0), -2), (dict(page=48), -5), (dict(page=8), -5), (dict(page=512), -5),
    (dict(S=-1), -2), (dict(T=-1), -2), (dict(offs=None), -2), (dict(pages=0), -2), (dict(width=0), -2), (dict(width=1 << 26), -2),
    (dict(pages=1 << 31), -2), (dict(T=1 << 23), -2), (dict(S=1 << 22, T=1), -2),
    (dict(cache=None), -1), (dict(tables=None), -1), (dict(lens=None), -1), (dict(cache=M8), -4), (dict(tables=M2), -4),
    (dict(lens=M2), -4), (dict(offs=M2), -4), (dict(K=None), -1), (dict(V=None), -1), (dict(K=M8), -4), (dict(V=M8), -4),
    (dict(ks=1020), -2), (dict(vs=-8), -2), (dict(Qo=None), -1), (dict(heads=0), -2), (dict(qos=4088), -2), (dict(wk=M8), -4),
    (dict(wq=M8), -4), (dict(rot=8), -2), (dict(eps=math.nan), -2), (dict(T=0, K=None), 0), (dict(S=0, K=None), 0),
])
def test_append_argument_errors(kw, status):
    assert append_call(**kw) == status


def read_call(cache=P, pages=10, page=64, tables=P, width=4, lens=P, offs=P, S=2, K=P, V=P, T=4, kv=8, D=128, ot=2):
    return qg.lib().qgemm_kv_read(cache, pages, page, tables, width, lens, offs, S, K, V, T, kv, D, ot, None)


@pytest.mark.parametrize("kw,status", [
    (dict(ot=3), -3), (dict(D=32), -2), (dict(kv=0), -2), (dict(page=1), -5), (dict(offs=None), -2), (dict(T=1 << 26), -2),
    (dict(cache=None), -1), (dict(K=None), -1), (dict(V=None), -1), (dict(K=M8), -4), (dict(V=M8), -4), (dict(T=0, K=None), 0),
])
def test_read_argument_errors(kw, status):
    assert read_call(**kw) == status


def attn_call(Q=P, qs=4096, cache=P, pages=10, page=64, tables=P, width=4, lens=P, offs=P, S=2, Y=P, T=4, heads=32, kv=8, D=128,
              window=0, scale=0.1, max_len=0, dtype=0, ws=P, wsb=1 << 40):
    return qg.lib().qgemm_kv_attention(Q, qs, cache, pages, page, tables, width, lens, offs, S, Y, T, heads, kv, D, window, scale,
                                       max_len, dtype, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -3), (dict(D=80), -2), (dict(kv=0), -2), (dict(heads=0), -2), (dict(heads=12), -2),
    (dict(heads=129, kv=1), -2), (dict(window=-1), -2), (dict(max_len=-1), -2), (dict(scale=math.nan), -2), (dict(page=20), -5),
    (dict(offs=None), -2), (dict(T=1 << 24), -2), (dict(Q=None), -1), (dict(Y=None), -1), (dict(cache=None), -1), (dict(Q=M8), -4),
    (dict(Y=M8), -4), (dict(ws=M8), -4), (dict(qs=4), -2), (dict(T=0, Q=None), 0), (dict(S=0, Q=None), 0),
])
def test_attention_argument_errors(kw, status):
    assert attn_call(**kw) == status


def test_binding_refuses():
    """The binding names what is wrong before any call reaches a device."""
    x = torch.zeros((4, 8, 128), dtype=torch.float16)
    cache = qg.kv_cache(3, 8, 128, 64, device="cpu")
    tables, lens = torch.zeros((4, 2), dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        qg.qk_norm_rope(x, x)
    with pytest.raises(ValueError, match="device"):
        qg.kv_append(cache, x, x, tables, lens)
    with pytest.raises(ValueError, match="device"):
        qg.kv_read(cache, tables, lens, 4, 8, 128)
    with pytest.raises(ValueError, match="device"):
        qg.kv_attention(x, cache, tables, lens, 8)
    with pytest.raises(TypeError):
        qg.kv_read(cache, tables, lens, 4, 8, 128, dtype=torch.int8)
    with pytest.raises(TypeError):
        qg.qk_norm_rope(x.float(), None)
    assert qg._kv_page(cache, 8, 128) == 64
    for bad in (cache[:, :-16].contiguous(), cache[0], cache.to(torch.int8), cache[:, ::2]):
        with pytest.raises(ValueError):
            qg._kv_page(bad, 8, 128)


def test_rows_apart():
    """Rows of a merged product's parts may interleave, and nothing else may overlap."""
    buf = torch.zeros((6, 48 * 128), dtype=torch.float16)
    part = lambda a, b: buf[:, a * 128:b * 128].view(6, b - a, 128)
    q, k = part(0, 32), part(32, 40)
    qg._rows_apart("out", q, [("k", k), ("none", None)])
    for other in (q, part(31, 40), part(0, 1), buf.view(-1)[128:128 + 5 * 1024].view(5, 8, 128)):
        with pytest.raises(ValueError, match="shares memory"):
            qg._rows_apart("out", q, [("other", other)])
        with pytest.raises(ValueError, match="shares memory"):
            qg._rows_apart("out", other, [("q", q)])
    qg._rows_apart("out", q, [("later", torch.zeros((6, 8, 128), dtype=torch.float16))])


def test_workspace_bytes():
    """None for one part or sizes that no call takes; a multiple of 16; the bound on the lengths only splits."""
    f = qg.kv_attention_workspace_bytes
    assert f(1, 1, 32, 8, 128, 384, False) == 0 and f(1, 1, 32, 8, 128, 4096, False) > 0
    assert f(658, 1, 32, 8, 128, 658, True) == 0 and f(64, 1, 32, 8, 128, 8000, True) > 0
    assert f(4096, 1, 32, 8, 128, 4096, True) == 0
    for bad in ((0, 1, 32, 8, 128, 99), (1, 0, 32, 8, 128, 99), (1, 1, 32, 7, 128, 99), (1, 1, 32, 8, 96, 99), (1, 1, 32, 8, 128, -1),
                (1 << 31, 1, 32, 8, 128, 99), (1, 1 << 30, 32, 8, 128, 99), (1 << 22, 1 << 22, 1, 1, 64, 99)):
        assert f(*bad, True) == 0
    for T, S, heads, kv in ((1, 1, 1, 1), (3, 3, 5, 1), (700, 2, 16, 2), (9, 4, 40, 1), (2000, 7, 7, 7)):
        for n in (0, 1, 385, 5000, 1 << 30):
            for D in (64, 128):
                b = f(T, S, heads, kv, D, n, True)
                assert b % 16 == 0 and b <= (T * heads + S * kv * 32) * 128 * (D + 2) * 4 + 4096, (T, S, heads, kv, n, D)


@pytest.mark.parametrize("kw", [dict(page=256, width=(1 << 22) + 1), dict(page=16, width=(1 << 26) + 1), dict(S=1 << 23, T=1 << 23),
                                dict(S=1 << 22, T=4, heads=1, kv=1)])
def test_sizes_beyond_the_kernels(kw):
    """Places from 2^30 on, and more sequences and heads than a launch holds."""
    assert attn_call(**kw) == -2
    if "width" in kw:
        assert append_call(**kw) == -2 and read_call(**kw) == -2
