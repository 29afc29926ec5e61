"""The mixture-of-experts entry points' refusals, without a GPU: every
argument error comes back before any launch."""
from __future__ import annotations

import ctypes

import pytest
import torch

import quantized_weight_prefill_amd as qg

P = ctypes.c_void_p(1 << 20)  # never dereferenced: every call here fails before a launch
M4 = ctypes.c_void_p((1 << 20) + 4)
M2 = ctypes.c_void_p((1 << 20) + 2)


def route(logits=P, lt=0, T=4, E=8, k=2, score=0, renorm=1, scale=1.0, ids=P, w=P, offs=P, rows=P):
    return qg.lib().qgemm_moe_route(logits, lt, T, E, k, score, renorm, scale, ids, w, offs, rows, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -2), (dict(E=0), -2), (dict(E=1025), -2), (dict(k=0), -2), (dict(k=9), -2), (dict(k=65, E=100), -2),
    (dict(T=1 << 31), -2), (dict(T=1 << 30, k=2), -2), (dict(T=(1 << 26) - 3, k=1), -2), (dict(lt=3), -3), (dict(lt=-1), -3), (dict(score=2), -5),
    (dict(logits=None), -1), (dict(ids=None), -1), (dict(w=None), -1), (dict(offs=None), -1), (dict(rows=None), -1),
    (dict(logits=M4), -4), (dict(ids=M4), -4), (dict(w=M2), -4), (dict(offs=M2), -4), (dict(rows=M2), -4),
])
def test_route_argument_errors(kw, status):
    assert route(**kw) == status


def group(ids=P, T=4, E=8, k=2, offs=P, rows=P):
    return qg.lib().qgemm_moe_group(ids, T, E, k, offs, rows, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -2), (dict(E=0), -2), (dict(E=1025), -2), (dict(k=0), -2), (dict(k=65), -2), (dict(T=1 << 30), -2),
    (dict(ids=None), -1), (dict(offs=None), -1), (dict(rows=None), -1), (dict(T=0, offs=None), -1),
    (dict(ids=M4), -4), (dict(offs=M2), -4), (dict(rows=M2), -4),
])
def test_group_argument_errors(kw, status):
    assert group(**kw) == status


def moe(fu=0, fd=1, X=P, Wu=P, Wd=P, w=P, offs=P, rows=P, res=None, Y=P, T=4, k=2, E=8, H=512, I=256, grp=0, zp=0, act=2,
        dtype=0, ws=P, wsb=1 << 20):
    return qg.lib().qgemm_moe(fu, fd, X, Wu, Wd, w, offs, rows, res, Y, T, k, E, H, I, grp, zp, act, dtype, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(fu=5), -5), (dict(fd=-1), -5), (dict(fu=2), -5), (dict(fd=2, grp=100), -5), (dict(act=9), -5),
    (dict(T=-1), -2), (dict(k=0), -2), (dict(E=0), -2), (dict(H=500), -2), (dict(I=128), -2), (dict(I=0), -2),
    (dict(fu=2, fd=2, grp=128, H=192, I=128), -2), (dict(fu=2, fd=2, grp=256, H=256, I=128), -2),
    (dict(T=513), -2), (dict(T=1025, k=1), -2), (dict(T=1 << 40, k=1 << 30), -2), (dict(k=1025, T=1), -2),
    (dict(I=(1 << 30) + 256), -2), (dict(dtype=2), -3),
    (dict(X=None), -1), (dict(Wu=None), -1), (dict(Wd=None), -1), (dict(w=None), -1), (dict(offs=None), -1),
    (dict(rows=None), -1), (dict(Y=None), -1),
    (dict(X=M4), -4), (dict(Wu=M4), -4), (dict(Wd=M4), -4), (dict(res=M4), -4), (dict(Y=M4), -4), (dict(w=M2), -4),
    (dict(offs=M2), -4), (dict(rows=M2), -4), (dict(ws=M4), -4),
    (dict(ws=None), -6), (dict(wsb=qg.moe_workspace_bytes(4, 2, 512, 256) - 1), -6),
])
def test_moe_argument_errors(kw, status):
    assert moe(**kw) == status


def test_empty_batches_launch_nothing():
    assert route(T=0, logits=None, ids=None, w=None, offs=None, rows=None) == 0
    assert moe(T=0, X=None, Wu=None, Wd=None, w=None, offs=None, rows=None, Y=None, ws=None, wsb=0) == 0


def test_workspace_bytes():
    """h, and the partial sums and counters of the panels that several
    workgroups share."""
    assert qg.moe_workspace_bytes(64, 8, 2048, 768) >= 64 * 8 * 768 * 2
    assert qg.moe_workspace_bytes(128, 8, 2048, 768) > qg.moe_workspace_bytes(64, 8, 2048, 768)
    for bad in ((129, 8, 256, 768), (-1, 8, 256, 768), (0, 8, 256, 768), (4, 0, 256, 768), (4, 8, 256, 0),
                (1 << 40, 1 << 40, 256, 768), (4, 8, 100, 768), (4, 8, 256, 100), (4, 8, 0, 768), (4, 8, 1 << 32, 768)):
        assert qg.moe_workspace_bytes(*bad) == 0


def test_binding_refusals():
    T, k, E, H, I = 3, 2, 4, 512, 256
    x = torch.zeros((T, H), dtype=torch.float16)
    up = torch.zeros(E * qg.packed_bytes("q4k", 2 * I, H), dtype=torch.uint8)
    dn = torch.zeros(E * qg.packed_bytes("q6k", H, I), dtype=torch.uint8)
    w, offs, rows = torch.zeros((T, k)), torch.zeros(E + 1, dtype=torch.int32), torch.zeros(T * k, dtype=torch.int32)
    ok = dict(x=x, w_up=up, w_down=dn, weights=w, offsets=offs, rows=rows, inter=I)

    def call(**kw):
        a = {**ok, **kw}
        return qg.moe("q4k", "q6k", a.pop("x"), a.pop("w_up"), a.pop("w_down"), a.pop("weights"), a.pop("offsets"),
                      a.pop("rows"), a.pop("inter"), **a)

    for kw, match in ((dict(act="swish"), "act"), (dict(weights=w.half()), "weights"), (dict(weights=w[:2]), "weights"),
                      (dict(offsets=offs.long()), "offsets"), (dict(rows=rows[:-1]), "rows"), (dict(offsets=offs[:1]), "offsets"),
                      (dict(residual=x[:, :-1]), "residual"), (dict(x=x[0]), "x must be"), ({}, "device")):
        with pytest.raises(ValueError, match=match):
            call(**kw)
    with pytest.raises(ValueError):
        qg.moe_group(torch.zeros((2, 2), dtype=torch.int64), 4)
    with pytest.raises(ValueError):
        qg.moe_group(torch.zeros(4, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="device"):
        qg.moe_group(torch.zeros((2, 2), dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="score"):
        qg.moe_route(x, 2, score="linear")
    with pytest.raises(ValueError):
        qg.moe_route(x[0], 2)
    with pytest.raises(ValueError, match="device"):
        qg.moe_route(x, 2)
    with pytest.raises(TypeError):
        qg.moe_route(x.long(), 2)
