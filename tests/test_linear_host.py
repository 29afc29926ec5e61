"""The linear layer's refusals and plans, without a GPU: every argument error
comes back before any launch, the binding names the argument it refuses, and
the gated form never asks for a rung that splits K across workgroups."""
from __future__ import annotations

import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import quantized_weight_prefill_amd as qg

P = ctypes.c_void_p(1 << 20)  # never dereferenced: every call here fails before a launch
MIS = ctypes.c_void_p((1 << 20) + 8)
NAMES = [qg.rung_name(r) for r in range(qg.num_rungs())]
SPLIT = [r for r, n in enumerate(NAMES) if n.endswith("-sk")]


def call(fmt=0, rung=-1, xl=0, X=P, W=P, bias=None, res=None, Y=P, yl=0, M=8, N=64, K=512, group=0, zp=0, act=0, gated=0,
         dtype=0, ws=None, wsb=0):
    return qg.lib().qgemm_linear(fmt, rung, xl, X, W, bias, res, Y, yl, M, N, K, group, zp, act, gated, dtype, ws, wsb,
                                 None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=7), -5), (dict(fmt=2, group=0), -5), (dict(fmt=2, group=48), -5), (dict(rung=99), -5), (dict(rung=-2), -5),
    (dict(xl=2), -5), (dict(xl=-1), -5), (dict(yl=2), -5), (dict(act=5), -5), (dict(act=-1), -5),
    (dict(M=-1), -2), (dict(N=0), -2), (dict(K=500), -2), (dict(K=0), -2), (dict(fmt=2, group=128, K=64), -2),
    (dict(gated=1, N=40), -2), (dict(gated=1, N=1 << 31), -2), (dict(gated=1, N=(1 << 30) + 16), -2),
    (dict(yl=1, N=64), -2), (dict(yl=1, N=200), -2), (dict(N=1 << 32), -2),
    (dict(dtype=2), -3), (dict(dtype=-1), -3),
    (dict(X=None), -1), (dict(W=None), -1), (dict(Y=None), -1),
    (dict(X=MIS), -4), (dict(W=MIS), -4), (dict(Y=MIS), -4), (dict(bias=MIS), -4), (dict(res=MIS), -4),
])
def test_argument_errors(kw, status):
    assert call(**kw) == status


def test_no_rows_is_no_launch():
    assert call(M=0, X=None, W=None, Y=None) == 0
    assert call(M=0, X=None, W=None, Y=None, gated=1, yl=1, N=128) == 0
    assert call(M=0, N=40, gated=1) == -2  # the shape is still checked


def test_split_rungs():
    """A rung that splits K needs its workspace; the gated form has none."""
    for sk in SPLIT:
        assert call(rung=sk, gated=1) == -5
        need = qg.lib().qgemm_linear_workspace_bytes(1, sk, 1, 64, 4096, 12288, 0, 0)
        assert need > 0 and need == qg.workspace_bytes("q6k", sk, 64, 4096, 12288, layout=qg.X_FRAG)
        big = dict(fmt=1, rung=sk, xl=1, M=64, N=4096, K=12288)
        assert call(**big) == -6
        assert call(**big, ws=P, wsb=need - 1) == -6
        assert call(**big, ws=MIS, wsb=need) == -4
        assert qg.lib().qgemm_linear_workspace_bytes(1, sk, 1, 64, 4096, 12288, 1, 0) == 0
    # the fragment-major ladder picks a split rung here, the gated one its next best
    for M, N, K in ((64, 4096, 12288), (658, 4096, 12288)):
        assert qg.linear_select_rung("q6k", M, N, K, layout=qg.X_FRAG)["rung"] in SPLIT
        info = qg.linear_select_rung("q6k", M, N // 2, K, gated=True, layout=qg.X_FRAG)
        assert info["rung"] not in SPLIT and info["tiles_m"] * info["rows"] >= M
        assert qg.lib().qgemm_linear_workspace_bytes(1, -1, 1, M, N // 2, K, 1, 0) == 0


@pytest.mark.parametrize("fmt", ["q4k", "q6k", "w4a16"])
@pytest.mark.parametrize("layout", [qg.X_ROW, qg.X_FRAG])
def test_plain_ladder_is_the_products(fmt, layout):
    sel = qg.select_rung if layout == qg.X_ROW else qg.select_rung_xf
    for M in (1, 7, 16, 17, 33, 48, 64, 65, 130, 400, 658, 2048):
        for N, K in ((16, 256), (33, 512), (640, 9216), (1024, 4096), (4096, 12288), (4128, 4096), (8192, 4096), (12288, 4096)):
            for dt in (qg.F16, qg.BF16):
                got, want = qg.linear_select_rung(fmt, M, N, K, False, dt, layout), sel(fmt, M, N, K, dt)
                if got["name"] != want["name"]:  # a panel and all rows per wave, where the products share four panels
                    assert got["name"] == "direct-small-m" and got["cols"] == 16 and got["rows"] >= min(M, 64)
                    assert M <= 64 or got["tiles_n"] * got["tiles_m"] <= 256
                    assert want["name"] == "direct-skinny-n" or (want["name"] == "mfma32-64x32-k4" and 32 < M <= 48)
                    assert N <= 64 or (layout == qg.X_ROW and M > 16)
                elif N <= 64 and (M <= 16 or (M <= 64 and N > 32)):
                    assert got["name"] == "direct-small-m" and got["cols"] == 16
                else:
                    assert got == want
                g = qg.linear_select_rung(fmt, M, 16 * -(-N // 16), K, True, dt, layout)
                assert g["rung"] not in SPLIT
                assert g["cols"] % 32 == 0 and g["cols"] * g["tiles_n"] >= 2 * N and g["rows"] * g["tiles_m"] >= M
    with pytest.raises(qg.QGemmError):
        qg.linear_select_rung(fmt, 4, 40, 512, True)
    with pytest.raises(qg.QGemmError):
        qg.linear_select_rung(fmt, 4, 64, 512, False, layout=3)


def test_binding_refusals():
    M, N, K = 8, 64, 512
    x = torch.zeros((M, K), dtype=torch.float16)
    xf = torch.zeros(qg.xf_bytes(M, K) // 2, dtype=torch.float16)
    wp = torch.zeros(qg.packed_bytes("q4k", N, K), dtype=torch.uint8)
    wp2 = torch.zeros(qg.packed_bytes("q4k", 2 * N, K), dtype=torch.uint8)
    h = lambda *s: torch.zeros(s, dtype=torch.float16)
    for kw, match in ((dict(act="swish"), "act"), (dict(bias=h(N + 1)), "bias"), (dict(bias=h(N).bfloat16()), "bias"),
                      (dict(residual=h(M, N + 1)), "residual"), (dict(residual=h(M, N).float()), "residual"),
                      (dict(out=h(M, N + 1)), "out"), (dict(out=h(M, N).float()), "out"), (dict(out_layout=3), "out_layout"),
                      (dict(gated=True), "packed weight")):
        with pytest.raises(ValueError, match=match):
            qg.linear("q4k", x, wp, N, **kw)
        with pytest.raises(ValueError, match=match):
            qg.linear_xf("q4k", xf, wp, M, N, K, **kw)
    with pytest.raises(ValueError, match="bias"):       # gated: both halves' biases
        qg.linear("q4k", x, wp2, N, gated=True, bias=h(N))
    with pytest.raises(ValueError, match="device"):     # host tensors
        qg.linear("q4k", x, wp, N)
    with pytest.raises(ValueError, match="fragment-major"):
        qg.linear_xf("q4k", xf[:-8], wp, M, N, K)
    with pytest.raises(TypeError):
        qg.linear("q4k", x.float(), wp, N)
    with pytest.raises(ValueError):
        qg.linear("q4k", x[0], wp, N)
    with pytest.raises(qg.QGemmError):                  # N is no multiple of 128
        qg.linear("q4k", x, wp, N, out_layout=qg.X_FRAG)


def test_missing_calls_module_fails_every_time():
    """Without the C++ calls the library does not load, at the first use or a
    later one (in a process of its own: here it is loaded)."""
    code = ("import sys, quantized_weight_prefill_amd as qg\n"
            "sys.modules['quantized_weight_prefill_amd._calls'] = None\n"
            "n = 0\n"
            "for _ in range(2):\n"
            "    try: qg.lib()\n"
            "    except ImportError: n += 1\n"
            "assert n == 2, n\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(qg.__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=300)
