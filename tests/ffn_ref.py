"""Plain 64-bit forms of the feed-forward operators and the error a right
kernel may make on them, for the GPU tests of the linear and the
mixture-of-experts layers.

Error model.  With W rounded once into the operand type, every operand is
exact and the products are exact in binary32.  A binary32 sum of K terms in any
order, each addition within one step of 2^-23 relative (the MFMA pipe may
truncate where it aligns), is within K * 2^-23 * B of the exact sum, B =
sum |x||w|.  An activation has a slope of at most 1.13 (SiLU 1.10, GELU 1.13)
and a kernel evaluates it within 2^-19 of its value (the exponent's rounding
for |v| < 16: |v| * 2^-24 * 1.5, exp2 and rcp 2^-23 each, erfc's fit 2^-21).
Bias, product and residual each round by 2^-24 of their result.  The store
rounds by at most eps/2 of the value, or half a subnormal step.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle
import quantized_weight_prefill_amd as qg

EPS32 = 2.0 ** -24
SUB = {qg.F16: 2.0 ** -25, qg.BF16: 2.0 ** -134}       # half a subnormal step
HALF = {qg.F16: 2.0 ** -11, qg.BF16: 2.0 ** -8}         # eps / 2, relative
MAXF = {qg.F16: 65504.0, qg.BF16: 3.38e38}


def act64(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2.0))
    if act == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def act_err(a, d, act):
    """Error of act(v) = a when v is off by d."""
    if act == "none":
        return d
    if act == "relu":
        return d
    return 1.13 * d + 2.0 ** -19 * a.abs()


def store_err(y, d, dtype):
    """Error of the stored value when the binary32 one is off by d."""
    return d + HALF[dtype] * (y.abs() + d) + SUB[dtype]


def bits64(bits, dtype):
    return torch.from_numpy(np.ascontiguousarray(oracle.bits_to_double_fast(np.ascontiguousarray(bits), dtype)))


def product(x, w):
    """(x . w, its error in binary32): x [M][K], w [K][N] float64."""
    K = x.shape[1]
    return x @ w, K * 2.0 ** -23 * (x.abs() @ w.abs())


def linear64(x, w, N, bias=None, res=None, act="none", gated=False):
    """(Y before the store's rounding, its error)."""
    v, d = product(x, w)
    if bias is not None:
        v = v + bias
        d = d + EPS32 * (v.abs() + d)
    if gated:
        g, u, dg, du = v[:, :N], v[:, N:], d[:, :N], d[:, N:]
        a = act64(g, act)
        da = act_err(a, dg, act)
        y = a * u
        d = da * u.abs() + a.abs() * du + da * du
        d = d + EPS32 * (y.abs() + d)
    else:
        y = act64(v, act)
        d = act_err(y, d, act)
    if res is not None:
        y = y + res
        d = d + EPS32 * (y.abs() + d)
    return y, d


def assert_within(got, y, d, dtype, what):
    """got: device tensor of the operator's type; y, d: its exact value and error."""
    g = got.detach().cpu().double()
    allow = store_err(y, d, dtype)
    # a value whose error reaches past the largest finite one may be infinite
    over = y.abs() + allow >= MAXF[dtype]
    bad = ~(((g - y).abs() <= allow) | over | (torch.isnan(g) & torch.isnan(y)))
    if bad.any():
        i = tuple(int(t) for t in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first {i}: got {g[i]}, want {y[i]}, "
                             f"allowed {allow[i]}")


def bits(t):
    return t.detach().contiguous().cpu().view(torch.int16)
