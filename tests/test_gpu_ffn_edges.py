"""The feed-forward operators where one expert is popular, where a weight
overflows the operand type, and where buffers, streams and sizes are at the
edge of what a call takes."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import quantized_weight_prefill_amd as qg
from quantized_weight_prefill_amd import synth
from tests.helpers import bytes_to_device
from tests.test_gpu_exact import DTYPES

pytestmark = pytest.mark.gpu

TORCH = {qg.F16: torch.float16, qg.BF16: torch.bfloat16}


def eye_fields(n):
    """Q4_K fields of the n x n unit matrix (d = 1, one scale for all)."""
    f = {k: np.zeros_like(v) for k, v in synth.q4k_fields(np.random.default_rng(0), n, n).items()}
    f["d"][:], f["sc"][:], f["q"][:] = 0x3C00, 1, np.eye(n, dtype=np.uint8)
    return f


def pack(f, N, K):
    return qg.pack("q4k", synth.encode("q4k", f), N, K)


def square_layer(x64, ids, E, dtype, down, **kw):
    """The layer of E equal experts with gate = up = I and no activation: h = x * x."""
    T, n = x64.shape
    eye = eye_fields(n)
    up = pack({k: np.concatenate([v, v]) for k, v in eye.items()}, 2 * n, n)
    ids = torch.as_tensor(ids, dtype=torch.int32).reshape(T, -1).cuda()
    offs, rows = qg.moe_group(ids, E)
    return qg.moe("q4k", "q4k", x64.to(TORCH[dtype]).cuda(), bytes_to_device(np.tile(up, E)),
                  bytes_to_device(np.tile(pack(down, n, n), E)), torch.ones(ids.shape, device="cuda"), offs, rows, n,
                  act="none", **kw).cpu().double()


def popular(T, E, share, rng):
    """One expert per token, `share` of them on expert E // 2."""
    ids = rng.integers(0, E, T)
    ids[rng.random(T) < share] = E // 2
    return ids


@pytest.mark.parametrize("dtype", DTYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("T,E,share", [(9, 8, 1.0), (16, 8, 1.0), (17, 8, 1.0), (20, 8, 1.0), (24, 8, 1.0), (25, 8, 0.7),
                                       (64, 16, 0.5), (120, 40, 0.4), (1024, 300, 0.3), (1024, 256, 1.0)])
def test_moe_keeps_both_parts_of_h_whatever_an_experts_share(T, E, share, dtype):
    """What is left of h = x * x after its rounding, exactly, when an expert
    has more rows than others (at most four per expert on average): x are
    whole numbers up to 255, so x * x has 16 bits, its rounding 11 or 8 and
    the rest at most 8, and Y = h - RN(h) has them all."""
    n = 256
    rng = np.random.default_rng(1200 + T)
    x64 = torch.from_numpy(rng.integers(-255, 256, (T, n)).astype(np.float64))
    res = -(x64 * x64).to(TORCH[dtype])
    left = x64 * x64 + res.double()
    assert bool((left != 0).any()) and torch.equal(left.to(TORCH[dtype]).double(), left)
    y = square_layer(x64, popular(T, E, share, rng), E, dtype, eye_fields(n), residual=res.cuda())
    bad = (y != left).any(1).nonzero().flatten().tolist()
    assert not bad, f"{len(bad)} rows differ, first {bad[:8]}"
