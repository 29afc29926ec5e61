"""What the feed-forward operators' binding refuses before any launch, without a GPU."""
from __future__ import annotations

import pytest
import torch

import quantized_weight_prefill_amd as qg


def test_overlapping_buffers():
    """The ranges that meet, by name; the same tensor where it is allowed;
    neighbours in one allocation, absent and empty tensors are none."""
    flat = torch.zeros(96, dtype=torch.uint8)
    a, b = flat[:32], flat[32:64]
    qg._apart("out", a, 32, (("x", b, 32), ("bias", None, 32), ("rows", flat[16:16], 0)))
    qg._apart("out", b, 32, (("x", a, 32), ("residual", flat[64:], 32)))
    qg._apart("out", a, 32, (("residual", a, 32),), ("residual",))
    qg._apart(None, None, 32, (("x", a, 32),))
    qg._apart("workspace", flat[8:], 0, (("x", a, 32),))  # a call that needs none
    for t, o in ((a, a), (a, flat), (flat, b), (flat[31:], a), (a, flat[31:])):
        with pytest.raises(ValueError, match="out shares memory with x"):
            qg._apart("out", t, t.nbytes, (("x", o, o.nbytes),), ("residual",))
    with pytest.raises(ValueError, match="out shares memory with residual"):
        qg._apart("out", flat[1:33], 32, (("residual", a, 32),), ("residual",))
