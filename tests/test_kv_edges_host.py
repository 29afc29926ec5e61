"""The attention layer's binding and entry points at the ends of strides and sizes, without a GPU."""
from __future__ import annotations

import pytest
import torch

import quantized_weight_prefill_amd as qg


def test_rows_that_lie_on_one_another():
    """Rows of stride 0 share memory with what lies there, and with nothing beside it."""
    buf = torch.zeros((6, 48 * 128), dtype=torch.float16)
    one = lambda at, heads: buf.view(-1)[at * 128:(at + heads) * 128].view(1, heads, 128).expand(3, heads, 128)
    for other in (one(0, 4), one(3, 2), one(2, 1)):
        with pytest.raises(ValueError, match="shares memory"):
            qg._rows_apart("out", one(0, 4), [("other", other)])
    for other in (one(4, 4), one(48, 2)):
        qg._rows_apart("out", one(0, 4), [("other", other)])
