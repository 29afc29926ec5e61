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


@pytest.mark.parametrize("beyond,status", [(15, -2), (1, -2), (16, -1)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads_that_one_launch_holds(D, beyond, status):
    """16 lanes to a head of 128, fewer than 2^32 lanes: up to 2^28 - 16 heads get as far as the missing pointer."""
    from tests.test_kv_host import P, attn_call, read_call, rope_call

    T = (1 << 28) - beyond
    missing = None if status == -1 else P  # sizes are refused first
    assert rope_call(Q=missing, qs=D, qos=D, K=None, Ko=None, T=T, heads=1, kv=0, D=D, rot=D) == status
    assert read_call(K=missing, T=T, kv=1, D=D) == status
    assert attn_call(Q=missing, qs=D, T=T, heads=1, kv=1, D=D) == status


def test_zero_rest_is_a_flag_of_two_calls():
    from tests.test_kv_host import append_call, attn_call, read_call, rope_call

    for dtype in (16, 17):  # QGEMM_ZERO_REST with float16 and bfloat16
        assert append_call(dtype=dtype, T=0, K=None) == 0 and attn_call(dtype=dtype, T=0, Q=None) == 0
        assert append_call(dtype=dtype, K=None) == -1 and attn_call(dtype=dtype, Q=None) == -1
        assert rope_call(dtype=dtype) == -3 and read_call(ot=dtype) == -3
    for dtype in (18, 32, -1):
        assert append_call(dtype=dtype) == -3 and attn_call(dtype=dtype) == -3
