"""Sizes that the attention kernels do not count (no GPU, no launch): more than 2^31 - 1 query rows
that share a key/value head wrapped in 32 bits and left rows unwritten; they are refused."""
from __future__ import annotations

import ctypes

import pytest

from fp8_weight_only_gemm_gb300 import binding
from fp8_weight_only_gemm_gb300.build import build_library
from test_host_decode_ops import attention, batch, cache, heads

RANGE = -8


@pytest.fixture(scope="module")
def lib():
    build_library()
    return binding.load()


@pytest.mark.parametrize("max_q,group", [(1 << 17, 1 << 14), (1 << 12, 1 << 20), ((1 << 31) - 1, 2)])
def test_more_rows_a_head_than_are_counted(lib, max_q, group):
    c, q = cache(kv_heads=1), heads(group, token=128 * group)
    b = batch(batch=1, tokens=max_q, max_q=max_q)
    assert attention(lib, c=c, b=b, q=q, out=q) == RANGE
    assert f"max_q={max_q}" in binding.last_error()
    assert lib.w8a16_kv_attention_workspace_bytes(ctypes.byref(c), 1, max_q, group) == 0
    assert f"max_q={max_q}" in binding.last_error()
