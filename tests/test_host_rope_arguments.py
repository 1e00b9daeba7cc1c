"""What kv_append's rotary arguments may be (no GPU: refused before any tensor is asked for its
device): one table without the other used to be taken as no rotation where cos was the missing one."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

import fp8_weight_only_gemm_gb300 as w8
from fp8_weight_only_gemm_gb300.build import build_library

CACHE = SimpleNamespace(_address=0, _index=0, head_dim=64)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_library()
    w8.load()


def append(**kw):
    k = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    return w8.kv_append(CACHE, k, k, torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32), **kw)


@pytest.mark.parametrize("name", ["cos", "sin"])
def test_one_table_without_the_other(name):
    with pytest.raises(ValueError, match="cos and sin"):
        append(**{name: torch.zeros(8, 32)})


def test_interleaved_without_a_truth_value():
    table = torch.zeros(8, 32)
    with pytest.raises(RuntimeError, match="ambiguous"):
        append(cos=table, sin=table, interleaved=torch.zeros(2))
