"""Attention where the softmax scale and the key scales lie far apart: only their product
with the query reaches the logits. The tolerance is the one of the attention tests (their
reference and bound take any scales)."""
from __future__ import annotations

import pytest
import torch

from test_gpu_kv_append import Case
from test_gpu_kv_attention import check, finite_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def w8():
    import fp8_weight_only_gemm_gb300 as w8
    from fp8_weight_only_gemm_gb300.build import build_library
    build_library()
    w8.load()
    w8.device_status(clear=True)
    yield w8
    assert w8.device_status(clear=True)[0] == 0


# exponents: of the softmax scale, of the key scales, of the queries
@pytest.mark.parametrize("scale,keys,queries", [
    (-100, 100, 0),      # a scale that brings huge keys back
    (-66, 62, 0),
    (0, 100, -100),      # tiny queries against huge keys
    (-60, 119, -63),
    (-3, 120, -120),
    (80, -50, -33),      # the other way round
    (60, 0, -64),
    (-140, 0, 0),        # logits that are all 0: averages over the visible keys
    (-126, -40, -100),
])
@pytest.mark.parametrize("form", ["few", "many", "wide"])
def test_scales_far_apart(w8, form, scale, keys, queries):
    counts, D = {"few": ([3, 9], 64), "many": ([70, 140], 128), "wide": ([5, 40], 256)}[form]
    case = Case([500, 130], counts, 4, 2, D, 16, "bf16", seed=61 + D)
    finite_cache(case, 62)
    case.ks = case.ks * 2.0 ** keys
    check(case, w8, scale=2.0 ** scale, q_scale=2.0 ** queries)
