"""Sequences that all end inside the shared prefix: what lies behind them on its pages, codes and scales, has no effect, as past any
sequence's end. (fill leaves NaN codes and NaN scales there.)"""
from __future__ import annotations

import pytest
import torch

from test_gpu_kv_append import Case
from test_gpu_kv_span import Span, check

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


# sequence 0 has no rows: its table names the prefix's pages
@pytest.mark.parametrize("counts,Hq,Hkv,D,P", [([0, 1, 1], 4, 2, 128, 32), ([0, 2, 3], 6, 1, 64, 16), ([0, 3, 2], 3, 3, 256, 64), ([0, 9, 5], 8, 1, 128, 16),
                                               ([0, 40, 70], 4, 2, 128, 64), ([0, 90, 33], 8, 1, 64, 32), ([0, 40, 7], 4, 2, 192, 16)])
@pytest.mark.parametrize("prefix", [368, 700])
def test_a_prefix_behind_all_rows(w8, counts, Hq, Hkv, D, P, prefix):
    check(Case([prefix, 242, 100], counts, Hq, Hkv, D, P, "bf16", seed=prefix + D), w8, Span(prefix=prefix), 3)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), -1.0, 0.0])
def test_scales_of_any_value_there(w8, value):
    for counts, Hq in (([0, 2, 1], 4), ([0, 60, 20], 8)):
        case = Case([700, 242, 100], counts, Hq, 2, 128, 32, "f16", seed=21)
        want = check(case, w8, Span(prefix=700), 4)
        case.ks[case.ks.isnan()] = value
        case.vs[case.vs.isnan()] = value
        case.to_gpu(w8)
        out = w8.kv_attention(case.cache, case.q, case.dtable, case.dlens, prefix_pages=torch.from_numpy(case.prefix_pages).cuda(), prefix_len=700,
                              cu_q=case.dcu, max_q=max(counts))
        assert (out.double().cpu().numpy() == want).all()
