"""Padding rows of attention (more rows than the sequence has tokens) give zeros whatever they
hold: their queries are filled with NaN and infinities, as rows that no one has written may be.
The other rows must have the bits that they have beside finite padding. Row blocks of padding
alone, shared with real rows, and split between CTAs, in the kernels for few and for many
query rows a key/value head."""
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


# lengths, rows of the call, query heads, key/value heads, head size
FORMS = {
    "few, 8 rows": ([3, 100, 1, 4], [8, 8, 8, 8], 2, 2, 64),
    "few, 16 rows and groups": ([9, 2, 300], [10, 9, 1], 6, 2, 128),
    "few, tiles of padding alone": ([5, 31], [32, 32], 1, 1, 128),
    "few, split items": ([200, 70], [250, 90], 2, 1, 256),
    "many, one tile": ([30, 90], [40, 50], 4, 2, 64),
    "many, blocks of padding alone and split items": ([300, 40, 700], [900, 300, 130], 2, 2, 128),
    "many, small heads": ([130], [400], 8, 1, 16),
}


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("form", FORMS)
def test_rows_without_keys_are_zero_whatever_they_hold(w8, form, fill):
    lens, counts, Hq, Hkv, D = FORMS[form]
    case = Case(lens, counts, Hq, Hkv, D, 16, "bf16", seed=D + len(lens))
    finite_cache(case, 51)
    finite = check(case, w8)
    padding = torch.zeros(case.q.shape[0], dtype=torch.bool)
    for b, (n, T) in enumerate(zip(lens, counts)):
        padding[case.cu[b]:case.cu[b] + max(T - n, 0)] = True
    assert padding.any()
    q = case.q.clone()
    q[padding.cuda(), :, ::3] = fill
    q[padding.cuda(), 0] = fill
    out = w8.kv_attention(case.cache, q, case.dtable, case.dlens, cu_q=case.dcu, max_q=max(counts)).double().cpu()
    assert torch.equal(out[padding], torch.zeros_like(out[padding]))
    assert torch.equal(out, torch.from_numpy(finite))
