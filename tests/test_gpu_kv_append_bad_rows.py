"""A token whose row of the rotary table does not exist: its query is left as it was, the dims that are not rotated too,
and the status holds the value that was out of range."""
from __future__ import annotations

import pytest
import torch

import kv_reference as ref
from test_gpu_kv_append import Case

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


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("count,bad", [(1, 50), (2, -1), (20, 1 << 30), (20, -(1 << 31))])
def test_an_axis_outside_the_table(w8, count, bad, interleaved):
    cos, sin = (t.cuda() for t in ref.rope_table(50, 32))
    case = Case([40, 60], [count, count], 6, 2, 128, 16, "bf16", seed=13).to_gpu(w8)
    pos = torch.randint(0, 50, (3, 2 * count), generator=torch.Generator().manual_seed(count), dtype=torch.int32)
    pos[1, count - 1] = bad                               # the last token of sequence 0
    out = torch.full_like(case.q, 7.0)
    w8.kv_append(case.cache, case.k, case.v, case.dtable, case.dlens, cos, sin, q=case.q, q_out=out, interleaved=interleaved,
                 positions=pos.cuda(), axes=w8.RopeAxes.sections((8, 4, 4)))
    code, _, detail = w8.device_status(clear=True)
    assert (code, detail) == (2, bad % (1 << 32))
    assert (out[count - 1] == 7).all()
    rest = torch.arange(2 * count, device="cuda") != count - 1
    assert torch.equal(out[rest][..., 32:], case.q[rest][..., 32:])


@pytest.mark.parametrize("count", [1, 20])
def test_a_place_outside_the_table(w8, count):
    cos, sin = (t.cuda() for t in ref.rope_table(50, 32))
    case = Case([50, 60], [count, count], 6, 2, 128, 16, "bf16", seed=14).to_gpu(w8)
    out = torch.full_like(case.q, 7.0)
    w8.kv_append(case.cache, case.k, case.v, case.dtable, case.dlens, cos, sin, q=case.q, q_out=out)
    code, _, detail = w8.device_status(clear=True)
    assert code == 2 and 50 <= detail < 60
    past = torch.arange(2 * count, device="cuda") >= count + max(0, count - 10)     # positions 50 .. 59 of sequence 1
    assert (out[past] == 7).all()
    assert torch.equal(out[~past][..., 32:], case.q[~past][..., 32:])
