"""Calls on a stream of their own that make their outputs and workspaces themselves, while the
current stream goes on allocating: blocks of all sizes that the call could have taken are filled
on the current stream, before the call (by work that is still queued, in blocks already freed) and
right after it (while the call's kernels still wait on their stream). The results must be
those of the same call on the current stream."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    import fp8_weight_only_gemm_gb300 as w8
    from fp8_weight_only_gemm_gb300.build import build_library
    build_library()
    w8.load()
    w8.device_status(clear=True)
    yield w8
    assert w8.device_status(clear=True)[0] == 0


def make_calls(w8):
    g = torch.Generator("cuda").manual_seed(3)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    A, N, K = randn(40, 512).to(torch.bfloat16), 300, 512
    W, S = w8.quantize_weights(randn(N, K))
    W4 = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    S4 = torch.rand(N, K // 64, generator=g, device="cuda")
    wide = randn(N, K)
    a8, s8 = w8.quantize_activations(A)
    terms = w8.split_activations(A)
    cache = w8.KVCache.empty(64, 32, 2, 128)
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(2, 32)
    lens = torch.tensor([1000, 900], dtype=torch.int32, device="cuda")
    k, v = (randn(1800, 2, 128).to(torch.bfloat16) for _ in range(2))
    w8.kv_append(cache, k, v, table, lens)
    cos = torch.rand(1000, 64, generator=g, device="cuda")
    q1, q40 = (randn(2 * t, 8, 128).to(torch.bfloat16) for t in (1, 40))
    return {
        "gemm": lambda s: w8.gemm(A, W, S, stream=s),
        "gemm_ws": lambda s: w8.gemm_ws(A, W, S, stream=s),
        "gemm_noalloc": lambda s: w8.gemm_noalloc(A, W, S, stream=s),
        "split_activations": lambda s: w8.split_activations(A, stream=s)[:2 * 40 * K],      # the codes: all are written
        "gemm_split_terms": lambda s: w8.gemm_split_terms(terms, 40, W, S, stream=s),
        "quantize_weights": lambda s: w8.quantize_weights(wide, stream=s),
        "quantize_activations": lambda s: w8.quantize_activations(A, stream=s),
        "gemm_w8a8": lambda s: w8.gemm_w8a8(a8, s8, W, S, stream=s),
        "gemm_w4": lambda s: w8.gemm_w4(A, W4, S4, stream=s),
        "kv_append": lambda s: w8.kv_append(cache, k[:80], v[:80], table, lens, cos, cos, q=q40, stream=s),
        "kv_attention, few rows": lambda s: w8.kv_attention(cache, q1, table, lens, stream=s),
        "kv_attention, many rows": lambda s: w8.kv_attention(cache, q40, table, lens, stream=s),
    }


NAMES = ["gemm", "gemm_ws", "gemm_noalloc", "split_activations", "gemm_split_terms", "quantize_weights", "quantize_activations", "gemm_w8a8",
         "gemm_w4", "kv_append", "kv_attention, few rows", "kv_attention, many rows"]
SIZES = [2 ** i for i in range(9, 26)]


def fill_blocks():
    return [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in SIZES for _ in range(2)]


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_own_allocations_on_another_stream(w8, name, as_handle):
    call = make_calls(w8)[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for delay_current, delay_side in ((20_000_000, 0), (0, 20_000_000)):
        if delay_current:
            torch.cuda._sleep(delay_current)
        fill_blocks()                         # queued behind the delay, and freed at once
        if delay_side:
            with torch.cuda.stream(side):
                torch.cuda._sleep(delay_side)
        got = call(side.cuda_stream if as_handle else side)
        after = fill_blocks()
        torch.cuda.synchronize()
        for x, y in zip(*((t if isinstance(t, tuple) else (t,)) for t in (got, want))):
            assert torch.equal(x, y)
        del after
