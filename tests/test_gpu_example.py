"""The example block against its FP32 form with an unquantised cache.

Tolerance: E4M3 rounds a key or value by at most 2^-4 of itself (page scales are powers of
two, so values near the page's maximum keep that), with an RMS of about 0.6 * 2^-4 / sqrt(3)
= 0.022 for values spread over a binade. Scores stay below 2 here, so their error moves the
weights by about as much; with the 16-bit roundings of q, k, v and the outputs (2^-9 each)
the output's relative RMS error is bounded by twice that, 0.045."""
from __future__ import annotations

import importlib.util
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu


def load():
    spec = importlib.util.spec_from_file_location("attention_block", Path(__file__).parent.parent / "examples" / "attention_block.py")
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("batch,prompt,chunk,steps", [(2, 300, 192, 9), (1, 1, 1, 3), (5, 70, 64, 5)])
def test_block(batch, prompt, chunk, steps):
    from fp8_weight_only_gemm_gb300.build import build_library
    build_library()
    torch.manual_seed(1)
    got, want, _ = load().run(batch, prompt, chunk, steps, hidden=1024, heads=8, kv_heads=2)
    err = ((got.float() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)).max().item()
    assert err < 0.045, err
    per_token = (got.float() - want).norm(dim=2) / want.norm(dim=2)
    assert per_token.max().item() < 4 * 0.045


def test_calls_queued_behind_each_other():
    """Chunks queued without waiting overlap at their ends (dependent launches): the waits inside
    the kernels meet other timings than one call at a time, and the results must be the same."""
    import fp8_weight_only_gemm_gb300 as w8
    m = load()
    batch, total, chunk = 32, 1000, 96
    results = []
    for synced in (True, False, False):
        block = m.AttentionBlock(batch, total, hidden=1024, heads=8, kv_heads=2)
        torch.manual_seed(2)
        x = torch.randn(batch, total, 1024, device="cuda").to(torch.bfloat16)
        outs = []
        for at in range(0, total, chunk):
            outs.append(block.forward(x[:, at:at + chunk].reshape(-1, 1024)))
            if synced:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert w8.device_status(clear=True)[0] == 0
        results.append(torch.cat(outs))
    assert torch.equal(results[0], results[1]) and torch.equal(results[0], results[2])
