"""The quantised norm's codes: E4M3 round to nearest even of the FP32 quotient y / scale with scale = amax / 448 rounded to
FP32, the rule of quantize_activations, also where the quotient lies next to the middle between two codes and where the scale is
subnormal. Rows of ones have mean square 1, so y is the weight, exactly: codes and scales are equal to the rule's, with no tolerance."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_reference as ref

pytestmark = pytest.mark.gpu
MIDDLES = (ref.E4M3[:126] + ref.E4M3[1:127]) / 2      # between the codes of 0 .. 448


@pytest.fixture(scope="module", autouse=True)
def w8():
    import fp8_weight_only_gemm_gb300 as w8
    from fp8_weight_only_gemm_gb300.build import build_library
    build_library()
    w8.load()
    return w8


def weights(groups, lo, hi, steps, seed):
    """[groups, 128]: a group's maximum, of magnitude 448 * 10^(lo .. hi), a zero, and values `steps` FP32 steps and fewer from its
    scale times a middle between codes."""
    g = np.random.default_rng(seed)
    top = (448.0 * 10.0 ** g.uniform(lo, hi, groups)).astype(np.float32)
    scale = (top / np.float32(448)).astype(np.float32)
    w = np.zeros((groups, 128), np.float32)
    w[:, 1] = top
    near = (MIDDLES[None, :] * scale[:, None].astype(np.float64)).astype(np.float32)
    near = (near.view(np.int32) + g.integers(-steps, steps + 1, near.shape).astype(np.int32) * (near > 0)).clip(0).view(np.float32)
    w[:, 2:] = np.minimum(near, top[:, None])
    return w * g.choice(np.array([-1, 1], np.float32), w.shape), scale


def check(w8, w, scale, M, kind="rms"):
    H = w.size
    x = torch.ones(M, H, dtype=torch.bfloat16, device="cuda")
    if kind == "layer":
        x[:, ::2] = -1
        w = w * np.tile(np.array([-1, 1], np.float32), 64)
    (codes, scales), _ = w8.norm_residual(x, None, torch.from_numpy(w.reshape(-1)).cuda(), eps=0.0, kind=kind, quantize=True)
    if kind == "layer":
        w = w * np.tile(np.array([-1, 1], np.float32), 64)
    codes, scales = codes.cpu().numpy().reshape(M, -1, 128), scales[:, :M].t().cpu().numpy()
    assert np.array_equal(scales, np.broadcast_to(scale, scales.shape))
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        q = np.where(scale[:, None] > 0, w / scale[:, None], np.float32(0))
    assert q.dtype == np.float32
    want = np.where(scale[:, None] > 0, ref.e4m3_encode(q), 0).astype(np.uint8)
    zero = (want & 0x7F) == 0                                    # of either sign
    wrong = (codes != want[None]) & ~(zero[None] & ((codes & 0x7F) == 0))
    assert not wrong.any(), f"{wrong.sum()} of {wrong.size} codes, first {np.argwhere(wrong)[:4].tolist()}"


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("M,H", [(1, 512), (3, 512), (2, 4096), (2, 16384), (330, 8192)])
def test_codes_next_to_a_middle(w8, M, H, kind):
    check(w8, *weights(H // 128, -3, 3, 3, seed=M + H), M, kind)


@pytest.mark.parametrize("lo,hi", [(-33, -32), (-38, -36), (-41, -38), (-45.5, -41)])
def test_codes_of_tiny_groups(w8, lo, hi):
    check(w8, *weights(128, lo, hi, 3, seed=int(-lo)), 2)


def test_codes_of_huge_groups(w8):
    check(w8, *weights(64, 33, 35.8, 3, seed=9), 2)
