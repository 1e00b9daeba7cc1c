"""How far below its neighbours an activation keeps all of its bits with one or two tokens, where a
chunk of 32 becomes FP16 times one power of two: 2^-31 of the largest (BF16) or 2^-28 (FP16) at even positions
of K, 2^-27 or 2^-24 at odd ones. The largest has code and zero point 0, so each output is one
product of a full significand, which must come back exactly; with more tokens nothing is lost at all."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
# significand bits and the stated exponents (even, odd positions)
TYPES = {"bf16": (torch.bfloat16, 8, 31, 27), "f16": (torch.float16, 11, 28, 24)}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 2, 5, 24])
def test_small_beside_large(dtype, M):
    import fp8_weight_only_gemm_gb300 as w8
    from fp8_weight_only_gemm_gb300.build import build_library
    build_library()
    dt, bits, even, odd = TYPES[dtype]
    K, group = 256, 32
    top = 0 if dtype == "bf16" else 14               # (FP16: its normal numbers must reach 2^-28 of the largest)
    full = 2.0 - 2.0 ** (1 - bits)                   # all bits set
    A = torch.zeros(M, K, dtype=torch.float64)
    A[:, 0::32] = 2.0 ** top
    for k in range(K):
        if k % 32:
            A[:, k] = full * 2.0 ** (top - (odd if k % 2 else even))
    # weight row k picks position k: code 1 there, 0 elsewhere
    codes = torch.eye(K, dtype=torch.uint8)
    W = codes[:, 0::2] | codes[:, 1::2] << 4
    zeros = torch.zeros(K, K // group, dtype=torch.uint8)
    scale = torch.full((K, K // group), 2.0 ** -top, dtype=torch.float32)
    if dtype == "f16":
        scale *= 2.0 ** 20                           # outputs back among FP16's normal numbers
        keep = [k for k in range(K) if k % 32]
    else:
        keep = list(range(K))
    a = A.to(dt)
    assert torch.equal(a.double(), A)
    C = w8.gemm_w4(a.cuda(), W.contiguous().cuda(), scale.cuda(), zeros=zeros.cuda()).double().cpu()
    want = A * scale[0, 0].double()
    assert torch.equal(C[:, keep], want[:, keep])
