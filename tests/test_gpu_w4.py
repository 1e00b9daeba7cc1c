"""The product with 4-bit weights and group scales against the plain 64-bit form.

Tolerance, from the arithmetic. Products a * code (or a * (code - zero)) are exact in the
tensor core's FP32 sums; a group's sum has at most 128 terms, and so has the sum of its
activations, which the zero point multiplies; groups add in FP32 (a few multiply-adds per
group part, K / 32 of them at most), then up to 32 parts in a CTA and 8 CTAs. With
B = sum_k |A| (code + zero) |scale| each of these roundings is at most 2^-23 B (the
tensor core may truncate), 128 + K / 32 + 44 of them; the result rounds once to the
activation type (2^-8 |C| for BF16, 2^-11 for FP16, and 2^-25 for FP16 subnormals)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def w8():
    import fp8_weight_only_gemm_gb300 as w8
    from fp8_weight_only_gemm_gb300.build import build_library
    build_library()
    w8.load()
    yield w8


def make(M, N, K, group, dtype, zeros, f32, seed, lda_pad=0):
    g = torch.Generator().manual_seed(seed)
    A = torch.randn(M, K + lda_pad, generator=g).to(DT[dtype])
    W = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scale = (torch.randn(N, K // group, generator=g) * 0.01).to(torch.float32 if f32 else DT[dtype])
    z = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8) if zeros else None
    return A, W, scale, z


def reference(A, W, scale, z, group):
    codes = np.stack((W.numpy() & 15, W.numpy() >> 4), -1).reshape(W.shape[0], -1).astype(np.float64)
    zero = np.repeat(z.numpy().astype(np.float64), group, 1) if z is not None else 8.0
    s = np.repeat(scale.double().numpy(), group, 1)
    a = A.double().numpy()[:, :codes.shape[1]]
    return a @ ((codes - zero) * s).T, np.abs(a) @ ((codes + zero) * np.abs(s)).T


def check(w8, M, N, K, group, dtype, zeros, f32, seed=0, lda_pad=0, ldc_pad=0, flags=0):
    A, W, scale, z = make(M, N, K, group, dtype, zeros, f32, seed, lda_pad)
    C = torch.full((M, N + ldc_pad), 7.0, dtype=DT[dtype], device="cuda")
    out = w8.gemm_w4(A.cuda()[:, :K], W.cuda(), scale.cuda(), C, zeros=None if z is None else z.cuda(), flags=flags)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    want, B = reference(A, W, scale, z, group)
    tol = U[dtype] * np.abs(want) + (128 + K / 32 + 44) * 2.0 ** -23 * B + (2.0 ** -25 if dtype == "f16" else 0.0)
    bad = ~(np.abs(got[:, :N] - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.max(np.abs(got[:, :N] - want) / tol)} of the bound"
    assert np.all(got[:, N:] == 7.0)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_types_and_groups(w8, group, zeros, f32, dtype):
    # odd group counts put 16-bit scale rows and zero rows at every alignment
    check(w8, 3, 200, 5 * 128 + group, group, dtype, zeros, f32, seed=group)
    check(w8, 1, 67, 3 * group, group, dtype, zeros, f32, seed=group + 1, lda_pad=8, ldc_pad=1)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 70])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (129, 544, 32), (1000, 2048, 128), (4097, 1088, 64)])
def test_token_counts_and_ragged_rows(w8, M, N, K, group):
    check(w8, M, N, K, group, "bf16", True, False, seed=M + N, lda_pad=40, ldc_pad=3)


@pytest.mark.parametrize("M", [9, 16])
def test_more_rows_than_tiles_at_once(w8, M):
    check(w8, M, 9763, 544, 32, "bf16", True, False, seed=M, lda_pad=8, ldc_pad=5)
    check(w8, M, 9763, 320, 64, "f16", False, True, seed=M)


@pytest.mark.parametrize("M", [17, 32, 33, 70])
def test_larger_products(w8, M):
    check(w8, M, 9763, 1600, 32, "bf16", True, False, seed=M, lda_pad=8, ldc_pad=5)
    check(w8, M, 9763, 1664, 128, "f16", True, True, seed=M + 1)
    check(w8, M, 9763, 1600, 64, "bf16", False, True, seed=M + 2)


@pytest.mark.parametrize("N,K", [(64, 8192), (256, 28672), (28672, 256), (512, 4096)])
def test_long_and_wide(w8, N, K):
    for M in (1, 12, 32):
        check(w8, M, N, K, 128, "f16", False, True, seed=N)


def test_flag_stream_and_repeatability(w8):
    a = check(w8, 5, 1000, 4096, 64, "bf16", True, True, seed=3)
    b = check(w8, 5, 1000, 4096, 64, "bf16", True, True, seed=3, flags=w8.FLAG_PDL)
    assert np.array_equal(a, b)
    A, W, scale, z = (t.cuda() for t in make(5, 1000, 4096, 64, "bf16", True, True, 3))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    C = w8.gemm_w4(A, W, scale, zeros=z, stream=s)
    s.synchronize()
    assert np.array_equal(C.double().cpu().numpy(), a)


def test_back_to_back_calls_feed_each_other(w8):
    """The second call's input is the first one's output, with and without the flag."""
    A, W, scale, _ = make(4, 512, 512, 64, "bf16", False, True, 5)
    for flags in (0, w8.FLAG_PDL):
        x = A.cuda()
        Wd, sd = W.cuda(), scale.cuda()
        for _ in range(20):
            x = w8.gemm_w4(x, Wd, sd, flags=flags)
        y = A.cuda()
        for _ in range(20):
            y = w8.gemm_w4(y, Wd, sd)
            torch.cuda.synchronize()
        assert torch.equal(x, y)


def test_nonfinite_activations_stay_in_their_row(w8):
    A, W, scale, _ = make(4, 100, 256, 32, "bf16", False, True, 6)
    A[1, 3] = float("inf")
    A[2, 200] = float("nan")
    W[:, 1] = 0x99                                        # codes 2, 3: code - 8 = 1, so the infinity is seen
    C = w8.gemm_w4(A.cuda(), W.cuda(), scale.cuda()).cpu()
    assert not torch.isfinite(C[1]).any() and C[2].isnan().all()
    assert torch.isfinite(C[0]).all() and torch.isfinite(C[3]).all()


def test_refusals(w8):
    A, W, scale, z = (t.cuda() for t in make(2, 64, 256, 64, "bf16", True, True, 7))
    with pytest.raises(TypeError):
        w8.gemm_w4(A.float(), W, scale)
    with pytest.raises(TypeError):
        w8.gemm_w4(A, W, scale.half())
    with pytest.raises(ValueError):
        w8.gemm_w4(A[:, :128], W, scale)
    with pytest.raises(ValueError):
        w8.gemm_w4(A, W, scale[:32])
    with pytest.raises(ValueError):
        w8.gemm_w4(A, W, scale, zeros=z[:, :1])
    with pytest.raises(ValueError):
        w8.gemm_w4(A, W, scale, torch.empty(2, 60, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        w8.gemm_w4(A, W.cpu(), scale)
    with pytest.raises(w8.W8A16Error):
        w8.gemm_w4(A, W, scale[:, :1].contiguous())       # group 256
    with pytest.raises(w8.W8A16Error):
        w8.gemm_w4(A, W, scale, flags=64)
    with pytest.raises(w8.W8A16Error):
        w8.gemm_w4(torch.empty(2, 260, dtype=torch.bfloat16, device="cuda")[:, 4:], W, scale)   # alignment


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 5, 20])
def test_nonfinite_scales_stay_in_their_column(w8, M, group):
    K = 9 * group   # the last stage of K is not full
    A, W, scale, z = make(M, 40, K, group, "bf16", True, True, seed=M)
    scale[7, -1] = float("inf")
    scale[30, 2] = float("nan")
    got = w8.gemm_w4(A.cuda(), W.cuda(), scale.cuda(), zeros=z.cuda()).double().cpu().numpy()
    assert not np.isfinite(got[:, [7, 30]]).any()
    assert np.isfinite(np.delete(got, [7, 30], 1)).all()
