"""Attention over the 8-bit paged cache against the plain 64-bit form.

Tolerance, from the arithmetic. Write the output as a weighted mean o = sum w_j v_j / sum w_j and
A = sum w_j |v_j| / sum w_j.
  weights   rounded once to FP16 (unit roundoff 2^-11): <= 2^-11 A;
  scores    FP32 sums of exact products, at most 256 + 16 terms: each logit off by at most
            2^-15 X with X = c ks sum_d |q_d k_d| (272 roundings of 2^-24), plus 2^-21 of the
            row maximum's terms for query elements below 2^-21 of it, plus 2^-22 |y| for its
            scaling: a relative error of a weight of at most 2^-14 X (numerator and
            denominator together: twice);
  exp2      hardware 2^x: 2^-22 relative, and sums over n keys in FP32: (n / 64 + 64) 2^-24
            in the order used (64-key units, then parts);
  output    rounded to the activation type: u |o|, u = 2^-8 (BF16), 2^-11 (FP16).
The bound below takes 2^-11 + 2^-13 (1 + X_max) + (n / 64 + 64) 2^-23 for the factor of A.
Rows that see no key are exactly zero."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_reference as ref
from test_gpu_kv_append import Case, DT

pytestmark = pytest.mark.gpu
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def w8():
    import fp8_weight_only_gemm_gb300 as w8
    from fp8_weight_only_gemm_gb300.build import build_library
    build_library()
    w8.load()
    w8.device_status(clear=True)
    yield w8
    assert w8.device_status(clear=True)[0] == 0


def finite_cache(case, seed, pow2=True):
    """Codes without NaN inside the sequences, scales of everyday size; NaN codes and
    huge scales everywhere else."""
    g = torch.Generator().manual_seed(seed)
    shape = case.kc.shape
    for name in ("kc", "vc"):
        x = (torch.randn(shape, generator=g) * 100.0).clamp(-448, 448)
        c = x.to(torch.float8_e4m3fn).view(torch.uint8)
        view = c.transpose(1, 2) if case.slot_major else c            # [pages, H, P, D]
        used = torch.zeros(view.shape[0], view.shape[2], dtype=torch.bool)
        for b, n in enumerate(case.lens):
            for pos in range(n):
                used[int(case.table[b, pos // case.P]), pos % case.P] = True
        view[~used[:, None, :, None].expand(view.shape)] = 0x7F
        setattr(case, name, c)
        case_used = used.any(1)
        s = torch.rand(view.shape[:2], generator=g) * 0.01 + 0.005
        if pow2:
            s = 2.0 ** torch.randint(-9, -5, view.shape[:2], generator=g).float()
        s[~case_used] = float("nan")
        setattr(case, "ks" if name == "kc" else "vs", s)


def reference(case, q, scale):
    """(out, A, X_max, visible) per row."""
    st = case.state()
    P, H = st["k"].shape[2], st["k"].shape[1]
    G = q.shape[1] // H
    out, A = np.zeros_like(q), np.zeros_like(q)
    X = np.zeros(q.shape[:2] + (1,))
    n_vis = np.zeros(q.shape[0], dtype=int)
    for b, n in enumerate(case.lens):
        r0, T = case.cu[b], case.cu[b + 1] - case.cu[b]
        if n <= 0 or T == 0:
            continue
        pages = [case.table[b][i] for i in range((n - 1) // P + 1)]
        for h in range(H):
            kk = np.concatenate([ref.E4M3[st["k"][p, h]] * st["k_scale"][p, h] for p in pages])
            vv = np.concatenate([ref.E4M3[st["v"][p, h]] * st["v_scale"][p, h] for p in pages])
            for t in range(T):
                end = n - T + t + 1
                if end <= 0:
                    continue
                n_vis[r0 + t] = end
                for gq in range(G):
                    qq = q[r0 + t, h * G + gq]
                    x = kk[:end] @ qq * scale
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    out[r0 + t, h * G + gq] = w @ vv[:end]
                    A[r0 + t, h * G + gq] = w @ np.abs(vv[:end])
                    X[r0 + t, h * G + gq] = (np.abs(kk[:end]) @ np.abs(qq)).max() * scale
    return out, A, X, n_vis


def check(case, w8, uniform=False, scale=None, q_scale=1.0, **kw):
    case.qkv = (case.qkv.float() * q_scale).to(case.qkv.dtype)
    case.to_gpu(w8)
    ragged = {} if uniform else {"cu_q": case.dcu, "max_q": max(case.counts)}
    out = w8.kv_attention(case.cache, case.q, case.dtable, case.dlens, softmax_scale=scale, **ragged, **kw)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    q = case.np_qkv()[0]
    want, A, X, n = reference(case, q, scale if scale else case.D ** -0.5)
    tol = U[case.dtype] * np.abs(want) + A * (2.0 ** -11 + 2.0 ** -13 * (1 + X) + (n[:, None, None] / 64 + 64) * 2.0 ** -23) + 1e-30
    if case.dtype == "f16":
        tol = tol + 2.0 ** -25                            # FP16 subnormal outputs
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want) / tol)} of the bound"
    assert np.all(got[n == 0] == 0)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hq,Hkv,P", [(128, 8, 2, 16), (64, 4, 4, 32), (256, 2, 1, 64), (80, 7, 1, 16), (96, 6, 2, 128),
                                        (16, 1, 1, 16), (128, 40, 1, 64), (192, 3, 3, 256)])
def test_single_tokens(w8, D, Hq, Hkv, P, dtype):
    case = Case([1, 16, 17, 63, 64, 65, 1000, 0], [1] * 8, Hq, Hkv, D, P, dtype, seed=D + P)
    finite_cache(case, 1)
    check(case, w8, uniform=True)


@pytest.mark.parametrize("slot_major,fused", [(False, False), (True, True)])
def test_several_tokens(w8, slot_major, fused):
    # ragged rows: causal edges inside pages, more tokens than the sequence has (padding), none
    case = Case([300, 5, 129, 40, 64, 7], [5, 5, 33, 0, 64, 9], 6, 2, 128, 32, "bf16", seed=4, slot_major=slot_major, fused=fused)
    finite_cache(case, 2)
    check(case, w8)


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16"), (256, "bf16")])
def test_prompt_chunks(w8, D, dtype):
    case = Case([401], [150], 4, 2, D, 64, dtype, seed=6)
    finite_cache(case, 3)
    check(case, w8, uniform=True)
    case = Case([203, 77], [203, 76], 2, 2, D, 16, dtype, seed=7)
    finite_cache(case, 4)
    check(case, w8)


def test_long_and_short_together(w8):
    case = Case([9001, 1, 33, 2500], [1, 1, 1, 1], 4, 1, 64, 16, "bf16", seed=8)
    finite_cache(case, 5)
    check(case, w8, uniform=True)


def test_scales_that_are_no_powers_of_two_and_a_temperature(w8):
    case = Case([500, 90], [2, 2], 4, 2, 128, 32, "bf16", seed=10)
    finite_cache(case, 6, pow2=False)
    check(case, w8, uniform=True, scale=0.25)


def test_sharp_softmax_and_wide_scales(w8):
    """Peaked weights, and value scales that differ by 2^40 between pages."""
    case = Case([400, 130], [1, 1], 4, 2, 64, 16, "bf16", seed=12)
    finite_cache(case, 7)
    g = torch.Generator().manual_seed(1)
    case.vs = torch.where(case.vs.isnan(), case.vs, 2.0 ** torch.randint(-30, 11, case.vs.shape, generator=g).float())
    check(case, w8, uniform=True, q_scale=4.0)


def test_tiny_and_huge_queries(w8):
    for q_scale in (2.0 ** -100, 2.0 ** 60):
        case = Case([100, 30], [1, 1], 2, 1, 128, 16, "bf16", seed=14)
        finite_cache(case, 8)
        check(case, w8, uniform=True, q_scale=q_scale, scale=2.0 ** -64 if q_scale > 1 else 0.1)


def test_nan_reaches_only_the_rows_that_see_it(w8):
    case = Case([70, 40], [6, 6], 4, 2, 64, 16, "bf16", seed=16)
    finite_cache(case, 9)
    page, slot = int(case.table[0, 67 // 16]), 67 % 16      # position 67: rows 3, 4, 5 of sequence 0
    case.vc[page, 1, slot, 10] = 0xFF
    page2, slot2 = int(case.table[1, 38 // 16]), 38 % 16    # position 38: rows 4, 5 of sequence 1
    case.kc[page2, 0, slot2, 3] = 0x7F
    case.qkv[0, 1, 2] = float("nan")
    case.to_gpu(w8)
    out = w8.kv_attention(case.cache, case.q, case.dtable, case.dlens)
    nan = out.isnan().cpu()
    want = torch.zeros_like(nan)
    want[3:6, 2:4, 10] = True
    want[10:12, 0:2, :] = True
    want[0, 1, :] = True
    assert torch.equal(nan, want)
    assert w8.device_status(clear=True)[0] == 0


def test_repeatable_workspace_stream_and_strides(w8):
    case = Case([3000, 700], [3, 3], 8, 2, 128, 16, "f16", seed=18, fused=True)
    finite_cache(case, 10)
    got = check(case, w8, uniform=True)
    ws = torch.full((w8.kv_attention_workspace_bytes(case.cache, 2, 3, 8),), 0xFF, dtype=torch.uint8, device="cuda")
    wide = torch.zeros(6, 8, 144, dtype=torch.float16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w8.kv_attention(case.cache, case.q, case.dtable, case.dlens, wide[:, :, :128], workspace=ws, stream=s)
    s.synchronize()
    assert np.array_equal(wide[:, :, :128].double().cpu().numpy(), got) and wide[:, :, 128:].abs().sum() == 0


def test_captured_graph_serves_growing_lengths(w8):
    case = Case([200, 90], [1, 1], 4, 2, 64, 32, "bf16", seed=20)
    finite_cache(case, 11)
    case.to_gpu(w8)
    ws = torch.empty(w8.kv_attention_workspace_bytes(case.cache, 2, 1, 4), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(case.q)
    lens = case.dlens.clone()
    w8.kv_attention(case.cache, case.q, case.dtable, lens, out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w8.kv_attention(case.cache, case.q, case.dtable, lens, out, workspace=ws)
    for n in ([200, 90], [17, 1], [150, 64]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        w8.kv_attention(case.cache, case.q, case.dtable, lens, out, workspace=ws)
        assert torch.equal(got, out)


def test_bad_indices_are_reported(w8):
    case = Case([20, 40], [1, 1], 2, 1, 64, 16, "bf16", seed=22)
    finite_cache(case, 12)
    case.to_gpu(w8)
    for table, lens in ((case.dtable + 1000, case.dlens), (case.dtable - 1000, case.dlens), (case.dtable, case.dlens + 100000)):
        w8.kv_attention(case.cache, case.q, table, lens)
        assert w8.device_status(clear=True)[0] == 2
    out = w8.kv_attention(case.cache, case.q, case.dtable, case.dlens * 0 - 5)          # negative lengths: no keys
    assert out.abs().sum() == 0 and w8.device_status(clear=True)[0] == 0


def test_refusals(w8):
    case = Case([20, 40], [1, 1], 4, 2, 64, 16, "bf16", seed=24).to_gpu(w8)
    c, q, t, n = case.cache, case.q, case.dtable, case.dlens
    with pytest.raises(TypeError):
        w8.kv_attention(c, q.float(), t, n)
    with pytest.raises(ValueError):
        w8.kv_attention(c, q[:, :, :32], t, n)
    with pytest.raises(ValueError):
        w8.kv_attention(c, q[:1], t, n)                                  # rows do not divide
    with pytest.raises(ValueError):
        w8.kv_attention(c, q, t, n, cu_q=case.dcu)                       # max_q missing
    with pytest.raises(ValueError):
        w8.kv_attention(c, q, t, n, torch.empty(2, 4, 64, dtype=torch.bfloat16))
    with pytest.raises(w8.W8A16Error):
        w8.kv_attention(c, q[:, :3], t, n)                               # 3 heads over 2
    with pytest.raises(w8.W8A16Error):
        w8.kv_attention(c, q, t, n, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(w8.W8A16Error):
            w8.kv_attention(c, q, t, n, softmax_scale=bad)


@pytest.mark.parametrize("D,Hq,Hkv,dtype", [(128, 8, 1, "bf16"), (64, 4, 4, "f16"), (112, 6, 2, "bf16"), (16, 2, 1, "f16")])
def test_many_rows_ragged(w8, D, Hq, Hkv, dtype):
    """Row blocks that are full, ragged and single-tiled, items split between CTAs, padding
    rows, sequences without rows or keys."""
    case = Case([700, 1200, 300, 64, 0, 257], [130, 257, 300, 0, 3, 90], Hq, Hkv, D, 32, dtype, seed=D)
    finite_cache(case, 30)
    check(case, w8)


def test_many_rows_long_context(w8):
    case = Case([20011], [70], 4, 1, 128, 64, "bf16", seed=31)
    finite_cache(case, 31)
    check(case, w8, uniform=True)
    case = Case([3001, 2999], [40, 40], 4, 2, 64, 16, "f16", seed=32)
    finite_cache(case, 32, pow2=False)
    check(case, w8, uniform=True, scale=0.5)


def test_many_rows_sharp_softmax_and_wide_scales(w8):
    case = Case([900, 500], [100, 100], 2, 2, 64, 16, "bf16", seed=33)
    finite_cache(case, 33)
    g = torch.Generator().manual_seed(1)
    case.vs = torch.where(case.vs.isnan(), case.vs, 2.0 ** torch.randint(-30, 11, case.vs.shape, generator=g).float())
    check(case, w8, uniform=True, q_scale=4.0)


def test_many_rows_nan_reaches_only_the_rows_that_see_it(w8):
    case = Case([300, 150], [150, 150], 2, 1, 64, 16, "bf16", seed=34)
    finite_cache(case, 34)
    for b, pos, d in ((0, 250, 10), (0, 20, 11), (1, 149, 12), (1, 0, 13)):
        case.vc[int(case.table[b, pos // 16]), 0, pos % 16, d] = 0x7F
    case.kc[int(case.table[0, 290 // 16]), 0, 290 % 16, 5] = 0xFF
    case.qkv[7, 1, 2] = float("-inf")
    case.to_gpu(w8)
    out = w8.kv_attention(case.cache, case.q, case.dtable, case.dlens)
    nan = out.isnan().cpu()
    want = torch.zeros_like(nan)
    want[100:150, :, 10] = True                  # row t of sequence 0 has position 150 + t
    want[:150, :, 11] = True
    want[140:150] = True
    want[299, :, 12] = True
    want[150:, :, 13] = True
    want[7, 1] = True
    assert torch.equal(nan, want)
    assert w8.device_status(clear=True)[0] == 0


def test_many_rows_repeatable_strides_and_graph(w8):
    case = Case([1000, 600], [80, 80], 4, 2, 128, 16, "bf16", seed=35, slot_major=True, fused=True)
    finite_cache(case, 35)
    got = check(case, w8, uniform=True)
    ws = torch.full((w8.kv_attention_workspace_bytes(case.cache, 2, 80, 4),), 0xFF, dtype=torch.uint8, device="cuda")
    wide = torch.zeros(160, 4, 136, dtype=torch.bfloat16, device="cuda")
    w8.kv_attention(case.cache, case.q, case.dtable, case.dlens, wide[:, :, :128], workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w8.kv_attention(case.cache, case.q, case.dtable, case.dlens, wide[:, :, :128], workspace=ws)
    wide.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(wide[:, :, :128].double().cpu().numpy(), got) and wide[:, :, 128:].abs().sum() == 0
    bad = w8.kv_attention(case.cache, case.q, case.dtable + 100000, case.dlens)
    assert bad.shape == case.q.shape and w8.device_status(clear=True)[0] == 2


@pytest.mark.parametrize("count,Hq", [(1, 4), (10, 8)])
def test_more_sequences_than_threads(w8, count, Hq):
    # 300 sequences: both kernels count the work of a block of them at a time
    g = torch.Generator().manual_seed(count)
    lens = (torch.randint(0, 70, (300,), generator=g) + count - 1).tolist()
    lens[7] = lens[299] = 0
    case = Case(lens, [count if n else 0 for n in lens], Hq, 2, 64, 16, "bf16", seed=41)
    finite_cache(case, 41)
    check(case, w8)
